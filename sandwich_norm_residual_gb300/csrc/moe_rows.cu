// Host side of what lies around the experts' products: tokens sorted by expert and back, the
// activation between the products. Argument checks (before any CUDA call) and the launches.
#include "moe_rows.cuh"
#include "swiglu.cuh"

#include <initializer_list>

#include "beam_boundary.h"
#include "device.h"
#include "host.h"

static_assert(BEAM_MOE_MAX_EXPERTS <= beam::kSortMaxExperts && beam::kSortMaxExperts <= beam::kSortThreads &&
                  BEAM_ROUTE_MAX_TOPK <= 16,
              "an expert a thread, the choices of a token in half a warp");

namespace {

using beam::misaligned;
using beam::overlaps;
using beam::RowsParams;
using beam::SortParams;

// Pairs of a block: one block up to 4096 pairs, where it takes one kernel; then 2048 at
// least and no more than 128 blocks, whose counts every block adds up.
void split(int64_t pairs, SortParams* p) {
    p->chunk = pairs;
    p->blocks = 1;
    if (pairs <= 4096) return;
    int64_t blocks = (pairs + 2047) / 2048;
    if (blocks > 128) blocks = 128;
    p->chunk = (pairs + blocks - 1) / blocks;
    p->blocks = (int)((pairs + p->chunk - 1) / p->chunk);
}

beam_status launch(const void* fn, dim3 blocks, int threads, size_t smem, void* p, cudaStream_t stream, bool pdl = false) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = blocks;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {p};
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

struct Span {
    const void* p;
    size_t n;
};

// no output overlaps an input or another output
bool apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    for (const Span* a = out.begin(); a != out.end(); ++a) {
        for (const Span& b : in)
            if (overlaps(a->p, a->n, b.p, b.n)) return false;
        for (const Span* b = out.begin(); b != a; ++b)
            if (overlaps(a->p, a->n, b->p, b->n)) return false;
    }
    return true;
}

bool bad_choices(int64_t T, int topk) {
    return T < 0 || topk < 1 || topk > BEAM_ROUTE_MAX_TOPK || T > BEAM_MOE_MAX_PAIRS / topk;
}

bool bad_rows(int64_t T, int topk, int64_t R, int64_t row_bytes) {
    return bad_choices(T, topk) || R < 0 || R > BEAM_MOE_MAX_PAIRS || row_bytes < 4 || (row_bytes & 3) || row_bytes > 4ll * BEAM_MAX_D;
}

// Warps that share a token: one where there are enough tokens for 16 warps on every SM, else as many as
// have a vector for each lane
void share(RowsParams* p, int sms) {
    const int64_t want = (int64_t)sms * 16;
    int64_t parts = p->T < want ? want / p->T : 1;
    const int64_t most = (p->vecs + 31) / 32;
    p->parts = (int)(parts > most ? most : parts);
}

beam_status launch_rows(const void* fn, const RowsParams& p, cudaStream_t stream) {
    const int64_t warps = p.T * p.parts, each = beam::kRowThreads / 32, blocks = (warps + each - 1) / each;
    return launch(fn, dim3((unsigned)blocks), beam::kRowThreads, 0, const_cast<RowsParams*>(&p), stream);
}

template <class V>
const void* gather_kernel(bool scale16) {
    return scale16 ? reinterpret_cast<const void*>(beam::moe_gather_kernel<V, uint4>)
                   : reinterpret_cast<const void*>(beam::moe_gather_kernel<V, uint32_t>);
}

template <bool F32>
const void* combine_kernel(int topk) {
    return topk <= 2   ? reinterpret_cast<const void*>(beam::moe_combine_kernel<F32, 2>)
           : topk <= 4 ? reinterpret_cast<const void*>(beam::moe_combine_kernel<F32, 4>)
                       : reinterpret_cast<const void*>(beam::moe_combine_kernel<F32, 8>);
}

// the shared end of combine and gather's backward
beam_status combine(beam_stream_t stream, const void* rows, const int32_t* slots, const float* w, bool weighted, int64_t T,
                    int topk, int64_t R, int D, int type, void* out) {
    if (D < 8 || (D & 7) || D > BEAM_MAX_D || bad_rows(T, topk, R, 4)) return BEAM_ERR_SHAPE;
    if (type != BEAM_OUT_BF16 && type != BEAM_OUT_FP32) return BEAM_ERR_ARG;
    if (T == 0) return BEAM_OK;
    if ((R && !rows) || !slots || (weighted && !w) || !out) return BEAM_ERR_NULL;
    if (misaligned(rows, 16) || misaligned(out, 16) || misaligned(slots, 4) || misaligned(w, 4)) return BEAM_ERR_ALIGN;
    const size_t row = (size_t)D * (type == BEAM_OUT_FP32 ? 4u : 2u), cb = (size_t)T * topk * 4u;
    if (!apart({{out, T * row}}, {{rows, R * row}, {slots, cb}, {w, w ? cb : 0}})) return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    RowsParams p{};
    p.slots = slots;
    p.w = w;
    p.T = T;
    p.R = R;
    p.K = topk;
    p.vecs = (int)(row / 16);
    p.rows = rows;
    p.out = out;
    p.status = dev.status_word;
    const int threads = p.vecs >= beam::kCombineThreads ? beam::kCombineThreads : (p.vecs + 31) / 32 * 32;
    // fewer tokens than the device holds blocks: several share one
    const int64_t room = (int64_t)dev.sms * 8, parts = T < room ? room / T : 1, most = (p.vecs + threads - 1) / threads;
    return launch(type == BEAM_OUT_FP32 ? combine_kernel<true>(topk) : combine_kernel<false>(topk),
                  dim3((unsigned)T, (unsigned)(parts < most ? parts : most)), threads, 0, &p, reinterpret_cast<cudaStream_t>(stream));
}

template <bool F32>
const void* backward_kernel(int topk) {
    return topk <= 2   ? reinterpret_cast<const void*>(beam::moe_combine_backward_kernel<F32, 2>)
           : topk <= 4 ? reinterpret_cast<const void*>(beam::moe_combine_backward_kernel<F32, 4>)
           : topk <= 8 ? reinterpret_cast<const void*>(beam::moe_combine_backward_kernel<F32, 8>)
                       : reinterpret_cast<const void*>(beam::moe_combine_backward_kernel<F32, 16>);
}

}  // namespace

extern "C" {

int64_t beam_moe_sort_workspace(int64_t T, int topk, int E) {
    if (bad_choices(T, topk) || E < 1 || E > BEAM_MOE_MAX_EXPERTS) return -1;
    SortParams p{};
    split(T * topk, &p);
    return p.blocks > 1 ? (int64_t)p.blocks * E * 4 : 0;
}

beam_status beam_moe_sort(beam_stream_t stream, const int32_t* topk_idx, int64_t T, int topk, int E, int32_t* offsets,
                          int32_t* slots, void* workspace, int64_t workspace_bytes) {
    const int64_t need = beam_moe_sort_workspace(T, topk, E);
    if (need < 0) return BEAM_ERR_SHAPE;
    if (workspace_bytes < need) return BEAM_ERR_ARG;
    if ((T && (!topk_idx || !slots)) || !offsets || (need && !workspace)) return BEAM_ERR_NULL;
    if (misaligned(topk_idx, 4) || misaligned(offsets, 4) || misaligned(slots, 4) || (need && misaligned(workspace, 16)))
        return BEAM_ERR_ALIGN;
    const size_t cb = (size_t)T * topk * 4u;
    if (!apart({{offsets, ((size_t)E + 1) * 4u}, {slots, cb}, {workspace, (size_t)need}}, {{topk_idx, cb}})) return BEAM_ERR_ALIAS;
    beam::Device dev;
    beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    SortParams p{};
    p.idx = topk_idx;
    p.pairs = T * topk;
    p.E = E;
    split(p.pairs, &p);
    p.counts = static_cast<int32_t*>(workspace);
    p.offsets = offsets;
    p.slots = slots;
    p.status = dev.status_word;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (p.blocks > 1) {
        st = launch(reinterpret_cast<const void*>(beam::moe_count_kernel), p.blocks, beam::kSortThreads, 0, &p, cs);
        if (st != BEAM_OK) return st;
    }
    return launch(reinterpret_cast<const void*>(beam::moe_place_kernel), p.blocks, beam::kSortThreads,
                  (size_t)beam::kSortWarps * E * 4u, &p, cs, p.blocks > 1);
}

beam_status beam_moe_gather(beam_stream_t stream, const void* x, int64_t row_bytes, const void* scale, int64_t scale_bytes,
                            const int32_t* slots, int64_t T, int topk, int64_t R, void* out, void* out_scale) {
    if (bad_rows(T, topk, R, row_bytes) || scale_bytes < 0 || (scale_bytes & 3) || scale_bytes > 4ll * BEAM_MAX_D) return BEAM_ERR_SHAPE;
    if (T == 0) return BEAM_OK;
    if (!x || !slots || (R && !out) || (scale_bytes && (!scale || (R && !out_scale)))) return BEAM_ERR_NULL;
    if (misaligned(x, 4) || misaligned(out, 4) || misaligned(slots, 4) || misaligned(scale, 4) || misaligned(out_scale, 4))
        return BEAM_ERR_ALIGN;
    if (!apart({{out, (size_t)R * row_bytes}, {out_scale, (size_t)R * scale_bytes}},
               {{x, (size_t)T * row_bytes}, {scale, (size_t)T * scale_bytes}, {slots, (size_t)T * topk * 4u}}))
        return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    const bool wide = row_bytes % 16 == 0 && !misaligned(x, 16) && !misaligned(out, 16);
    const bool scale16 = scale_bytes % 16 == 0 && !misaligned(scale, 16) && !misaligned(out_scale, 16);
    RowsParams p{};
    p.slots = slots;
    p.T = T;
    p.R = R;
    p.K = topk;
    p.vecs = (int)(row_bytes / (wide ? 16 : 4));
    p.x = x;
    p.out = out;
    p.scale_vecs = (int)(scale_bytes / (scale16 ? 16 : 4));
    p.scale = scale;
    p.out_scale = out_scale;
    p.status = dev.status_word;
    share(&p, dev.sms);
    return launch_rows(wide ? gather_kernel<uint4>(scale16) : gather_kernel<uint32_t>(scale16), p,
                       reinterpret_cast<cudaStream_t>(stream));
}

beam_status beam_moe_gather_backward(beam_stream_t stream, const void* drows, const int32_t* slots, int64_t T, int topk,
                                     int64_t R, int D, int type, void* dx) {
    return combine(stream, drows, slots, nullptr, false, T, topk, R, D, type, dx);
}

beam_status beam_moe_combine(beam_stream_t stream, const void* rows, const int32_t* slots, const float* topk_w, int64_t T,
                             int topk, int64_t R, int D, int type, void* out) {
    return combine(stream, rows, slots, topk_w, true, T, topk, R, D, type, out);
}

beam_status beam_moe_combine_backward(beam_stream_t stream, const void* dx, const void* rows, const int32_t* slots,
                                      const float* topk_w, int64_t T, int topk, int64_t R, int D, int type, void* drows,
                                      float* dw) {
    if (D < 8 || (D & 7) || D > BEAM_MAX_D || bad_rows(T, topk, R, 4)) return BEAM_ERR_SHAPE;
    if (type != BEAM_OUT_BF16 && type != BEAM_OUT_FP32) return BEAM_ERR_ARG;
    if (T == 0) return BEAM_OK;
    if (!dx || (R && (!rows || !drows)) || !slots || !topk_w || !dw) return BEAM_ERR_NULL;
    if (misaligned(dx, 16) || misaligned(rows, 16) || misaligned(drows, 16) || misaligned(slots, 4) || misaligned(topk_w, 4) ||
        misaligned(dw, 4))
        return BEAM_ERR_ALIGN;
    const size_t row = (size_t)D * (type == BEAM_OUT_FP32 ? 4u : 2u), cb = (size_t)T * topk * 4u;
    if (!apart({{drows, R * row}, {dw, cb}}, {{dx, T * row}, {rows, R * row}, {slots, cb}, {topk_w, cb}})) return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    RowsParams p{};
    p.slots = slots;
    p.w = topk_w;
    p.T = T;
    p.R = R;
    p.K = topk;
    p.vecs = (int)(row / 16);
    p.rows = rows;
    p.dx = dx;
    p.drows = drows;
    p.dw = dw;
    p.status = dev.status_word;
    const int threads = p.vecs >= beam::kBackThreads ? beam::kBackThreads : (p.vecs + 31) / 32 * 32;
    return launch(type == BEAM_OUT_FP32 ? backward_kernel<true>(topk) : backward_kernel<false>(topk), dim3((unsigned)T), threads, 0, &p,
                  reinterpret_cast<cudaStream_t>(stream));
}

beam_status beam_swiglu_fp8(beam_stream_t stream, const uint16_t* gate_up, const int32_t* live_rows, int64_t R, int F,
                            uint8_t* y_fp8, float* y_scale) {
    if (R < 0 || R > BEAM_MOE_MAX_PAIRS || F < 16 || (F & 15) || F > BEAM_MATMUL_MAX_K) return BEAM_ERR_SHAPE;
    if (R == 0) return BEAM_OK;
    if (!gate_up || !y_fp8 || !y_scale) return BEAM_ERR_NULL;
    if (misaligned(gate_up, 16) || misaligned(y_fp8, 8) || misaligned(y_scale, 4) || misaligned(live_rows, 4)) return BEAM_ERR_ALIGN;
    const size_t blocks = ((size_t)F + 127) / 128;
    if (!apart({{y_fp8, (size_t)R * F}, {y_scale, (size_t)R * blocks * 4u}},
               {{gate_up, (size_t)R * F * 4u}, {live_rows, live_rows ? 4u : 0u}}))
        return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    beam::SwigluParams p{};
    p.x = gate_up;
    p.y = y_fp8;
    p.scale = y_scale;
    p.live = live_rows;
    p.R = R;
    p.F = F;
    p.blocks = (int)blocks;
    p.chunks = (F + 255) / 256;
    p.status = dev.status_word;
    const int64_t warps = R * p.chunks, each = beam::kSwigluThreads / 32, most = (int64_t)dev.sms * 8;
    int64_t grid = (warps + each - 1) / each;
    if (grid > most) grid = most;
    return launch(reinterpret_cast<const void*>(beam::swiglu_fp8_kernel), dim3((unsigned)grid), beam::kSwigluThreads, 0, &p,
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
