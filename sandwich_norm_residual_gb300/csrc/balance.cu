// Host side of the router's balance loss: argument checks (before any CUDA
// call), the split into blocks and the launches.
#include "balance.cuh"

#include <cmath>

#include "beam_boundary.h"
#include "device.h"
#include "host.h"

namespace {

using beam::BalanceParams;
using beam::misaligned;
using beam::overlaps;

bool bad_shape(int64_t T, int E, int K, int64_t S, const void* off) {
    return T < 0 || T > 0x7FFFFFFF || E < 4 || (E & 3) || E > BEAM_BALANCE_MAX_EXPERTS || K < 1 ||
           K > BEAM_ROUTE_MAX_TOPK || S < 1 || S > BEAM_BALANCE_MAX_SEQUENCES || (!off && S != 1);
}

// Whether one kernel does it all
bool one_kernel(int64_t T, int E, int64_t S) {
    return T <= beam::kBalanceSmall && T * E <= S * beam::kBalanceSmallLogits;
}

// Tokens a block: at least one for each warp, few enough blocks that two are
// resident on every SM, and at most 64 for each warp, which adds them in FP32
void split(int64_t T, BalanceParams* p) {
    int64_t chunk = (T + beam::kBalanceBlocks - 1) / beam::kBalanceBlocks;
    if (chunk < beam::kBalanceWarps) chunk = beam::kBalanceWarps;
    if (chunk > 64 * beam::kBalanceWarps) chunk = 64 * beam::kBalanceWarps;
    p->chunk = (int)chunk;
    p->blocks = (int)((T + chunk - 1) / chunk);
}

// float4 a lane for E experts: 1, 2 or 4
int vectors(int E) { return E <= 128 ? 1 : E <= 256 ? 2 : 4; }

const void* records_kernel(int E) {
    switch (vectors(E)) {
    case 1: return reinterpret_cast<const void*>(beam::balance_records_kernel<1>);
    case 2: return reinterpret_cast<const void*>(beam::balance_records_kernel<2>);
    default: return reinterpret_cast<const void*>(beam::balance_records_kernel<4>);
    }
}

const void* small_kernel(int E) {
    switch (vectors(E)) {
    case 1: return reinterpret_cast<const void*>(beam::balance_small_kernel<1>);
    case 2: return reinterpret_cast<const void*>(beam::balance_small_kernel<2>);
    default: return reinterpret_cast<const void*>(beam::balance_small_kernel<4>);
    }
}

const void* grad_kernel(int E) {
    switch (vectors(E)) {
    case 1: return reinterpret_cast<const void*>(beam::balance_grad_kernel<1>);
    case 2: return reinterpret_cast<const void*>(beam::balance_grad_kernel<2>);
    default: return reinterpret_cast<const void*>(beam::balance_grad_kernel<4>);
    }
}

beam_status launch(const void* fn, int blocks, int threads, BalanceParams* p, cudaStream_t stream, bool after_records) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = after_records ? 1 : 0;
    void* args[] = {p};
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

}  // namespace

extern "C" {

int64_t beam_moe_balance_workspace(int64_t T, int E, int64_t S) {
    if (bad_shape(T, E, 1, S, &T)) return -1;
    if (one_kernel(T, E, S)) return 0;
    BalanceParams p{};
    split(T, &p);
    return ((int64_t)p.blocks + S) * E * 8;
}

beam_status beam_moe_balance_loss(beam_stream_t stream, const float* logits, const int32_t* topk_idx,
                                  const int32_t* seq_offsets, int64_t T, int E, int topk, int64_t S, float alpha,
                                  float* loss, int32_t* counts, void* workspace, int64_t workspace_bytes) {
    if (bad_shape(T, E, topk, S, seq_offsets)) return BEAM_ERR_SHAPE;
    const int64_t need = beam_moe_balance_workspace(T, E, S);
    if (!std::isfinite(alpha) || workspace_bytes < need) return BEAM_ERR_ARG;
    if ((T && (!logits || !topk_idx)) || !loss || !counts || (need && !workspace)) return BEAM_ERR_NULL;
    if (misaligned(logits, 16) || misaligned(topk_idx, 4) || misaligned(seq_offsets, 4) || misaligned(loss, 4) ||
        misaligned(counts, 16) || (need && misaligned(workspace, 16)))
        return BEAM_ERR_ALIGN;
    const struct {
        const void* p;
        size_t n;
    } in[] = {{logits, (size_t)T * E * 4u}, {topk_idx, (size_t)T * topk * 4u},
              {seq_offsets, seq_offsets ? ((size_t)S + 1) * 4u : 0}},
      out[] = {{loss, (size_t)S * 4u}, {counts, (size_t)S * E * 4u}, {workspace, (size_t)need}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& o : in)
            if (overlaps(out[i].p, out[i].n, o.p, o.n)) return BEAM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return BEAM_ERR_ALIAS;
    }
    beam::Device dev;
    beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    BalanceParams p{};
    p.logits = logits;
    p.idx = topk_idx;
    p.off = seq_offsets;
    p.T = T;
    p.E = E;
    p.K = topk;
    p.S = (int)S;
    p.factor = (double)alpha * E / topk;
    p.loss = loss;
    p.counts = counts;
    p.status = dev.status_word;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (one_kernel(T, E, S)) return launch(small_kernel(E), p.S, beam::kBalanceThreads, &p, cs, false);
    split(T, &p);
    p.rec_q = static_cast<float*>(workspace);
    p.rec_c = reinterpret_cast<int32_t*>(p.rec_q + ((size_t)p.blocks + (size_t)S) * (size_t)E);
    st = launch(records_kernel(E), p.blocks, beam::kBalanceThreads, &p, cs, false);
    if (st != BEAM_OK) return st;
    return launch(reinterpret_cast<const void*>(beam::balance_loss_kernel), p.S, beam::kBalanceFinalThreads, &p, cs, true);
}

beam_status beam_moe_balance_loss_backward(beam_stream_t stream, const float* dloss, const float* logits,
                                           const int32_t* counts, const int32_t* seq_offsets, int64_t T, int E,
                                           int topk, int64_t S, float alpha, float* dlogits) {
    if (bad_shape(T, E, topk, S, seq_offsets)) return BEAM_ERR_SHAPE;
    if (!std::isfinite(alpha)) return BEAM_ERR_ARG;
    if (T == 0) return BEAM_OK;
    if (!dloss || !logits || !counts || !dlogits) return BEAM_ERR_NULL;
    if (misaligned(dloss, 4) || misaligned(logits, 16) || misaligned(counts, 16) || misaligned(seq_offsets, 4) ||
        misaligned(dlogits, 16))
        return BEAM_ERR_ALIGN;
    const size_t rows = (size_t)T * E * 4u;
    if (overlaps(dlogits, rows, logits, rows) || overlaps(dlogits, rows, dloss, (size_t)S * 4u) ||
        overlaps(dlogits, rows, counts, (size_t)S * E * 4u) ||
        (seq_offsets && overlaps(dlogits, rows, seq_offsets, ((size_t)S + 1) * 4u)))
        return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    BalanceParams p{};
    p.logits = logits;
    p.off = seq_offsets;
    p.T = T;
    p.E = E;
    p.K = topk;
    p.S = (int)S;
    split(T, &p);
    p.factor = (double)alpha * E / topk;
    p.counts = const_cast<int32_t*>(counts);
    p.dloss = dloss;
    p.dlogits = dlogits;
    p.status = dev.status_word;
    return launch(grad_kernel(E), p.blocks, beam::kBalanceThreads, &p, reinterpret_cast<cudaStream_t>(stream), false);
}

}  // extern "C"
