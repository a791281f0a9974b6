// Host side of the 8-bit integer product: argument checks (before any CUDA
// call), the choice of the kernel and the launch.
#include "matmul_int8_tc.cuh"

#include <atomic>

#include "beam_boundary.h"
#include "device.h"
#include "host.h"
#include "tensor_map.h"

namespace {

using beam::encode_tiled;
using beam::EncodeTiled;
using beam::MatmulParams;
using beam::misaligned;
using beam::overlaps;
using beam::Shape;

// Kernel for up to 8 tokens, and its channels a warp. At N = 6144, K = 5120 the
// shapes below take 6.5, 7.4, 9.0 and 11.2 us for 1, 2, 4 and 8 tokens; two
// channels a warp take 9.7 and 24 us for 4 and 8, four take 7.2 us for 1, and a
// second set of weights in flight (fewer warps an SM) 8.4 us for 1. The tensor cores'
// tile of 16 tokens takes 14 us there at any of these M. At N = 5120, K = 20480 it
// takes 25 us, these shapes 17, 21, 23 and 36 us for 1, 2, 4 and 8 tokens: from 5
// tokens on a long k would be faster there, but sums are exact here.
template <bool F32>
const void* few_kernel(int64_t M, int* channels) {
    *channels = M <= 2 ? 2 : 4;
    if (M <= 1) return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<1, 2, 4, F32>);
    if (M <= 2) return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<2, 2, 4, F32>);
    if (M <= 4) return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<4, 4, 3, F32>);
    return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<8, 4, 2, F32>);
}

beam_status launch(const void* fn, dim3 grid, dim3 block, void** args, size_t smem, cudaStream_t stream, bool pdl,
                   int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)n;
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

// int8 rows of K in tiles of `rows` by one step of k, 128-byte swizzle
bool row_map(CUtensorMap* map, const int8_t* base, int64_t rows_total, int K, int rows) {
    const EncodeTiled encode = encode_tiled();
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows_total}, strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {beam::kStepK, (cuuint32_t)rows}, unit[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box, unit,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the same for groups of 32 whole rows, taken in the order that the tile kernel's
// wide stores want: place 8 b + 2 j + e of a group holds row 8 j + 2 b + e
bool permuted_map(CUtensorMap* map, const int8_t* base, int64_t rows_total, int K) {
    const EncodeTiled encode = encode_tiled();
    const cuuint64_t k = (cuuint64_t)K;
    const cuuint64_t dims[5] = {k, 2, 4, 4, (cuuint64_t)(rows_total / 32)}, strides[4] = {k, 8 * k, 2 * k, 32 * k};
    const cuuint32_t box[5] = {beam::kStepK, 2, 4, 4, beam::kTileN / 32}, unit[5] = {1, 1, 1, 1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<int8_t*>(base), dims, strides, box, unit,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// raises a kernel's shared-memory limit, once on each device
beam_status allow_smem(const void* fn, size_t bytes, std::atomic<unsigned long long>* done, int device) {
    const unsigned long long bit = 1ull << (device & 63);
    if (done->load(std::memory_order_acquire) & bit) return BEAM_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    done->fetch_or(bit, std::memory_order_release);
    return BEAM_OK;
}

template <int NT, int CG, bool F32>
beam_status launch_tile(const MatmulParams& p, const beam::Device& dev, void* part, cudaStream_t stream,
                        uint32_t flags) {
    const bool pdl = (flags & BEAM_OPT_PDL) != 0, drop = (flags & BEAM_OPT_TEST_WAIT_TIMEOUT) != 0;
    using C = beam::TileConfig<NT, CG>;
    static std::atomic<unsigned long long> allowed{0};
    const void* fn = reinterpret_cast<const void*>(beam::matmul_int8_tile_kernel<NT, CG, F32>);
    beam_status st = allow_smem(fn, C::kSmem, &allowed, dev.ordinal);
    if (st != BEAM_OK) return st;
    beam::MatmulTcParams q{};
    static_cast<beam::TilePlan&>(q) = beam::launch_plan<NT, CG>(p.M, p.N, p.K, dev.sms);
    q.p = p;
    q.wide = !F32 && p.N % 8 == 0 && p.N >= beam::kTileN && !misaligned(p.out, 16);
    CUtensorMap wmap, pmap, amap;
    if (!row_map(&wmap, p.w, p.N, p.K, beam::kTileN) || !row_map(&amap, p.a, p.M, p.K, C::kRows)) return BEAM_ERR_CUDA;
    if (!q.wide) pmap = wmap;
    else if (!permuted_map(&pmap, p.w, p.N, p.K)) return BEAM_ERR_CUDA;
    q.part = static_cast<float*>(part);
    q.wait_ns = drop ? beam::kMatmulTestWaitNs : beam::kMatmulWaitNs;
    q.drop = drop;
    q.status = dev.status_word;
    const uint32_t workers = q.waves ? (q.tiles < q.workers ? q.tiles : q.workers) : q.sharers;
    void* args[] = {&wmap, &pmap, &amap, &q};
    st = launch(fn, dim3(workers * CG), dim3(C::kThreads), args, C::kSmem, stream, pdl, CG);
    const uint32_t shared = q.split / q.steps;  // tiles
    if (st != BEAM_OK || shared == 0) return st;
    void* join_args[] = {&q};
    // started early where it follows the shared steps alone: behind whole waves its
    // blocks, waiting on the SMs that are done, cost 2 us
    return launch(reinterpret_cast<const void*>(beam::matmul_int8_join_kernel<NT, CG, F32>),
                  dim3(shared, NT / beam::Join<NT>::kCols, CG), dim3(beam::kTileN), join_args, 0, stream, q.waves == 0);
}

template <bool F32>
beam_status launch_tiles(Shape shape, const MatmulParams& p, const beam::Device& dev, void* part,
                         cudaStream_t stream, uint32_t flags) {
    switch (shape) {
    case Shape::k16: return launch_tile<16, 1, F32>(p, dev, part, stream, flags);
    case Shape::k32: return launch_tile<32, 1, F32>(p, dev, part, stream, flags);
    case Shape::k64: return launch_tile<64, 1, F32>(p, dev, part, stream, flags);
    case Shape::k128: return launch_tile<128, 1, F32>(p, dev, part, stream, flags);
    default: return launch_tile<256, 2, F32>(p, dev, part, stream, flags);
    }
}

bool bad_shape(int64_t M, int N, int K) {
    // the last: tiles are counted in 32 bits (out would have 2^46 elements)
    return M < 0 || M > 0x7FFFFFFF || N < 0 || K < 16 || (K & 15) || K > BEAM_MATMUL_MAX_K ||
           ((M + 127) / 128) * ((N + 127ll) / 128) > 0x7FFFFFFF;
}

}  // namespace

extern "C" {

int64_t beam_matmul_int8_workspace(int64_t M, int N, int K) {
    if (bad_shape(M, N, K)) return -1;
    if (M == 0 || N == 0) return 0;
    return beam::workspace_bytes(M, N, K);
}

beam_status beam_matmul_int8(beam_stream_t stream, const int8_t* a, const float* a_scale, const int8_t* w,
                             const float* w_scale, int64_t M, int N, int K, int out_type, void* out, void* workspace,
                             int64_t workspace_bytes, uint32_t flags) {
    if (bad_shape(M, N, K)) return BEAM_ERR_SHAPE;
    const int64_t need = beam_matmul_int8_workspace(M, N, K);
    if ((out_type != BEAM_OUT_BF16 && out_type != BEAM_OUT_FP32) || workspace_bytes < need ||
        (flags & ~(BEAM_OPT_PDL | BEAM_OPT_TEST_WAIT_TIMEOUT)) ||
        ((flags & BEAM_OPT_TEST_WAIT_TIMEOUT) && beam::choose(M, N, K) == Shape::kFew))
        return BEAM_ERR_ARG;
    if (M == 0 || N == 0) return BEAM_OK;
    if (!a || !a_scale || !w || !w_scale || !out || (need && !workspace)) return BEAM_ERR_NULL;
    const bool f32 = out_type == BEAM_OUT_FP32;
    const unsigned out_size = f32 ? 4u : 2u;
    if (misaligned(a, 16) || misaligned(w, 16) || misaligned(a_scale, 4) || misaligned(w_scale, 4) ||
        misaligned(out, out_size) || (need && misaligned(workspace, 16)))
        return BEAM_ERR_ALIGN;
    const size_t ob = (size_t)M * (size_t)N * out_size, nb = (size_t)need;
    const struct {
        const void* p;
        size_t n;
    } in[] = {{a, (size_t)M * (size_t)K}, {w, (size_t)N * (size_t)K}, {a_scale, (size_t)M * 4u},
              {w_scale, (size_t)N * 4u}};
    for (const auto& i : in)
        if (overlaps(out, ob, i.p, i.n) || overlaps(workspace, nb, i.p, i.n)) return BEAM_ERR_ALIAS;
    if (overlaps(out, ob, workspace, nb)) return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    MatmulParams p{a, a_scale, w, w_scale, out, M, N, K};
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const Shape shape = beam::choose(M, N, K);
    if (shape != Shape::kFew)
        return f32 ? launch_tiles<true>(shape, p, dev, workspace, cs, flags)
                   : launch_tiles<false>(shape, p, dev, workspace, cs, flags);
    void* args[] = {&p};
    int channels = 0;
    const void* fn = f32 ? few_kernel<true>(M, &channels) : few_kernel<false>(M, &channels);
    const int per_block = channels * beam::kFewWarps;
    return launch(fn, dim3((unsigned)(((int64_t)N + per_block - 1) / per_block)), dim3(32 * beam::kFewWarps), args, 0, cs,
                  (flags & BEAM_OPT_PDL) != 0);
}

}  // extern "C"
