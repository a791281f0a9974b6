// Host side of the 8-bit integer product: argument checks (before any CUDA
// call), the choice of the kernel and the launch.
#include "matmul_int8.cuh"

#include "beam_boundary.h"
#include "device.h"

namespace {

using beam::MatmulParams;

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return na && nb && a0 < b0 + nb && b0 < a0 + na;
}

bool misaligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0; }

template <bool F32>
const void* few_kernel(int mb) {
    switch (mb) {
    case 1: return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<1, 2, 4, F32>);
    case 2: return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<2, 2, 4, F32>);
    case 4: return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<4, 2, 4, F32>);
    default: return reinterpret_cast<const void*>(beam::matmul_int8_few_kernel<8, 2, 4, F32>);
    }
}

beam_status launch(const void* fn, dim3 grid, dim3 block, void** args, size_t smem, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

}  // namespace

extern "C" beam_status beam_matmul_int8(beam_stream_t stream, const int8_t* a, const float* a_scale,
                                        const int8_t* w, const float* w_scale, int64_t M, int N, int K,
                                        int out_type, void* out, uint32_t flags) {
    if (M < 0 || M > 0x7FFFFFFF || N < 0 || K < 16 || (K & 15) || K > BEAM_MATMUL_MAX_K) return BEAM_ERR_SHAPE;
    if ((out_type != BEAM_OUT_BF16 && out_type != BEAM_OUT_FP32) || (flags & ~BEAM_OPT_PDL)) return BEAM_ERR_ARG;
    if (M == 0 || N == 0) return BEAM_OK;
    if (!a || !a_scale || !w || !w_scale || !out) return BEAM_ERR_NULL;
    const bool f32 = out_type == BEAM_OUT_FP32;
    const unsigned out_size = f32 ? 4u : 2u;
    if (misaligned(a, 16) || misaligned(w, 16) || misaligned(a_scale, 4) || misaligned(w_scale, 4) ||
        misaligned(out, out_size))
        return BEAM_ERR_ALIGN;
    const size_t ob = (size_t)M * (size_t)N * out_size;
    if (overlaps(out, ob, a, (size_t)M * (size_t)K) || overlaps(out, ob, w, (size_t)N * (size_t)K) ||
        overlaps(out, ob, a_scale, (size_t)M * 4u) || overlaps(out, ob, w_scale, (size_t)N * 4u))
        return BEAM_ERR_ALIAS;
    beam::Device dev;
    const beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    MatmulParams p{a, a_scale, w, w_scale, out, M, N, K};
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool pdl = (flags & BEAM_OPT_PDL) != 0;
    void* args[] = {&p};
    const int mb = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8;
    const void* fn = f32 ? few_kernel<true>(mb) : few_kernel<false>(mb);
    // M in grid.y: at most 65535 groups a launch
    constexpr int kR = 2, kWarps = 8;
    const unsigned gx = (unsigned)((N + kR * kWarps - 1) / (kR * kWarps));
    for (int64_t m = 0; m < M; m += 65535ll * mb) {
        p.M = M - m < 65535ll * mb ? M - m : 65535ll * mb;
        p.a = a + (size_t)m * (size_t)K;
        p.a_scale = a_scale + m;
        p.out = static_cast<char*>(out) + (size_t)m * (size_t)N * out_size;
        const beam_status s = launch(fn, dim3(gx, (unsigned)((p.M + mb - 1) / mb)), dim3(256), args, 0, cs, pdl);
        if (s != BEAM_OK) return s;
    }
    return BEAM_OK;
}
