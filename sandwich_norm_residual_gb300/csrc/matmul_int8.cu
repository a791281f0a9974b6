// Host side of the 8-bit integer product: argument checks (before any CUDA
// call), the choice of the kernel and the launch.
#include "matmul_int8_tc.cuh"

#include <atomic>

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

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void*> cached{nullptr};
    void* fn = cached.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        cached.store(fn, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(fn);
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

template <int NT, bool F32>
beam_status launch_tile(const MatmulParams& p, const beam::Device& dev, cudaStream_t stream, bool pdl) {
    using C = beam::TileConfig<NT>;
    static std::atomic<unsigned long long> allowed{0};
    const void* fn = reinterpret_cast<const void*>(beam::matmul_int8_tile_kernel<NT, F32>);
    const beam_status st = allow_smem(fn, C::kSmem, &allowed, dev.ordinal);
    if (st != BEAM_OK) return st;
    CUtensorMap wmap, amap;
    if (!row_map(&wmap, p.w, p.N, p.K, beam::kTileN) || !row_map(&amap, p.a, p.M, p.K, NT)) return BEAM_ERR_CUDA;
    beam::MatmulTcParams q{};
    q.p = p;
    q.n_tiles = (p.N + beam::kTileN - 1) / beam::kTileN;
    q.m_tiles = (int)((p.M + NT - 1) / NT);
    const int64_t tiles = (int64_t)q.n_tiles * q.m_tiles;
    // k is split where there are too few tiles for the SMs: as many CTAs a tile
    // as fit at once, each with two steps at least
    const int steps = (p.K + beam::kStepK - 1) / beam::kStepK;
    int64_t splits = (int64_t)dev.sms * C::kCtas / tiles;
    if (splits > steps / 2) splits = steps / 2;
    q.splits = splits < 1 ? 1 : splits > 8 ? 8 : (int)splits;
    if (tiles * q.splits > 0x7FFFFFFF) return BEAM_ERR_SHAPE;
    q.wait_ns = beam::kMatmulWaitNs;
    q.status = dev.status_word;
    void* args[] = {&wmap, &amap, &q};
    return launch(fn, dim3((unsigned)(tiles * q.splits)), dim3(C::kThreads), args, C::kSmem, stream, pdl, q.splits);
}

template <bool F32>
beam_status launch_tiles(const MatmulParams& p, const beam::Device& dev, cudaStream_t stream, bool pdl) {
    if (p.M <= 16) return launch_tile<16, F32>(p, dev, stream, pdl);
    if (p.M <= 32) return launch_tile<32, F32>(p, dev, stream, pdl);
    if (p.M <= 64) return launch_tile<64, F32>(p, dev, stream, pdl);
    return launch_tile<128, F32>(p, dev, stream, pdl);
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
    if (M > 8) return f32 ? launch_tiles<true>(p, dev, cs, pdl) : launch_tiles<false>(p, dev, cs, pdl);
    void* args[] = {&p};
    const int mb = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8;
    const void* fn = f32 ? few_kernel<true>(mb) : few_kernel<false>(mb);
    constexpr int kR = 2, kWarps = 8;
    return launch(fn, dim3((unsigned)((N + kR * kWarps - 1) / (kR * kWarps))), dim3(256), args, 0, cs, pdl);
}
