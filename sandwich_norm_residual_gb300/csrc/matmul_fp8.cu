// Host side of the 8-bit floating-point product: argument checks (before any CUDA
// call), the choice of the kernel and the launch.
#include "matmul_fp8_small.cuh"

#include <atomic>

#include "beam_boundary.h"
#include "device.h"
#include "host.h"
#include "tensor_map.h"

static_assert(BEAM_MOE_MAX_EXPERTS <= beam::kFp8MaxExperts, "the table of experts");

namespace {

using beam::encode_tiled;
using beam::EncodeTiled;
using beam::Fp8Params;
using beam::Fp8Room;
using beam::misaligned;
using beam::overlaps;

// matrices of 8-bit rows of K, one behind the other, in tiles of `rows` rows of one matrix by
// one step of k, 128-byte swizzle; dims = 2: one matrix
bool tile_map(CUtensorMap* map, const void* base, int dims, int64_t matrices, int64_t rows_each, int K, int rows) {
    const EncodeTiled encode = encode_tiled();
    const cuuint64_t size[3] = {(cuuint64_t)K, (cuuint64_t)rows_each, (cuuint64_t)matrices};
    const cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)K * (cuuint64_t)rows_each};
    const cuuint32_t box[3] = {beam::kFp8Step, (cuuint32_t)rows, 1}, unit[3] = {1, 1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)dims, const_cast<void*>(base), size, strides, box, unit,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FEW>
const void* kernel(bool f32) {
    return f32 ? reinterpret_cast<const void*>(beam::matmul_fp8_kernel<FEW, true>)
               : reinterpret_cast<const void*>(beam::matmul_fp8_kernel<FEW, false>);
}

template <bool FEW>
cudaLaunchConfig_t config(int clusters, int split, cudaStream_t stream, cudaLaunchAttribute* attr) {
    using C = beam::Fp8Tile<FEW>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * split));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)(split);
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cfg;
}

// Also that the adding warps' registers are there: a request for more than the launch has would wait forever
template <bool FEW>
bool allow_smem() {
    using C = beam::Fp8Tile<FEW>;
    for (int f32 = 0; f32 < 2; ++f32) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel<FEW>(f32)) != cudaSuccess) return false;
        if (!FEW && attr.numRegs * C::kThreads < 32 * (C::kAddWarps * C::kAddRegs + 4 * C::kOtherRegs)) return false;
        if (cudaFuncSetAttribute(kernel<FEW>(f32), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)beam::Fp8Tile<FEW>::kSmem) !=
            cudaSuccess)
            return false;
    }
    return true;
}

// Raises the kernels' shared-memory limits and asks how many clusters fit, once on each device
beam_status room(const beam::Device& dev, Fp8Room* out) {
    static std::atomic<uint64_t> known[64];  // 0: not yet
    std::atomic<uint64_t>& slot = known[dev.ordinal & 63];
    uint64_t v = slot.load(std::memory_order_acquire);
    if (!v) {
        if (!allow_smem<true>() || !allow_smem<false>()) {
            cudaGetLastError();
            return BEAM_ERR_CUDA;
        }
        cudaLaunchAttribute attr;
        for (int i = 0; i < 4; ++i) {  // both kernels fill an SM
            int n = dev.sms;
            const cudaLaunchConfig_t cfg = config<true>(1, 1 << i, nullptr, &attr);
            if (i > 0 && cudaOccupancyMaxActiveClusters(&n, kernel<true>(false), &cfg) != cudaSuccess) {
                cudaGetLastError();
                return BEAM_ERR_CUDA;
            }
            v |= (uint64_t)(n < 0 ? 0 : n > 0xFFFF ? 0xFFFF : n) << (16 * i);
        }
        slot.store(v, std::memory_order_release);
    }
    for (int i = 0; i < 4; ++i) out->clusters[i] = (int)(v >> (16 * i)) & 0xFFFF;
    return BEAM_OK;
}

template <bool FEW>
beam_status launch(const Fp8Params& q, const beam::Fp8Plan& plan, const uint8_t* a, const uint8_t* w, int K, bool f32, cudaStream_t stream) {
    CUtensorMap wmap, amap;
    if (!tile_map(&wmap, w, 3, q.E, q.N, K, 128) || !tile_map(&amap, a, 2, 1, q.R, K, FEW ? 16 : 128)) return BEAM_ERR_CUDA;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config<FEW>(plan.clusters, plan.split, stream, &attr);
    void* args[] = {&wmap, &amap, const_cast<Fp8Params*>(&q)};
    if (cudaLaunchKernelExC(&cfg, kernel<FEW>(f32), args) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

// Eight warps share a block's k, and four where there are channels enough for 13 blocks on every SM
// (N = 20480, 8 and 4 warps: 21.4 and 21.9 us; N = 40960: 38.6 and 36.2; sixteen experts of N = 5120:
// 84 and 74)
template <int WARPS, int BLOCKS, int NT>
beam_status launch_small(const beam::Fp8SmallParams& p, bool f32, dim3 grid, cudaStream_t stream) {
    const void* fn = f32 ? reinterpret_cast<const void*>(beam::matmul_fp8_small_kernel<WARPS, BLOCKS, NT, true>)
                         : reinterpret_cast<const void*>(beam::matmul_fp8_small_kernel<WARPS, BLOCKS, NT, false>);
    void* args[] = {const_cast<beam::Fp8SmallParams*>(&p)};
    if (cudaLaunchKernel(fn, grid, dim3(32 * WARPS), args, 0, stream) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_ERR_CUDA;
    }
    return BEAM_OK;
}

beam_status product(beam_stream_t stream, const uint8_t* a, const float* a_scale, const int32_t* offsets, bool grouped,
                    const uint8_t* w, const float* w_scale, int64_t R, int E, int N, int K, int out_type, void* out,
                    uint32_t flags) {
    if (R < 0 || R > BEAM_MATMUL_FP8_MAX_ROWS || N < 0 || N > BEAM_MATMUL_FP8_MAX_ROWS || K < 16 || (K & 15) ||
        K > BEAM_MATMUL_MAX_K || E < 1 || E > BEAM_MOE_MAX_EXPERTS || (int64_t)N * K >= (int64_t(1) << 40) ||
        beam::fp8_most_tiles(R, E, beam::kFp8Few) * (((int64_t)N + 127) / 128) > 0x7FFFFFFF)
        return BEAM_ERR_SHAPE;
    if ((out_type != BEAM_OUT_BF16 && out_type != BEAM_OUT_FP32) || (flags & ~BEAM_OPT_TEST_WAIT_TIMEOUT) ||
        ((flags & BEAM_OPT_TEST_WAIT_TIMEOUT) && K <= beam::kFp8Step))
        return BEAM_ERR_ARG;
    if (R == 0 || N == 0) return BEAM_OK;
    if (!a || !a_scale || !w || !w_scale || !out || (grouped && !offsets)) return BEAM_ERR_NULL;
    const bool f32 = out_type == BEAM_OUT_FP32;
    const unsigned out_size = f32 ? 4u : 2u;
    if (misaligned(a, 16) || misaligned(w, 16) || misaligned(a_scale, 4) || misaligned(w_scale, 4) ||
        misaligned(offsets, 4) || misaligned(out, out_size))
        return BEAM_ERR_ALIGN;
    const size_t steps = ((size_t)K + 127) / 128, ob = (size_t)R * (size_t)N * out_size;
    const struct {
        const void* p;
        size_t n;
    } in[] = {{a, (size_t)R * (size_t)K}, {w, (size_t)E * (size_t)N * (size_t)K}, {a_scale, (size_t)R * steps * 4u},
              {w_scale, (size_t)E * (((size_t)N + 127) / 128) * steps * 4u}, {offsets, grouped ? ((size_t)E + 1) * 4u : 0}};
    for (const auto& i : in)
        if (overlaps(out, ob, i.p, i.n)) return BEAM_ERR_ALIAS;
    beam::Device dev;
    beam_status st = beam::device(&dev);
    if (st != BEAM_OK) return st;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool sectors = (int64_t)N * out_size % 32 == 0 && !misaligned(out, 32);
    const bool drop = (flags & BEAM_OPT_TEST_WAIT_TIMEOUT) != 0;
    Fp8Room fits;
    st = room(dev, &fits);
    if (st != BEAM_OK) return st;
    const beam::Fp8Plan plan = beam::fp8_plan(R, E, N, K, sectors, fits);
    if (!drop && beam::fp8_small(R, E, N, K, plan)) {
        beam::Fp8SmallParams p{a, w, {}, K};
        p.q.a_scale = a_scale;
        p.q.w_scale = w_scale;
        p.q.out = out;
        p.q.offsets = offsets;
        p.q.R = R;
        p.q.E = E;
        p.q.N = N;
        p.q.steps = (uint32_t)steps;
        p.q.status = dev.status_word;
        const int64_t groups = R < E ? R : E, blocks = ((int64_t)N + beam::kFp8SmallChannels - 1) / beam::kFp8SmallChannels;
        const dim3 grid((unsigned)blocks, (unsigned)(E == 1 ? 1 : beam::fp8_most_tiles(R, E, beam::kFp8SmallPart)));
        if (E == 1 && R > 8) return launch_small<8, 3, 2>(p, f32, grid, cs);
        return blocks * groups >= 13 * (int64_t)dev.sms ? launch_small<4, 6, 1>(p, f32, grid, cs) : launch_small<8, 3, 1>(p, f32, grid, cs);
    }
    Fp8Params q{};
    q.a_scale = a_scale;
    q.w_scale = w_scale;
    q.out = out;
    q.offsets = offsets;
    q.R = R;
    q.E = E;
    q.N = N;
    q.steps = (uint32_t)steps;
    q.width = (uint32_t)plan.width;
    q.n_tiles = beam::fp8_up((uint32_t)N, q.width);
    q.split = plan.split;
    q.scales16 = steps % 4 == 0 && !misaligned(a_scale, 16);
    q.wide = sectors;
    q.wait_ns = drop ? beam::kFp8TestWaitNs : beam::kFp8WaitNs;
    q.drop = drop;
    q.status = dev.status_word;
    return plan.few ? launch<true>(q, plan, a, w, K, f32, cs) : launch<false>(q, plan, a, w, K, f32, cs);
}

}  // namespace

extern "C" {

beam_status beam_matmul_fp8(beam_stream_t stream, const uint8_t* a, const float* a_scale, const uint8_t* w,
                            const float* w_scale, int64_t M, int N, int K, int out_type, void* out, uint32_t flags) {
    return product(stream, a, a_scale, nullptr, false, w, w_scale, M, 1, N, K, out_type, out, flags);
}

beam_status beam_matmul_fp8_experts(beam_stream_t stream, const uint8_t* a, const float* a_scale, const int32_t* offsets,
                                    const uint8_t* w, const float* w_scale, int64_t R, int E, int N, int K, int out_type,
                                    void* out, uint32_t flags) {
    return product(stream, a, a_scale, offsets, true, w, w_scale, R, E, N, K, out_type, out, flags);
}

}  // extern "C"
