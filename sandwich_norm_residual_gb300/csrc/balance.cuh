// Balance loss of a sigmoid router, its per-expert counts, and its gradient.
//
// For the tokens t of a sequence of length n (E experts, K choices a token):
//   s = sigmoid(z_t), p = s / sum_e s, Q_e = sum_t p_e, c_e = choices of expert e
//   loss = alpha E / (K n^2) sum_e c_e Q_e
//   dloss/dz_te = alpha E / (K n^2) s_e (1 - s_e) / (sum s) (c_e - sum_i c_i p_i)
// Both passes are bound by the logits' way from (and the gradient's way to)
// HBM: 4 E bytes a token read forward, 4 E read and 4 E written backward. One
// warp holds a token's row in registers (4 experts a lane for every 128), so
// the row is read once and its sums are shuffles.
//
// Sequences are ragged, so the split goes by tokens: block b takes the tokens
// [b C, (b + 1) C) and writes one record (Q and c) for every sequence it meets,
// at index b + s. Along the staircase of (block, sequence) pairs that overlap,
// b + s grows, so no two pairs share a record, nothing needs to be zeroed, there
// are no floating-point atomics and the result is the same in every run. A
// second kernel adds a sequence's records in order.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "packed.cuh"
#include "tma.cuh"

namespace beam {

constexpr int kBalanceThreads = 512;
constexpr int kBalanceWarps = kBalanceThreads / 32;
constexpr int kBalanceBlocks = 304;  // two blocks on each of 152 SMs
constexpr int kBalanceSmall = 512;   // tokens up to which one kernel may do it all (balance_small_kernel)
constexpr int kBalanceSmallLogits = 384 * 256;  // ... and logits for each sequence
constexpr int kBalanceFinalThreads = 1024;
constexpr int kBalanceFinalSums = 4 * kBalanceFinalThreads;  // 4 experts a thread

struct BalanceParams {
    const float* logits;    // [T, E]
    const int32_t* idx;     // [T, K]
    const int32_t* off;     // [S + 1], or NULL: one sequence of T tokens
    long long T;
    int E, K, S;
    int chunk;              // tokens a block
    int blocks;
    float* rec_q;           // [blocks + S, E]
    int32_t* rec_c;         // [blocks + S, E]
    double factor;          // alpha E / K
    float* loss;            // [S]
    int32_t* counts;        // [S, E] (written forward, read backward)
    const float* dloss;     // [S]
    float* dlogits;         // [T, E]
    unsigned int* status;
};

__device__ __forceinline__ long long seq_begin(const BalanceParams& p, int s) {
    return p.off ? (long long)__ldg(p.off + s) : 0;
}
__device__ __forceinline__ long long seq_end(const BalanceParams& p, int s) {
    return p.off ? (long long)__ldg(p.off + s + 1) : p.T;
}

// The first sequence that ends behind token t (S: none does); the whole warp. 32
// places are looked at in one way to memory, where halving the range takes one for
// each bit of S.
__device__ __forceinline__ int find_seq(const BalanceParams& p, long long t) {
    int lo = 0, n = p.S;  // the answer lies in [lo, lo + n]; 32 steps stay below 2^31 (n <= 2^31 - 64)
    const int lane = threadIdx.x & 31;
    while (n > 0) {
        const int step = (n + 31) / 32, at = lo + min((lane + 1) * step, n) - 1;
        const unsigned behind = __ballot_sync(0xFFFFFFFFu, seq_end(p, at) > t);
        // the sequences before the first place that lies behind t do not
        const int k = behind ? __ffs(behind) - 1 : 32;
        const int skipped = min(k * step, n);
        lo += skipped;
        n = behind ? min(step, n - skipped) - 1 : 0;
    }
    return lo;
}

// Calls body(s, lo, hi) for every sequence s and its tokens [lo, hi) within
// [t0, t1), and gap(lo, hi) for tokens of no sequence. Every call advances s,
// so it ends whatever the offsets hold.
template <class Body, class Gap>
__device__ __forceinline__ void for_sequences(const BalanceParams& p, long long t0, long long t1, Body body, Gap gap) {
    long long t = t0;
    for (int s = find_seq(p, t0); s < p.S && t < t1; ++s) {
        const long long b = min(max(seq_begin(p, s), t), t1), e = min(max(seq_end(p, s), b), t1);
        if (b > t) gap(t, b);
        if (e > b) body(s, b, e);
        t = e;
    }
    if (t < t1) gap(t, t1);
}

// a b + c, rounded once
__device__ __forceinline__ float2 fma2_rn(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// s = sigmoid(z) and e = exp(-z) of two logits on the special-function unit, where
// expf and a division would keep the forward pass busy for as long as its memory
// traffic. e = 2^t 2^r: t is -z log2(e) rounded, r what the rounding of the product
// and of the constant leave out, so that the error does not grow with |z|. In units of
// 2^-24: e has 4 of the exponential (its documented bound, 2^-22), 1 of 2^r and 1 of
// their product, which 1 + e goes without; that adds 1, the reciprocal 2 (one unit in
// the last place): s is within 8 (measured: 5). Below 2^-126 both are 0. Without r
// the error reached 65 at z = -85; at T = 16384, E = 256, 8 sequences the forward
// pass takes 13.2 us instead of 13.0, the backward 8.1 either way.
__device__ __forceinline__ void sigmoid_e(float2 z, float2& s, float2& e) {
    const float2 hi = make_float2(-0x1.715476p+0f, -0x1.715476p+0f);  // -log2(e), and the rest of it
    const float2 lo = make_float2(-0x1.4ae0cp-26f, -0x1.4ae0cp-26f);
    const float2 ln2 = make_float2(0x1.62e43p-1f, 0x1.62e43p-1f);
    const float2 t = mul2_rn(z, hi), r = fma2_rn(z, lo, fma2_rn(z, hi, make_float2(-t.x, -t.y)));
    // 2^r = 1 + r ln 2 (r below 2^-15 where 2^t is neither 0 nor infinite; there, and
    // for an infinite z, it only has to be a positive number)
    float2 m = fma2_rn(r, ln2, make_float2(1.0f, 1.0f));
    m = make_float2(fminf(fmaxf(m.x, 0.5f), 2.0f), fminf(fmaxf(m.y, 0.5f), 2.0f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(__fmaf_rn(e.x, m.x, 1.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(__fmaf_rn(e.y, m.y, 1.0f)));
    e = make_float2(__fmul_rn(e.x, m.x), __fmul_rn(e.y, m.y));
}

// (s, c) += t with the rounding error of s kept in c (Knuth's TwoSum)
__device__ __forceinline__ void sum_into(float& s, float& c, float t) {
    const float n = __fadd_rn(s, t), b = __fsub_rn(n, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(n, b)), __fsub_rn(t, b)));
    s = n;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// V float4 a lane: experts 128 v + 4 lane + i. Slots behind E hold logits of
// -inf, whose sigmoid is 0.
template <int V>
__device__ __forceinline__ void load_row(const BalanceParams& p, long long t, int lane, float4 (&z)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 128 * v + 4 * lane;
        if (e < p.E) {
            const float* a = p.logits + (size_t)t * (size_t)p.E + e;
            asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(z[v].x), "=f"(z[v].y), "=f"(z[v].z), "=f"(z[v].w) : "l"(a));
        } else {
            z[v] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
    }
}

// 1 / sum, or 0 when every sigmoid of the token is 0 (NaN stays)
__device__ __forceinline__ float inverse_or_zero(float sum) { return sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum); }

// the choices of tokens [lo, hi), K a token, counted in shared memory by the block
__device__ __forceinline__ void count_choices(const BalanceParams& p, long long lo, long long hi, int* counts) {
    for (long long i = lo * p.K + threadIdx.x; i < hi * p.K; i += kBalanceThreads) {
        const int e = __ldg(p.idx + i);
        if ((unsigned)e < (unsigned)p.E) atomicAdd(&counts[e], 1);
        else atomicOr(p.status, 2u);
    }
}

// q += sigmoid(z) / sum of the token's sigmoids
template <int V>
__device__ __forceinline__ void add_probabilities(float4 (&z)[V], float4 (&q)[V]) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float2 a, b, unused;
        sigmoid_e(make_float2(z[v].x, z[v].y), a, unused);
        sigmoid_e(make_float2(z[v].z, z[v].w), b, unused);
        z[v] = make_float4(a.x, a.y, b.x, b.y);
        sum += (z[v].x + z[v].y) + (z[v].z + z[v].w);
    }
    const float inv = inverse_or_zero(warp_sum(sum));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        q[v].x = __fmaf_rn(z[v].x, inv, q[v].x);
        q[v].y = __fmaf_rn(z[v].y, inv, q[v].y);
        q[v].z = __fmaf_rn(z[v].z, inv, q[v].z);
        q[v].w = __fmaf_rn(z[v].w, inv, q[v].w);
    }
}

template <int V>
__global__ void __launch_bounds__(kBalanceThreads) balance_records_kernel(const BalanceParams p) {
    __shared__ float sq[kBalanceWarps][V * 128];
    __shared__ int sc[V * 128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    const long long t0 = (long long)blockIdx.x * p.chunk, t1 = min(t0 + p.chunk, p.T);
    // this warp's tokens, across the sequences; the next one's row is on its way
    // before anything else is known
    long long t = t0 + warp;
    float4 nx[V];
    if (t < t1) load_row<V>(p, t, lane, nx);
    auto skip = [&](long long hi) {
        if (t >= hi) return;
        t += (hi - t + kBalanceWarps - 1) / kBalanceWarps * kBalanceWarps;
        if (t < t1) load_row<V>(p, t, lane, nx);
    };
    for_sequences(p, t0, t1, [&](int s, long long lo, long long hi) {
        for (int e = tid; e < V * 128; e += kBalanceThreads) sc[e] = 0;
        __syncthreads();
        count_choices(p, lo, hi, sc);
        float4 q[V];
#pragma unroll
        for (int v = 0; v < V; ++v) q[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (; t < hi; t += kBalanceWarps) {
            float4 z[V];
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = nx[v];
            if (t + kBalanceWarps < t1) load_row<V>(p, t + kBalanceWarps, lane, nx);
            add_probabilities<V>(z, q);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) *reinterpret_cast<float4*>(&sq[warp][128 * v + 4 * lane]) = q[v];
        __syncthreads();
        const size_t rec = ((size_t)blockIdx.x + (size_t)s) * (size_t)p.E;
        for (int e = tid; e < p.E; e += kBalanceThreads) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kBalanceWarps; ++w) a += sq[w][e];
            p.rec_q[rec + e] = a;
            p.rec_c[rec + e] = sc[e];
        }
        __syncthreads();
    }, [&](long long, long long hi) { skip(hi); });
}

// One block a sequence: its records added in order (groups of threads take
// every G-th record, then the groups in order), the counts and the loss. Sums are
// FP32 pairs: FP64 additions, 64 times slower than FP32 ones on this GPU, took 45
// us for a sequence in 304 blocks.
__global__ void __launch_bounds__(kBalanceFinalThreads) balance_loss_kernel(const BalanceParams p) {
    __shared__ float2 sq[kBalanceFinalSums];  // [groups][E]
    __shared__ double part[kBalanceFinalThreads / 32];
    const int tid = threadIdx.x, s = blockIdx.x, quads = p.E / 4;
    pdl_wait();
    const long long b = seq_begin(p, s), e = seq_end(p, s);
    if (tid == 0 && (b < 0 || e < b || e > p.T)) atomicOr(p.status, 2u);
    const long long lo = max(b, 0ll), hi = min(e, p.T);
    const long long n = hi > lo ? hi - lo : 0;
    const int first = n ? (int)(lo / p.chunk) : 0, last = n ? (int)((hi - 1) / p.chunk) : -1;
    const int groups = kBalanceFinalThreads / quads;
    const int g = tid / quads, quad = tid % quads;
    float q[4] = {0, 0, 0, 0}, qc[4] = {0, 0, 0, 0};
    int c[4] = {0, 0, 0, 0};
    if (g < groups) {
#pragma unroll 4
        for (int r = first + g; r <= last; r += groups) {
            const size_t at = ((size_t)r + (size_t)s) * (size_t)p.E + 4 * quad;
            const float4 f = __ldcg(reinterpret_cast<const float4*>(p.rec_q + at));
            const int4 k = __ldcg(reinterpret_cast<const int4*>(p.rec_c + at));
            sum_into(q[0], qc[0], f.x);
            sum_into(q[1], qc[1], f.y);
            sum_into(q[2], qc[2], f.z);
            sum_into(q[3], qc[3], f.w);
            c[0] += k.x, c[1] += k.y, c[2] += k.z, c[3] += k.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sq[g * p.E + 4 * quad + i] = make_float2(q[i], qc[i]);
    }
    __syncthreads();
    float sum = 0.f, comp = 0.f;
    if (tid < p.E)
        for (int k = 0; k < groups; ++k) {
            const float2 v = sq[k * p.E + tid];
            sum_into(sum, comp, v.x);
            comp += v.y;
        }
    __syncthreads();
    int* scn = reinterpret_cast<int*>(sq);
    if (g < groups) {
#pragma unroll
        for (int i = 0; i < 4; ++i) scn[g * p.E + 4 * quad + i] = c[i];
    }
    __syncthreads();
    double term = 0;
    if (tid < p.E) {
        int count = 0;
        for (int k = 0; k < groups; ++k) count += scn[k * p.E + tid];
        p.counts[(size_t)s * (size_t)p.E + tid] = count;
        term = (double)count * ((double)sum + (double)comp);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
    if ((tid & 31) == 0) part[tid >> 5] = term;
    __syncthreads();
    if (tid == 0) {
        double total = 0;
        for (int w = 0; w < (p.E + 31) / 32; ++w) total += part[w];
        p.loss[s] = n ? (float)(p.factor / ((double)n * (double)n) * total) : 0.0f;
    }
}

// Few tokens: a block a sequence, without records and without a second kernel: one
// launch and one workspace less, which are 5 us of the host (a pass both ways through
// the binding 33 us instead of 38). On the GPU its one block for a sequence grows with
// the rows that each warp takes in turn, where records keep near 8 us. One sequence,
// one kernel against two, us: E = 256: T = 128 7.0, 7.9; 192 8.5, 8.0; 384 13.0, 8.5;
// 512 16.1, 8.4. E = 64: 256 8.6, 8.0; 512 13.6, 7.9. E = 512: 128 8.9, 9.0; 192 11.2,
// 9.3; 512 24.6, 10.0. Four sequences, T = 512: E = 256 6.9, 8.1; E = 512 9.4, 9.2. The
// limits are near where the GPU loses what the host gains.
template <int V>
__global__ void __launch_bounds__(kBalanceThreads) balance_small_kernel(const BalanceParams p) {
    __shared__ float sq[kBalanceWarps][V * 128];
    __shared__ int sc[V * 128];
    __shared__ double part[kBalanceWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, s = blockIdx.x;
    for (int e = tid; e < V * 128; e += kBalanceThreads) sc[e] = 0;
    const long long b = seq_begin(p, s), e = seq_end(p, s);
    if (tid == 0 && (b < 0 || e < b || e > p.T)) atomicOr(p.status, 2u);
    const long long lo = max(b, 0ll), hi = max(min(e, p.T), lo), n = hi - lo;
    __syncthreads();
    count_choices(p, lo, hi, sc);
    float4 q[V], nx[V];
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    long long t = lo + warp;
    if (t < hi) load_row<V>(p, t, lane, nx);
    for (; t < hi; t += kBalanceWarps) {
        float4 z[V];
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = nx[v];
        if (t + kBalanceWarps < hi) load_row<V>(p, t + kBalanceWarps, lane, nx);
        add_probabilities<V>(z, q);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) *reinterpret_cast<float4*>(&sq[warp][128 * v + 4 * lane]) = q[v];
    __syncthreads();
    double term = 0;
    if (tid < p.E) {
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < kBalanceWarps; ++w) a += sq[w][tid];
        p.counts[(size_t)s * (size_t)p.E + tid] = sc[tid];
        term = (double)sc[tid] * (double)a;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
    if (lane == 0) part[warp] = term;
    __syncthreads();
    if (tid == 0) {
        double total = 0;
        for (int w = 0; w < kBalanceWarps; ++w) total += part[w];
        p.loss[s] = n ? (float)(p.factor / ((double)n * (double)n) * total) : 0.0f;
    }
}

template <int V>
__global__ void __launch_bounds__(kBalanceThreads) balance_grad_kernel(const BalanceParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (long long)blockIdx.x * p.chunk, t1 = min(t0 + p.chunk, p.T);
    const float factor = (float)p.factor;
    long long t = t0 + warp;  // this warp's tokens, across the sequences
    float4 nx[V];
    if (t < t1) load_row<V>(p, t, lane, nx);
    for_sequences(p, t0, t1, [&](int s, long long, long long hi) {
        // in FP32, a few roundings: FP64 here took 4 us of every block
        const float n = (float)(min(seq_end(p, s), p.T) - max(seq_begin(p, s), 0ll));
        const float g = __fdiv_rn(__fdiv_rn(__fmul_rn(__ldg(p.dloss + s), factor), n), n);
        float4 c[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 128 * v + 4 * lane;
            const int4 k = e < p.E ? __ldg(reinterpret_cast<const int4*>(p.counts + (size_t)s * (size_t)p.E + e))
                                   : make_int4(0, 0, 0, 0);
            c[v] = make_float4((float)k.x, (float)k.y, (float)k.z, (float)k.w);
        }
        for (; t < hi; t += kBalanceWarps) {
            float4 z[V], d[V];  // d: s (1 - s)
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = nx[v];
            if (t + kBalanceWarps < t1) load_row<V>(p, t + kBalanceWarps, lane, nx);
            float sum = 0.f, mix = 0.f;
            // 1 - s is e s, which keeps its digits where s is near 1; where z < 0
            // (e may be infinite there) 1 - s itself loses none
            auto two = [&](float2 zi, float& dx, float& dy, float2 ci) {
                float2 s2, e2;
                sigmoid_e(zi, s2, e2);
                dx = s2.x * (zi.x < 0.0f ? 1.0f - s2.x : e2.x * s2.x);
                dy = s2.y * (zi.y < 0.0f ? 1.0f - s2.y : e2.y * s2.y);
                sum += s2.x;
                sum += s2.y;
                mix = __fmaf_rn(ci.x, s2.x, mix);
                mix = __fmaf_rn(ci.y, s2.y, mix);
            };
#pragma unroll
            for (int v = 0; v < V; ++v) {
                two(make_float2(z[v].x, z[v].y), d[v].x, d[v].y, make_float2(c[v].x, c[v].y));
                two(make_float2(z[v].z, z[v].w), d[v].z, d[v].w, make_float2(c[v].z, c[v].w));
            }
            const float inv = inverse_or_zero(warp_sum(sum));
            const float mean = warp_sum(mix) * inv;
            // d inv is at most 1; g inv would leave FP32 where every sigmoid is near
            // 2^-126 and g carries a loss scale
            auto out = [&](float di, float ci) { return (di * inv) * (g * (ci - mean)); };
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = 128 * v + 4 * lane;
                if (e < p.E)
                    __stcs(reinterpret_cast<float4*>(p.dlogits + (size_t)t * (size_t)p.E + e),
                           make_float4(out(d[v].x, c[v].x), out(d[v].y, c[v].y), out(d[v].z, c[v].z),
                                       out(d[v].w, c[v].w)));
            }
        }
    }, [&](long long, long long hi) {
        // tokens of no sequence: no gradient
        for (; t < hi; t += kBalanceWarps) {
            for (int e = 4 * lane; e < p.E; e += 128)
                __stcs(reinterpret_cast<float4*>(p.dlogits + (size_t)t * (size_t)p.E + e),
                       make_float4(0.f, 0.f, 0.f, 0.f));
            if (t + kBalanceWarps < hi) continue;
            if (t + kBalanceWarps < t1) load_row<V>(p, t + kBalanceWarps, lane, nx);
        }
    });
}

}  // namespace beam
