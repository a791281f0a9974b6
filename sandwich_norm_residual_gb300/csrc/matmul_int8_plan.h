// How the 8-bit integer product is divided: tiles, shared steps, workspaces, the
// choice of a tile. Host arithmetic without CUDA, so that it can be tested anywhere;
// N and M go up to 2^31 - 1, so sums with them are taken in 64 bits.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BEAM_HOST_DEVICE __host__ __device__
#else
#define BEAM_HOST_DEVICE
#endif

namespace beam {

constexpr int kStepK = 128;    // k of one ring slot and of one operand slot
constexpr int kTileN = 128;    // channels of a CTA: the lanes of tensor memory
constexpr int kMaxSms = 152;   // workers of a launch at most, and what workspaces are sized for

// whether the 128 channels from n0 on all exist (n0 + 128 may be 2^31)
BEAM_HOST_DEVICE constexpr bool whole_channels(int N, int n0) { return N - n0 >= kTileN; }

// The split of a product into tiles of NT tokens by 128 CG channels
struct TilePlan {
    uint32_t m_tiles;  // tiles of NT tokens
    uint32_t steps;    // of k
    uint32_t tiles;
    // `workers` CTAs (CG = 1) or pairs (CG = 2). Worker c takes the whole tiles
    // c, c + workers, ... of the first waves * workers, and of the `split` steps of
    // the tiles behind those its share of an even split among the first `sharers`
    // (split * sharers < 2^32: fewer than 152 tiles of at most 512 steps).
    uint32_t waves, workers, sharers, split;
};

// What a join takes in steps of k: the sums written, the second kernel
template <int CG>
constexpr uint32_t kJoinSteps = CG == 1 ? 8 : 26;

template <int NT, int CG>
TilePlan plan(int64_t M, int64_t N, int K, int sms) {
    TilePlan q{};
    q.m_tiles = (uint32_t)((M + NT - 1) / NT);
    q.steps = (uint32_t)((K + kStepK - 1) / kStepK);
    q.tiles = q.m_tiles * (uint32_t)((N + kTileN * CG - 1) / (kTileN * CG));
    q.workers = (uint32_t)(sms / CG);
    // The tiles behind the last full wave are shared, with four steps a worker at
    // least, where that shortens the wave by more than the join takes (kJoinSteps).
    // Single CTAs: M = 517, N = 2565, K = 2576, 105 tiles of 21 steps: 19.6 us
    // unshared, 20.9 us shared; M = 64, N = 5120, K = 20480, 40 of 160: 75 and 29 us.
    // Pairs: M = 1024, N = 5120, K = 5120, 80 tiles of 40 steps: 53 and 41 us; M = 512,
    // 40 tiles: 31 and 39 us.
    q.waves = q.tiles / q.workers;
    q.split = (q.tiles - q.waves * q.workers) * q.steps;
    const uint32_t most = (q.split + 3) / 4;
    q.sharers = most < q.workers ? most : q.workers;
    if (q.split && q.steps <= (q.split + q.sharers - 1) / q.sharers + kJoinSteps<CG>) {
        q.waves += 1;
        q.split = q.sharers = 0;
    }
    return q;
}

template <int NT, int CG>
int64_t part_bytes(const TilePlan& q) {
    return (int64_t)q.sharers * CG * 2 * NT * kTileN * 4;
}

// The plan of a launch on `sms` SMs. Workspaces are sized and checked for kMaxSms:
// with fewer, tiles that need more than that are not shared.
template <int NT, int CG>
TilePlan launch_plan(int64_t M, int64_t N, int K, int sms) {
    TilePlan q = plan<NT, CG>(M, N, K, sms < kMaxSms ? sms : kMaxSms);
    if (part_bytes<NT, CG>(q) > part_bytes<NT, CG>(plan<NT, CG>(M, N, K, kMaxSms))) {
        q.waves += 1;
        q.split = q.sharers = 0;
    }
    return q;
}

// Tokens a tile: as few as hold M; beyond 128, single CTAs or pairs, whichever
// finishes first by what a step (0.52 and 0.60 us), a join and a result that nothing
// hides (0.7 and 1.5 us) take. Both were timed for M = 129 to 1500 in 12 sizes at
// (N, K) = (5120, 5120), (6144, 5120), (20480, 5120), (5120, 20480), (2565, 2576) and
// (2048, 2048): these weights take the faster at all 72. In a long run of steps single
// CTAs take 0.45 us a step and pairs 0.58; with 0.45 as the weight six of the sizes
// take the slower shape, by up to a quarter (M = 200, N = 20480, K = 5120: 49.5 us in
// single CTAs, 39.8 in pairs; M = 512, N = K = 5120: 30.0 and 29.0).
enum class Shape { kFew, k16, k32, k64, k128, kPair };

inline Shape choose(int64_t M, int64_t N, int K) {
    if (M <= 8) return Shape::kFew;
    if (M <= 16) return Shape::k16;
    if (M <= 32) return Shape::k32;
    if (M <= 64) return Shape::k64;
    if (M <= 128) return Shape::k128;
    auto ns = [](const TilePlan& q, uint32_t join, double step, double result) {
        const uint32_t shared = q.split ? (q.split + q.sharers - 1) / q.sharers + join : 0;
        return q.waves * (q.steps * step + result) + shared * step;
    };
    return ns(plan<128, 1>(M, N, K, kMaxSms), kJoinSteps<1>, 520, 700) <
                   ns(plan<256, 2>(M, N, K, kMaxSms), kJoinSteps<2>, 600, 1500)
               ? Shape::k128
               : Shape::kPair;
}

inline int64_t workspace_bytes(int64_t M, int64_t N, int K) {
    switch (choose(M, N, K)) {
    case Shape::kFew: return 0;
    case Shape::k16: return part_bytes<16, 1>(plan<16, 1>(M, N, K, kMaxSms));
    case Shape::k32: return part_bytes<32, 1>(plan<32, 1>(M, N, K, kMaxSms));
    case Shape::k64: return part_bytes<64, 1>(plan<64, 1>(M, N, K, kMaxSms));
    case Shape::k128: return part_bytes<128, 1>(plan<128, 1>(M, N, K, kMaxSms));
    default: return part_bytes<256, 2>(plan<256, 2>(M, N, K, kMaxSms));
    }
}

}  // namespace beam
