// How the 8-bit floating-point product is divided: tiles of tokens and channels, their
// order, the steps of k that several CTAs share. Arithmetic without CUDA, so that it
// can be tested anywhere.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define BEAM_HOST_DEVICE __host__ __device__
#else
#define BEAM_HOST_DEVICE
#endif

namespace beam {

constexpr int kFp8Step = 128;      // k of a step: the block that shares a scale
constexpr int kFp8Block128 = 128;  // channels that share a scale
constexpr int kFp8Few = 64;        // few tokens: tiles of 128 channels by up to 64 tokens
constexpr int kFp8Many = 128;      // many: tiles of 128 tokens
constexpr int kFp8Width = 256;     // ... by up to 256 channels
constexpr int kFp8Band = 8;        // tiles of tokens that a band of tiles is high
constexpr int kFp8MaxSplit = 8;    // CTAs of a cluster at most

BEAM_HOST_DEVICE constexpr uint32_t fp8_up(uint32_t v, uint32_t to) { return (v + to - 1) / to; }

// tokens of a tile at most
BEAM_HOST_DEVICE constexpr uint32_t fp8_most(bool few) { return few ? kFp8Few : kFp8Many; }

// n rows of one expert in tiles: as many as needed; few tokens alike as far as the matrix
// instruction's columns (multiples of 16) allow
struct Fp8Rows {
    uint32_t tiles, each;
};
template <bool FEW>
BEAM_HOST_DEVICE Fp8Rows fp8_rows(uint32_t n) {
    const uint32_t tiles = fp8_up(n, fp8_most(FEW));
    if (!FEW) return Fp8Rows{tiles, kFp8Many};
    return Fp8Rows{tiles, tiles ? fp8_up(fp8_up(n, tiles), 16) * 16 : 0u};
}

// Tile `u` of an expert's m by n tiles: bands of kFp8Band tiles of tokens, in a band
// channel by channel. The CTAs at work at a time then share about as many rows of
// tokens as of channels, and read the fewest bytes through L2.
BEAM_HOST_DEVICE inline void fp8_place(uint32_t u, uint32_t m_tiles, uint32_t n_tiles, uint32_t* m, uint32_t* n) {
    const uint32_t band = u / (kFp8Band * n_tiles), left = m_tiles - band * kFp8Band;
    const uint32_t high = left < kFp8Band ? left : kFp8Band, v = u - band * kFp8Band * n_tiles;
    *n = v / high;
    *m = band * kFp8Band + v % high;
}

// Tiles of R rows by `experts` experts at most (which rows are whose is known on the
// device only): every expert with rows has a tile that may not be whole.
inline int64_t fp8_most_tiles(int64_t R, int experts, int most) {
    const int64_t live = R < experts ? R : experts;
    return (R - live) / most + live;
}

// Whether rows go straight to registers. Up to 8 tokens, unless few channels' long rows are better
// shared by clusters (M = 4: N = 2560, K = 20480 17.3 us and 19.4 in tiles, K = 65536 48.8 and 40.7, but N
// = 5120 64.7 and 70.7); up to 16 on up to 8192 channels (M = 16: N = 6144, K = 5120 10.8 and 14.7, K = 10240
// 18.6 and 20.1, but N = 12800, K = 5120 18.6 and 17.4; N = 2560, K = 20480 25.8 and 19.5); up to 32 rows of
// experts, which seldom have more than 8 of them each (N = K = 5120: 32 rows of 31 experts 122 and 128, 64
// of 57 experts 225 and 214; 24 of 8 experts 35 and 49).
inline bool fp8_small(int64_t R, int experts, int64_t N, int K) {
    if (experts > 1) return R <= 32;
    return R <= 8 ? K <= 20480 || N >= 4096 : R <= 16 && N <= 8192 && K <= 10240;
}

// How many clusters of 1, 2, 4 and 8 CTAs (one an SM) the device holds at a time
struct Fp8Room {
    int clusters[4];
};

struct Fp8Plan {
    bool few;
    int width;      // channels of a tile
    int split;      // CTAs of a cluster, which share the steps of the tiles behind the last full wave
    int clusters;   // of the launch
    double ns;
};

// What tiles of a kind take, in ns: a step that waits for nothing but its own chain of loads,
// products and additions; a step with all SMs at work, which share the way to memory (in
// proportion for fewer); sharing a tile in a cluster: its launch, the sums' way, the wait for the
// last CTA. Fitted to all kinds and splits at 319 sizes (M from 2 to 3000, N from 640 to 20480, K
// from 256 to 20480, operands not in L2): the choice takes 0.9% more than the best on average, 14% at
// most but for one size, and over 5% at 19; a step without the first part, joins of 1600 to
// 3000 ns, 11% on average and up to 62%. M = 64, N = 6144, K = 1280: 11.3 -> 8.3 us; M = 128, N =
// 2565, K = 5120: 19.7 -> 13.4; M = 517, N = 640, K = 5120: 18.6 -> 12.9.
struct Fp8Cost {
    double alone, all, join;
    double step(int64_t ctas, int sms) const { return all * ctas > alone * sms ? all * ctas / sms : alone; }
};
constexpr Fp8Cost kFp8FewCost{200, 420, 3500}, kFp8NarrowCost{260, 350, 3500}, kFp8WideCost{380, 420, 5000};

// The split of tiles of one kind that ends first. Many tokens' shared tiles have one round at
// most; with offsets on the device the number of tiles is only known within bounds, so there
// clusters of two, which leave no SM out.
inline Fp8Plan fp8_plan_of(bool few, int width, const Fp8Cost& cost, int64_t R, int experts, int64_t N, int K, const Fp8Room& room) {
    Fp8Plan best{};
    best.few = few;
    best.width = width;
    const int64_t tiles = fp8_most_tiles(R, experts, (int)fp8_most(few)) * ((N + width - 1) / width);
    const int64_t steps = (K + kFp8Step - 1) / kFp8Step;
    for (int i = 0; i < 4; ++i) {
        const int64_t split = 1 << i, clusters = tiles < room.clusters[i] ? tiles : room.clusters[i];
        if (clusters < 1 || split > steps) continue;
        const int64_t ctas = clusters * split, waves = tiles / ctas, rest = tiles % ctas;
        if (i > 0 && !few && (rest > clusters || (experts > 1 && i > 1))) continue;
        const double step = cost.step(ctas, room.clusters[0]);
        double ns = waves * steps * step;
        if (rest && i == 0) ns += steps * step;
        else if (rest) ns += (rest + clusters - 1) / clusters * ((steps + split - 1) / split * step + cost.join);
        if (best.clusters == 0 || ns < best.ns) {
            best.split = (int)split;
            best.clusters = (int)clusters;
            best.ns = ns;
        }
    }
    return best;
}

// Few tokens' tiles or many tokens', whichever end first. Up to 32 rows always the first: a copy
// of 128 rows of which the tensor has fewer than 32 takes twice as long (N = 20480, K = 5120, many
// tokens' tiles: 52 us for 1 to 16 rows, 24 us for 32 to 64).
inline Fp8Plan fp8_plan(int64_t R, int experts, int64_t N, int K, const Fp8Room& room) {
    const Fp8Plan few = fp8_plan_of(true, 128, kFp8FewCost, R, experts, N, K, room);
    const Fp8Plan narrow = fp8_plan_of(false, 128, kFp8NarrowCost, R, experts, N, K, room);
    const Fp8Plan wide = fp8_plan_of(false, kFp8Width, kFp8WideCost, R, experts, N, K, room);
    const Fp8Plan& many = narrow.ns < wide.ns ? narrow : wide;
    return R <= 32 || few.ns <= many.ns ? few : many;
}

}  // namespace beam
