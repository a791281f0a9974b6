// How the 8-bit floating-point product is divided: tiles of tokens and channels, their
// order, the steps of k that several CTAs share. Arithmetic without CUDA, so that it
// can be tested anywhere.
#pragma once

#include <cmath>
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
constexpr int kFp8SmallRows = 512; // of experts whose rows go straight to registers, at most
constexpr int kFp8SmallPart = 8;   // ... of an expert's that a block has

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
// products and additions; a step with all SMs at work on weights that several tiles share, and on
// weights that one tile reads from memory (in proportion for fewer SMs); sharing a tile in a
// cluster, and for each of its CTAs; a tile's first step and stores, where rows of out are not whole
// sectors and where they are.
// Fitted, with the cost of rows that go straight to registers, to all kinds and splits at 702 sizes
// (dense: M from 2 to 3000, N from 640 to 20480, K from 256 to 20480; 382 products of 1 to 256
// experts with 0.1 to 3000 rows for each; operands not in L2): at these the choice takes 0.8% more than the
// best on average, over 5% at 20 and 19% at most, but for one (165 rows of 210 experts, N = 2432, K = 384: 52
// us and 41). With one cost a step, joins of 1600 to 3000 ns and, for experts, the most tiles that there can be,
// it was 11% for the dense ones, up to 62%, and 25% for experts, up to three times: M = 64, N =
// 6144, K = 1280: 11.3 -> 8.3 us; M = 128, N = 2565, K = 5120: 19.7 -> 13.4; 55 rows of 211 experts, N = 1383, K =
// 1152: 50 -> 23; 3045 of 166, N = 314, K = 336: 34 -> 21.
// Joins have since come to take 0.3 (few tokens) to 0.7 us more, at the cluster's scope. With that in the constants the
// choice would be another at 54 of 3000 random dense sizes, near ties all.
struct Fp8Cost {
    double alone, shared, once, join, tile, tile_of_sectors;
    double step(double ctas, int sms, double m_tiles) const {
        const double busy = (shared + (once - shared) / m_tiles) * ctas / sms;
        return busy > alone ? busy : alone;
    }
};
constexpr Fp8Cost kFp8FewCost{250, 530, 350, 3600, 300, 300}, kFp8NarrowCost{290, 300, 420, 2600, 1200, 200},
    kFp8WideCost{400, 390, 650, 5600, 2200, 300};
constexpr double kFp8JoinEach = 520;

// Experts that have rows, on average, if R rows fall among them alike
inline double fp8_live(int64_t R, int experts) {
    return experts == 1 ? 1.0 : experts * (1.0 - std::exp(-(double)R / experts));
}

// The split of tiles of one kind that ends first. Many tokens' shared tiles have one round at
// most. How many tiles experts make is known on the device only: here as many as rows that fall alike
// make on average, and clusters of two at most for many tokens.
inline Fp8Plan fp8_plan_of(bool few, int width, const Fp8Cost& cost, int64_t R, int experts, int64_t N, int K, bool sectors, const Fp8Room& room) {
    Fp8Plan best{};
    best.few = few;
    best.width = width;
    const double live = fp8_live(R, experts), most = fp8_most(few), per = R / live / most + 0.5;
    const int64_t n_tiles = (N + width - 1) / width, limit = fp8_most_tiles(R, experts, (int)most) * n_tiles;
    const double m_tiles = experts == 1 ? (double)fp8_most_tiles(R, 1, (int)most) : per > 1.0 ? per : 1.0;  // of an expert
    const int64_t tiles = experts == 1 ? limit : (int64_t)std::ceil(live * m_tiles * n_tiles);
    const int64_t steps = (K + kFp8Step - 1) / kFp8Step;
    const double tail = sectors ? cost.tile_of_sectors : cost.tile;
    for (int i = 0; i < 4; ++i) {
        const int64_t split = 1 << i, clusters = tiles < room.clusters[i] ? tiles : room.clusters[i];
        if (clusters < 1 || split > steps) continue;
        const int64_t ctas = clusters * split, waves = tiles / ctas, rest = tiles % ctas;
        if (i > 0 && !few && (rest > clusters || (experts > 1 && i > 1))) continue;
        const double step = cost.step((double)ctas, room.clusters[0], m_tiles);
        double ns = waves * (steps * step + tail);
        if (rest && i == 0) ns += steps * step + tail;
        else if (rest) ns += (rest + clusters - 1) / clusters * ((steps + split - 1) / split * step + cost.join + kFp8JoinEach * split + tail);
        if (best.clusters == 0 || ns < best.ns) {
            best.split = (int)split;
            best.clusters = (int)(limit < room.clusters[i] ? limit : room.clusters[i]);
            best.ns = ns;
        }
    }
    return best;
}

// Few tokens' tiles or many tokens', whichever end first. Up to 32 rows always the first: a copy
// of 128 rows of which the tensor has fewer than 32 takes twice as long (N = 20480, K = 5120, many
// tokens' tiles: 52 us for 1 to 16 rows, 24 us for 32 to 64).
inline Fp8Plan fp8_plan(int64_t R, int experts, int64_t N, int K, bool sectors, const Fp8Room& room) {
    const Fp8Plan few = fp8_plan_of(true, 128, kFp8FewCost, R, experts, N, K, sectors, room);
    if (R <= 32) return few;
    const Fp8Plan narrow = fp8_plan_of(false, 128, kFp8NarrowCost, R, experts, N, K, sectors, room);
    const Fp8Plan wide = fp8_plan_of(false, kFp8Width, kFp8WideCost, R, experts, N, K, sectors, room);
    const Fp8Plan& many = narrow.ns < wide.ns ? narrow : wide;
    return few.ns <= many.ns ? few : many;
}

// Whether rows go straight to registers. Dense: up to 8 tokens, unless few channels' long rows are better
// shared by clusters (M = 4: N = 2560, K = 20480 17.3 us and 19.4 in tiles, K = 65536 48.8 and 40.7, but N
// = 5120 64.7 and 70.7); up to 16 on up to 8192 channels (M = 16: N = 6144, K = 5120 10.8 and 14.7, K = 10240
// 18.6 and 20.1, but N = 12800, K = 5120 18.6 and 17.4; N = 2560, K = 20480 25.8 and 19.5). Experts: where the
// weights' way from memory, or a warp's blocks of k one after the other, and the further eights of an
// expert's rows end before the tiles do, less the 1.3 us by which those start later (55 rows of 211
// experts, N = 1383, K = 1152: 21 us and 29 in tiles; 252 of 18, N = 3601, K = 656: 24 and 20). Fitted while the
// eights of an expert followed one another in its blocks; they now have blocks of their own, which cost a tenth to a
// quarter less, and no more where rows do not fall alike.
inline bool fp8_small(int64_t R, int experts, int64_t N, int K, const Fp8Plan& tiles) {
    if (experts == 1) return R <= 8 ? K <= 20480 || N >= 4096 : R <= 16 && N <= 8192 && K <= 10240;
    if (R > kFp8SmallRows) return false;
    const double live = fp8_live(R, experts), per = R / live / 8 + 0.5;
    const double way = live * (double)N * K / 6000, chain = 900 * ((K + kFp8Step * 16 - 1) / (kFp8Step * 16));
    return (way > chain ? way : chain) * (1 + 0.7 * ((per > 1 ? per : 1) - 1)) - 1300 < tiles.ns;
}

}  // namespace beam
