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
constexpr int kFp8Many = 256;      // many: tiles of 256 tokens ...
constexpr int kFp8Width = 256;     // ... by up to 256 channels
constexpr int kFp8Band = 8;        // tiles of tokens that a band of tiles is high
constexpr int kFp8MaxSplit = 8;    // CTAs of a cluster at most

BEAM_HOST_DEVICE constexpr uint32_t fp8_up(uint32_t v, uint32_t to) { return (v + to - 1) / to; }

// n rows of one expert in tiles: as many as needed; few tokens alike as far as the matrix
// instruction's columns (multiples of 16) allow
struct Fp8Rows {
    uint32_t tiles, each;
};
template <bool FEW>
BEAM_HOST_DEVICE Fp8Rows fp8_rows(uint32_t n) {
    const uint32_t tiles = fp8_up(n, FEW ? kFp8Few : kFp8Many);
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

struct Fp8Plan {
    bool few;
    int width;      // channels of a tile
    int split;      // CTAs of a cluster, which share the steps of some tiles (few tokens only)
    int64_t tiles;  // at most
    int clusters;   // (many tokens: pairs)
};

// How many clusters of 1, 2, 4 and 8 CTAs (one an SM) with few tokens and how many pairs the device holds at a time
struct Fp8Room {
    int clusters[4];
    int pairs;
};

constexpr int kFp8JoinSteps = 4;  // what a join takes in steps

// Few tokens' tiles up to 64 rows an expert on average, where the weights' way from memory
// bounds the product; many tokens' beyond. Few tokens' tiles behind the last full wave
// are shared by clusters where that ends sooner, counted in steps.
inline Fp8Plan fp8_plan(int64_t R, int experts, int64_t N, int K, const Fp8Room& room) {
    const int64_t live = R < experts ? R : experts;
    Fp8Plan q{};
    q.few = R <= live * kFp8Few;
    q.width = q.few ? 128 : kFp8Width;
    q.tiles = fp8_most_tiles(R, experts, q.few ? kFp8Few : kFp8Many) * ((N + q.width - 1) / q.width);
    q.split = 1;
    int64_t fit = q.few ? room.clusters[0] : room.pairs;
    if (q.few) {
        const int64_t steps = (K + kFp8Step - 1) / kFp8Step;
        int64_t best = (q.tiles + fit - 1) / fit * steps;
        for (int i = 1; i < 4; ++i) {
            const int64_t split = 1 << i, clusters = room.clusters[i];
            if (clusters < 1 || split > steps) break;
            const int64_t waves = q.tiles / (clusters * split), rest = q.tiles - waves * clusters * split;
            const int64_t cost = waves * steps + (rest + clusters - 1) / clusters * ((steps + split - 1) / split + kFp8JoinSteps);
            if (cost < best) {
                best = cost;
                q.split = (int)split;
                fit = clusters;
            }
        }
    }
    q.clusters = (int)(q.tiles < fit ? q.tiles : fit);
    return q;
}

}  // namespace beam
