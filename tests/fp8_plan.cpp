// The division of the 8-bit floating-point product, for tests on the host.
#include "matmul_fp8_plan.h"

using namespace beam;

extern "C" {

void plan_fields(int64_t R, int experts, int64_t N, int K, const int* clusters, int64_t* out) {
    Fp8Room room;
    for (int i = 0; i < 4; ++i) room.clusters[i] = clusters[i];
    const Fp8Plan q = fp8_plan(R, experts, N, K, N % 16 == 0, room);
    out[0] = q.few;
    out[1] = q.width;
    out[2] = q.split;
    out[3] = q.clusters;
}

int plan_small(int64_t R, int experts, int64_t N, int K, const int* clusters) {
    Fp8Room room;
    for (int i = 0; i < 4; ++i) room.clusters[i] = clusters[i];
    return fp8_small(R, experts, N, K, fp8_plan(R, experts, N, K, N % 16 == 0, room));
}

int64_t plan_most_tiles(int64_t R, int experts, int most) { return fp8_most_tiles(R, experts, most); }

void plan_rows(int few, uint32_t n, uint32_t* out) {
    const Fp8Rows r = few ? fp8_rows<true>(n) : fp8_rows<false>(n);
    out[0] = r.tiles;
    out[1] = r.each;
}

void plan_place(uint32_t u, uint32_t m_tiles, uint32_t n_tiles, uint32_t* out) { fp8_place(u, m_tiles, n_tiles, out, out + 1); }

}
