// The division of the 8-bit integer product, for tests on the host.
#include "matmul_int8_plan.h"

#include <algorithm>

using namespace beam;

namespace {

template <class F>
void with_shape(int shape, F f) {
    switch ((Shape)shape) {
    case Shape::kFew: return;
    case Shape::k16: return f.template operator()<16, 1>();
    case Shape::k32: return f.template operator()<32, 1>();
    case Shape::k64: return f.template operator()<64, 1>();
    case Shape::k128: return f.template operator()<128, 1>();
    default: return f.template operator()<256, 2>();
    }
}

}  // namespace

extern "C" {

int plan_choose(int64_t M, int64_t N, int K) { return (int)choose(M, N, K); }
int plan_whole_channels(int N, int n0) { return whole_channels(N, n0); }
int64_t plan_workspace(int64_t M, int64_t N, int K) { return workspace_bytes(M, N, K); }

// m_tiles, steps, tiles, waves, workers, sharers, split, bytes of partial sums
void plan_fields(int shape, int64_t M, int64_t N, int K, int sms, int64_t* out) {
    with_shape(shape, [&]<int NT, int CG>() {
        const TilePlan q = plan<NT, CG>(M, N, K, sms);
        const int64_t v[8] = {q.m_tiles, q.steps, q.tiles, q.waves, q.workers, q.sharers, q.split, part_bytes<NT, CG>(q)};
        std::copy(v, v + 8, out);
    });
}

// the same for the plan of a launch on a device of `sms` SMs
void launch_fields(int shape, int64_t M, int64_t N, int K, int sms, int64_t* out) {
    with_shape(shape, [&]<int NT, int CG>() {
        const TilePlan q = launch_plan<NT, CG>(M, N, K, sms);
        const int64_t v[8] = {q.m_tiles, q.steps, q.tiles, q.waves, q.workers, q.sharers, q.split, part_bytes<NT, CG>(q)};
        std::copy(v, v + 8, out);
    });
}

}
