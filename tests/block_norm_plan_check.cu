// block_norm_plan_check.cu -- host-only check of the block norms' ring plans (the
// kernels are compiled with the translation unit, never launched): whatever the shape, the rings,
// sums and meeting places fit the shared memory that is opted in to, groups and
// threads stay inside the kernels' arrays and barriers, and the rows of all
// items are every row once.  Prints "ok <plans checked>" or the first violation.
#include "../up_projection_b200/csrc/block_norm.cu"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>

using namespace swiglu;

#define REQUIRE(c)                                                                                    \
    do {                                                                                              \
        if (!(c)) {                                                                                   \
            std::printf("violation: %s at M=%lld D=%d f32=%d gates=%lld\n", #c, (long long)M, D, f32,    \
                        (long long)gates);                                                            \
            std::exit(1);                                                                             \
        }                                                                                             \
    } while (0)

static int checked = 0;

static void check(int64_t M, int D, int f32, int64_t gates, int sms) {
    const int nvec = D / (f32 ? 4 : 8);
    const RingShape s = ring_shape(D, f32, true), fs = ring_shape(D, f32, false);
    REQUIRE(s.T % 32 == 0 && s.T * s.v >= nvec && s.T <= kRingThreads);
    REQUIRE(s.groups >= 1 && s.groups <= kMaxGroups && s.groups * s.T <= kRingThreads);
    REQUIRE(s.T == 32 || s.groups <= 8);   // slots and named barriers
    REQUIRE(f32 ? (s.v == 2 || s.v == 4) : (s.v == 1 || s.v == 2 || s.v == 4));
    if (nvec >= 64 && fs.v * (f32 ? 4 : 8) <= 16) {   // the forward's ring
        REQUIRE(fs.v == (f32 ? 4 : 2) && fs.T % 32 == 0 && fs.T * fs.v >= nvec && fs.T <= kRingThreads);
        REQUIRE(fs.groups >= 1 && fs.groups <= kMaxGroups && fs.groups * fs.T <= kRingThreads);
        REQUIRE(fs.T == 32 || fs.groups <= 8);
        const uint32_t row = 2u * 16u * fs.v * fs.T;
        REQUIRE(kRingRoom / (row * fs.groups) >= 2);
    }
    const bool per_row = gates > 1;
    const BwdPlan p = bwd_plan(M, D, f32, per_row, gates, true, true, true, sms);
    const uint32_t pitch = 16u * p.v * p.T;
    REQUIRE(p.groups >= 1 && p.groups <= s.groups && p.stages >= 1 && p.stages <= kMaxRing);
    const uint32_t rings = p.groups * p.stages * 4u * pitch;
    const uint32_t sums = per_row ? 4u * D * (1u + (p.groups > 1 ? p.groups : 0u)) : 0u;
    REQUIRE(p.smem == rings + sums && p.smem <= kRingRoom);
    REQUIRE((p.groups - 1) * 2u * D * 4u <= rings);          // the groups' sums meet in the rings
    REQUIRE(p.blocks >= 1 && p.blocks <= sms && p.splits >= 1);
    const int64_t per = M / gates;
    REQUIRE(p.groups <= per && p.splits <= per);
    const int64_t items = gates * p.splits;
    REQUIRE(p.blocks == (items < sms ? items : sms));
    size_t floats = 2 * static_cast<size_t>(p.blocks) * D + (per_row && p.splits > 1 ? static_cast<size_t>(items) * D : 0);
    REQUIRE(p.bytes == 4 * floats);
    int64_t at = 0;
    for (int64_t item = 0; item < items; ++item) {
        const int64_t gr = item / p.splits, sp = item - gr * p.splits;
        const int64_t each = per / p.splits, longer = per % p.splits;
        const int64_t row0 = gr * per + sp * each + std::min(sp, longer), row1 = row0 + each + (sp < longer ? 1 : 0);
        REQUIRE(row0 == at && row1 > row0 && row1 <= (gr + 1) * per);
        at = row1;
    }
    REQUIRE(at == M);
    ++checked;
}

int main(int argc, char **argv) {
    const int n = argc > 1 ? std::atoi(argv[1]) : 20000;
    std::mt19937 rng(7);
    auto log_up_to = [&](int64_t top) {
        const double x = std::exp(std::log(static_cast<double>(top)) * std::uniform_real_distribution<>(0, 1)(rng));
        return std::min<int64_t>(top, std::max<int64_t>(1, static_cast<int64_t>(x)));
    };
    for (int f32 = 0; f32 < 2; ++f32)   // every row length
        for (int nvec = 1; nvec <= 2048; ++nvec)
            for (int64_t gates : {1, 2, 12}) check(gates * 37, nvec * (f32 ? 4 : 8), f32, gates, 148);
    for (int i = 0; i < n; ++i) {
        const int f32 = rng() & 1, D = static_cast<int>(log_up_to(2048)) * (f32 ? 4 : 8);
        const int64_t gates = rng() & 1 ? 1 : log_up_to(400);
        check(gates * log_up_to(2000), D, f32, gates, rng() & 1 ? 148 : 1 + static_cast<int>(rng() % 200));
    }
    std::printf("ok %d\n", checked);
    return 0;
}
