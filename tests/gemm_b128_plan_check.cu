// gemm_b128_plan_check.cu -- host-only check of the block-scaled products'
// tiles for M > 32 (the kernel is compiled with the translation unit, never
// launched): tiles cover the columns, TMA boxes within 256, the MMA's N legal
// and inside a TMEM buffer, every group's columns inside it.
// Prints "ok <plans checked>" or the first violation.
#include "../up_projection_b200/csrc/gemm_b128.cu"

#include <algorithm>
#include <cstdio>

namespace {

int fail(const char *what, int M, int N, int K, int mode, int pairs) {
    std::printf("violation: %s at M=%d N=%d K=%d mode=%d pairs=%d\n", what, M, N, K, mode, pairs);
    return 1;
}

int check(int M, int N, int K, int mode, int pairs) {
    using namespace swiglu;
    const bool gated = mode == kGated;
    const PairPlan p = make_pair_plan(M, N, K, gated, mode == kRowScales, pairs);
    if (p.tiles_m * 256ll < M || (p.tiles_m - 1) * 256ll >= M) return fail("row tiles", M, N, K, mode, pairs);
    if (p.groups * 32ll < N || (p.groups - 1) * 32ll >= N) return fail("groups", M, N, K, mode, pairs);
    if (p.tiles_n < 1 || p.tiles_n > p.groups) return fail("tiles", M, N, K, mode, pairs);
    if (static_cast<long long>(p.num_kb) * 128 < K) return fail("blocks", M, N, K, mode, pairs);
    if (p.half_rows % 16 || p.half_rows < 16 || p.half_rows > 128 || p.half_rows * 128u > kPairStageBytes - 16384u)
        return fail("B rows", M, N, K, mode, pairs);
    if (2 * p.half_rows % 32 || 2 * p.half_rows > kPairBufCols) return fail("MMA columns", M, N, K, mode, pairs);
    if (p.s_cols > 256 || (mode == kRowScales && p.s_cols != 2 * p.half_rows))
        return fail("scale box", M, N, K, mode, pairs);
    for (int t = 0; t < p.tiles_n; ++t) {
        const int g0 = static_cast<int>(static_cast<long long>(p.groups) * t / p.tiles_n);
        const int cnt = static_cast<int>(static_cast<long long>(p.groups) * (t + 1) / p.tiles_n) - g0;
        if (cnt < 1 || (gated ? 32 : 16) * cnt > p.half_rows) return fail("groups per tile", M, N, K, mode, pairs);
        for (int half = 0; half < 2; ++half) {
            const int first = half ? (cnt + 1) / 2 : 0, mine = half ? cnt / 2 : (cnt + 1) / 2;
            if (mine > (gated ? 2 : 4)) return fail("groups per warp", M, N, K, mode, pairs);
            const int read = mine == 0 ? 0 : (gated ? 4 : (mine + 1) / 2 * 2);
            for (int o = 0; o < read; ++o) {
                const int col0 = 32 * first, col2 = gated ? col0 + p.half_rows : col0 + 64;
                const int col = (o < 2 ? col0 : col2) + 32 * (o & 1);
                if (kPairBufCols + col + 32 > kTmemCols) return fail("TMEM read", M, N, K, mode, pairs);
                if (mode == kRowScales && 4 * (3 * p.s_cols + col + 32) > kSlotBlocks * 1024)
                    return fail("scale read", M, N, K, mode, pairs);
            }
        }
    }
    return 0;
}

}  // namespace

int main() {
    long checked = 0;
    const int Ms[] = {33, 64, 65, 128, 129, 256, 257, 300, 1000, 2048, 4097, 8192, 100000};
    const int Ks[] = {16, 128, 144, 1536, 14336, 1 << 20};
    for (int pairs : {1, 4, 66, 72, 74, 80})
        for (int mode = 0; mode < 3; ++mode)
            for (int M : Ms)
                for (int N = 8; N <= 16384; N += N < 1200 ? 8 : 264)
                    for (int K : Ks) {
                        if (check(M, N, K, mode, pairs)) return 1;
                        ++checked;
                    }
    for (int mode = 0; mode < 3; ++mode)
        if (check(8192, 1 << 20, 4096, mode, 74)) return 1;
    std::printf("ok %ld\n", checked);
    return 0;
}
