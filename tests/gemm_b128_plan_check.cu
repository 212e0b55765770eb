// gemm_b128_plan_check.cu -- host-only check of the block-scaled products'
// launch plans (the kernel is compiled with the translation unit, never
// launched): shared memory within the opt-in limit, ring regions disjoint and
// aligned, the A operand's reads past its box and the B operand's reads of an
// odd unit count inside the allocation, TMA boxes within 256, TMEM reads and
// MMA writes inside their buffer, unit counts of q or q + 1 per tile.
// Prints "ok <plans checked>" or the first violation.
#include "../up_projection_b200/csrc/gemm_b128.cu"

#include <algorithm>
#include <cstdio>

namespace {

int fail(const char *what, int M, int N, int K, int mode, int sms) {
    std::printf("violation: %s at M=%d N=%d K=%d mode=%d sms=%d\n", what, M, N, K, mode, sms);
    return 1;
}

int check(int M, int N, int K, int mode, int sms) {
    using namespace swiglu;
    const bool gated = mode == kGated;
    const Plan p = make_plan(M, N, K, gated, mode == kRowScales, sms);
    if (p.smem > kMaxSmem) return fail("shared memory", M, N, K, mode, sms);
    if (p.bufs < 2 || p.bufs > kMaxBufs || p.bufs * p.buf_cols > kTmemCols)
        return fail("TMEM buffers", M, N, K, mode, sms);
    if (p.stages < 2 || p.stages > kMaxStages || p.slots > kMaxSlots || p.slots < p.stages)
        return fail("ring", M, N, K, mode, sms);
    if (p.tiles_n < 1 || p.tiles_n > p.units || p.q < 1 || p.q != p.units / p.tiles_n)
        return fail("tiles", M, N, K, mode, sms);
    if (p.tiles_m * 128ll < M || (p.tiles_m - 1) * 128ll >= M) return fail("row tiles", M, N, K, mode, sms);
    if (static_cast<long long>(p.num_kb) * 128 < K) return fail("blocks", M, N, K, mode, sms);
    const int hi = p.units % p.tiles_n ? p.q + 1 : p.q;
    if (8 * hi > 256 || p.a_rows > 128 || p.a_rows % 8 || p.s_cols > 256)
        return fail("TMA box", M, N, K, mode, sms);
    if (mode == kRowScales && p.s_cols != 8 * hi) return fail("scale box", M, N, K, mode, sms);
    if (p.slot_bytes < 512u + 4u * p.s_cols) return fail("scale slot", M, N, K, mode, sms);
    if (p.stage_bytes % 1024 || p.off_slots % 128 || p.slot_bytes % 128 || p.off_out % 16 || p.off_bar % 8)
        return fail("alignment", M, N, K, mode, sms);
    if (p.off_out < p.off_slots + p.slots * p.slot_bytes || p.off_bar < p.off_out + kEpiWarps * kStageOutBytes ||
        p.smem < p.off_bar + 8 * kNumBars + 32 + 1024)
        return fail("regions", M, N, K, mode, sms);
    // the last stage's A operand is read 128 rows deep
    if (p.stages * p.stage_bytes - p.stage_bytes + 128u * 128u > p.off_slots)
        return fail("A rows past the box", M, N, K, mode, sms);
    for (int cnt = p.q; cnt <= hi; ++cnt) {
        const int cols = (gated ? 16 : 8) * cnt;
        const int mma_n = (cols + 15) / 16 * 16;
        if (mma_n > 256 || mma_n > p.buf_cols) return fail("MMA columns", M, N, K, mode, sms);
        if (mma_n > p.b_rows) return fail("B rows", M, N, K, mode, sms);
        const int split = std::min(cnt, ((cnt + 1) / 2 + 3) / 4 * 4);
        for (int half = 0; half < 2; ++half) {
            const int first = half ? split : 0, mine = half ? cnt - split : split;
            if (mine > (gated ? 8 : 16)) return fail("units per warp", M, N, K, mode, sms);
            for (int j = 0; j < 4; ++j) {
                if (4 * (gated ? (j & 1) : j) >= mine) continue;
                const int c0 = 8 * first, c2 = gated ? c0 + 8 * cnt : c0 + 64;
                const int col = (j < 2 ? c0 : c2) + 32 * (j & 1);
                if (col + 32 > p.buf_cols) return fail("TMEM read", M, N, K, mode, sms);
                if (mode == kRowScales && 512u + 4u * (col + 32) > p.slot_bytes)
                    return fail("scale read", M, N, K, mode, sms);
            }
        }
    }
    return 0;
}

}  // namespace

int main() {
    long checked = 0;
    const int Ms[] = {1, 7, 8, 9, 64, 127, 128, 129, 256, 300, 1000, 2048, 4097, 8192, 100000};
    const int Ks[] = {16, 128, 144, 1536, 4096, 14336, 1 << 20};
    for (int sms : {1, 8, 132, 148, 160})
        for (int mode = 0; mode < 3; ++mode)
            for (int M : Ms)
                for (int N = 8; N <= 16384; N += N < 1200 ? 8 : 264)
                    for (int K : Ks) {
                        if (check(M, N, K, mode, sms)) return 1;
                        ++checked;
                    }
    for (int mode = 0; mode < 3; ++mode)
        if (check(8192, 1 << 20, 4096, mode, 148)) return 1;
    std::printf("ok %ld\n", checked);
    return 0;
}
