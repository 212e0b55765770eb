// gemm_b128_stream_plan_check.cu -- host-only check of the block-scaled
// products' plans for M <= 64 (the kernel is compiled with the translation
// unit, never launched): shared memory within the opt-in limit, ring regions
// disjoint and aligned, the MMA's reads past a tile's rows and the exchange of
// sums inside the allocation, TMA boxes within 256, the MMA's N and the TMEM
// reads inside their buffer, scale reads inside their slot, unit counts of q or
// q + 1 per tile, every CTA's steps an exact partition of the blocks.
// Prints "ok <plans checked>" or the first violation.
#include "../up_projection_b200/csrc/gemm_b128_stream.cu"

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
    const int sides = gated ? 2 : 1;
    const int max_clusters[4] = {sms, sms / 2, sms * 4 / 5 / 4, sms * 4 / 5 / 8};
    const StreamPlan p = make_stream_plan(M, N, K, gated, mode == kRowScales, max_clusters);
    const int num_kb = (K + 127) / 128;
    if (p.stages < 2 || p.stages > kMaxStages || p.slots > kMaxSlots || p.slots < p.stages)
        return fail("ring", M, N, K, mode, sms);
    if (p.smem > kMaxSmem) return fail("shared memory", M, N, K, mode, sms);
    if (p.tiles < 1 || p.tiles > p.units || p.q < 1 || p.q != p.units / p.tiles)
        return fail("tiles", M, N, K, mode, sms);
    if (p.cluster != 1 && p.cluster != 2 && p.cluster != 4 && p.cluster != 8) return fail("cluster", M, N, K, mode, sms);
    if (p.cluster > kMaxCluster || p.cluster > num_kb) return fail("cluster size", M, N, K, mode, sms);
    if (p.a_rows < M || p.a_rows % 8 || p.a_rows > 128 || p.mma_n < M || p.mma_n % 16 || p.mma_n > 128)
        return fail("rows of A", M, N, K, mode, sms);
    const int hi = p.units % p.tiles ? p.q + 1 : p.q;
    if (p.rows != 8 * sides * hi || p.rows > 256 || (p.mma_m != 64 && p.mma_m != 128) || (p.mma_m == 64 && p.nrt != 1) ||
        p.nrt != (p.rows + p.mma_m - 1) / p.mma_m)
        return fail("weight rows", M, N, K, mode, sms);
    if (p.kbs > 8 || 4 * p.kbs > 32) return fail("TMA box", M, N, K, mode, sms);
    if (p.kbs % p.g || p.g * p.nrt * p.acc_cols > static_cast<int>(kBufCols) || p.mma_n > p.acc_cols)
        return fail("TMEM buffer", M, N, K, mode, sms);
    // the columns the two warps of a row read
    for (int half = 0; half < 2; ++half) {
        const int tok0 = p.parity ? 0 : p.tok * half;
        if (tok0 >= M) continue;
        if ((p.g * p.nrt - 1) * p.acc_cols + tok0 + p.tok > static_cast<int>(kBufCols))
            return fail("TMEM read", M, N, K, mode, sms);
    }
    if ((p.parity ? p.tok : 2 * p.tok) < M) return fail("rows per warp", M, N, K, mode, sms);
    if (p.stage_bytes % 1024 || p.off_slots % 128 || p.slot_bytes % 128 || p.slot_b % 128 || p.off_bar % 8)
        return fail("alignment", M, N, K, mode, sms);
    if (p.stage_bytes < static_cast<uint32_t>(p.kbs * (p.rows + p.a_rows)) * 128u ||
        p.off_bar < p.off_slots + p.slots * p.slot_bytes || p.smem < p.off_bar + 8 * kNumBars + 32 + 1024)
        return fail("regions", M, N, K, mode, sms);
    // scales: A's, then the weights' (row) or four per block
    const uint32_t weights = mode == kRowScales ? 4u * p.rows * p.kbs : 16u * p.kbs;
    if (p.slot_b < 4u * p.kbs * p.a_rows || p.slot_bytes < p.slot_b + weights) return fail("slot", M, N, K, mode, sms);
    if (p.off_slots + p.slots * p.slot_bytes + 512u > p.smem) return fail("scale reads past the slots", M, N, K, mode, sms);
    // MMA: 128 rows from every group of a block
    for (int cnt = p.q; cnt <= hi; ++cnt) {
        const int R = 8 * sides * cnt;
        const uint32_t last = (p.stages - 1) * p.stage_bytes +
                              static_cast<uint32_t>((p.kbs - 1) * R + ((R + p.mma_m - 1) / p.mma_m - 1) * 128) * 128u;
        if (last + static_cast<uint32_t>(p.mma_m) * 128u > p.off_slots) return fail("rows past the tile", M, N, K, mode, sms);
        // tile scales: at most four values
        for (int t = 0; t < p.tiles && mode != kRowScales; t += std::max(1, p.tiles / 7)) {
            const int u0 = static_cast<int>(static_cast<long long>(p.units) * t / p.tiles);
            const int n = static_cast<int>(static_cast<long long>(p.units) * (t + 1) / p.tiles) - u0;
            const int span = (8 * u0 + 8 * n - 1) / 128 - u0 / 16;
            if (span > (gated ? 1 : 3)) return fail("tile scales", M, N, K, mode, sms);
        }
    }
    // exchange of sums in the stages
    const int slices = p.cluster * (p.parity ? 2 : 1);
    if (p.part_m < (p.parity ? M : 2 * p.tok) ||
        4ull * slices * p.part_m * p.rows > static_cast<unsigned long long>(p.off_slots))
        return fail("exchange", M, N, K, mode, sms);
    for (int rank = 0; rank < p.cluster; ++rank) {
        const int b = static_cast<int>(static_cast<long long>(num_kb) * rank / p.cluster);
        const int e = static_cast<int>(static_cast<long long>(num_kb) * (rank + 1) / p.cluster);
        if (e <= b) return fail("empty share", M, N, K, mode, sms);
        int kb = b;
        while (kb < e) {
            const int nb = kb < p.full ? std::min(p.kbs, std::min(e, p.full) - kb) : 1;
            if (nb < 1) return fail("step", M, N, K, mode, sms);
            kb += nb;
        }
        if (kb != e) return fail("steps", M, N, K, mode, sms);
    }
    return 0;
}

}  // namespace

int main() {
    long checked = 0;
    const int Ms[] = {1, 7, 8, 9, 16, 17, 24, 31, 32, 33, 40, 48, 63, 64};
    const int Ks[] = {16, 128, 144, 256, 400, 1024, 1536, 2000, 4096, 14336, 1 << 20};
    for (int sms : {2, 16, 132, 148, 160})
        for (int mode = 0; mode < 3; ++mode)
            for (int M : Ms)
                for (int N = 8; N <= 40000; N += N < 1200 ? 8 : 264)
                    for (int K : Ks) {
                        if (check(M, N, K, mode, sms)) return 1;
                        ++checked;
                    }
    for (int mode = 0; mode < 3; ++mode)
        if (check(64, 1 << 20, 4096, mode, 148)) return 1;
    std::printf("ok %ld\n", checked);
    return 0;
}
