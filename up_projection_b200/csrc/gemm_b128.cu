// gemm_b128.cu -- products of e4m3 operands with one fp32 scale per block of
// 128 along the reduction, on the fp8 tensor cores (tcgen05 kind::f8f6f4):
//
//   Y[m, n] = sum_b As[m, b] Bs[n, b] sum_{k in block b} A[m, k] B[n, k]
//
// with Bs one value per row of B ("row") or per 128 rows ("tile"); and the
// gated pair, H = act(alpha G) * U with G and U such products of one A.  This
// file: all but the few rows (b128_few_rows) of gemm_b128_stream.cu.
//
// The scales differ from block to block, so the tensor cores accumulate one
// 128-deep block only: four MMAs (K = 32) into one of two buffers of tensor
// memory, which eight warps read back, multiply by the block's scales and add
// to the running sums in their registers (fp32, round to nearest: 128 x 256
// sums are 128 registers of 256 threads), while the next block's MMAs fill the
// other buffer.
//
// Each MMA covers 256 rows over the two CTAs of a cluster (cta_group::2).  A
// CTA holds its own 128 rows of A and half of the tile's rows of B (gated: the
// even CTA the rows of Wg, the odd one those of Wu), so a stage is 32 KB
// instead of 48 and both the copies' writes and the MMAs' reads of shared
// memory shrink by a third; each CTA accumulates its own 128 rows.
//
//  * warps 0..7: accumulation and epilogue: warp w holds rows 32 (w mod 4)
//    .. +31 and half of the tile's columns;
//  * warp 8, 10 (one thread each): TMA producers of B and of A; one thread
//    issuing every copy took longer than a block's MMAs;
//  * warp 11: the scales, in slots of four blocks (they outlive the stages:
//    the accumulating warps free them, later than the MMAs free a stage);
//  * warp 9 of the even CTA (one thread): MMA issuer for the pair.
//
// Waits are bounded; a stuck pipeline sets the status word, the MMAs and
// copies in flight are drained and TMEM is freed before the kernel returns.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "b128.cuh"
#include "kernels.cuh"
#include "status.cuh"
#include "tmap.cuh"

namespace swiglu {

// Status word of this translation unit's kernel (bit 0 = a wait gave up).
__device__ unsigned int g_gemm_b128_status;

namespace {

using namespace b128;
using gemm::tile_coords;

constexpr int kGroupM = 8;        // 256-row tiles per raster group
constexpr int kPairStages = 4;
constexpr int kSlotBlocks = 4;    // blocks of the reduction per slot of scales
constexpr int kPairBufCols = 256;
constexpr uint32_t kPairStageBytes = 32 * 1024;
constexpr int kPairMaxSlots = 4;
constexpr uint32_t kPairBars = 2 * kPairStages + 2 * kPairMaxSlots + 2 * 2 + 1;

// Output staging of a warp: 32 rows by 32 columns leave by one TMA store, so
// the warp goes on to its next tile while they drain.
constexpr uint32_t kOutBytes = 8192;   // four such boxes of bf16, two of fp32

template <int kMode>
struct PairLayout {
    // per slot: row scales of A [4][128], then of B [4][s_cols], or tile
    // scales [4][half of the tile][group of the half]
    static constexpr int kSlots = kMode == kRowScales ? 2 : 4;
    static constexpr uint32_t kOffB = kSlotBlocks * 512;
    static constexpr uint32_t kSlotBytes = kOffB + kSlotBlocks * (kMode == kRowScales ? 1024 : 32);
    static constexpr uint32_t kOffOut = kPairStages * kPairStageBytes;
    static constexpr uint32_t kOffSlots = kOffOut + kEpiWarps * kOutBytes;
    static constexpr uint32_t kOffBar = kOffSlots + kSlots * kSlotBytes;
    static constexpr uint32_t kSmem = kOffBar + 8 * kPairBars + 32 + 1024;
    static_assert(kSmem <= kMaxSmem, "exceeds the 227 KB opt-in shared memory");
};

struct PairPlan {
    int tiles_m, tiles_n;
    int groups;      // of 32 output columns
    int half_rows;   // rows of B per CTA and stage: half the MMA's N
    int s_cols;      // row scales of B per block
    int num_kb;
};

__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    const uint32_t z = 0;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;"
        "\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(z)
        : "memory");
}

// Arrive on the barrier at this offset of both CTAs' shared memory when every
// MMA issued so far by this thread has completed.
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        "\n\t}\n" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// The same on this CTA's barrier alone.
__device__ __forceinline__ void mma_commit_own(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
        : "memory");
}

// 16 lanes x 32 columns of TMEM as fragments: registers 4 j .. + 3 hold columns
// 8 j + 2 (lane mod 4), + 1 of rows lane / 4 and lane / 4 + 8.
template <int kAt>
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[kAt]), "=r"(r[kAt + 1]), "=r"(r[kAt + 2]), "=r"(r[kAt + 3]), "=r"(r[kAt + 4]),
          "=r"(r[kAt + 5]), "=r"(r[kAt + 6]), "=r"(r[kAt + 7]), "=r"(r[kAt + 8]), "=r"(r[kAt + 9]),
          "=r"(r[kAt + 10]), "=r"(r[kAt + 11]), "=r"(r[kAt + 12]), "=r"(r[kAt + 13]), "=r"(r[kAt + 14]),
          "=r"(r[kAt + 15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void sts_b32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sts_b64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// A block's 32 columns of a warp's 32 rows into its running sums, with row
// scales.  A lane that holds a whole row needs all 32 of B's scales, 512 bytes
// a warp for every 128-byte broadcast; as fragments (sums 8 h + 2 j + i: rows
// 16 h + 8 i + lane / 4, columns 8 j + 2 (lane mod 4), + 1) it needs 8 of them
// and four of A's.  sb: the scales of this lane's first two columns.
__device__ __forceinline__ void add_fragments(unsigned long long (&acc)[16], const uint32_t (&v)[32],
                                              const float (&sa)[4], uint32_t sb) {
    unsigned long long sa2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sa2[i] = pair2(sa[i], sa[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        unsigned long long w;
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w) : "r"(sb + 32u * j));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                fma2(acc[8 * h + 2 * j + i], v[16 * h + 4 * j + 2 * i], v[16 * h + 4 * j + 2 * i + 1],
                     mul2(w, sa2[2 * h + i]));
    }
}

// tm_b: rows of B (gated: of Wg), tm_u: of Wu, boxes of half_rows rows.
template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    swiglu_gemm_b128_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                                 const __grid_constant__ CUtensorMap tm_as,
                                 const __grid_constant__ CUtensorMap tm_b,
                                 const __grid_constant__ CUtensorMap tm_u,
                                 const __grid_constant__ CUtensorMap tm_bs,
                                 const __grid_constant__ CUtensorMap tm_y,
                                 const __grid_constant__ CUtensorMap tm_yg,
                                 const __grid_constant__ CUtensorMap tm_yu,
                                 const float *bs0, const float *bs1,
                                 const Out out, int M, int N, const PairPlan p) {
    using L = PairLayout<kMode>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar_full = base + L::kOffBar;
    const uint32_t bar_empty = bar_full + 8 * kPairStages;
    const uint32_t bar_sfull = bar_empty + 8 * kPairStages;
    const uint32_t bar_sempty = bar_sfull + 8 * kPairMaxSlots;
    const uint32_t bar_tfull = bar_sempty + 8 * kPairMaxSlots;
    const uint32_t bar_tempty = bar_tfull + 16;
    const uint32_t bar_drain = bar_tempty + 16;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(gbase + L::kOffBar + 8 * kPairBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::kOffBar + 8 * kPairBars + 16);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (known uniform)
    const int lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = static_cast<int>(blockIdx.x) / 2;
    const int num_pairs = static_cast<int>(gridDim.x) / 2;
    const int num_tiles = p.tiles_m * p.tiles_n;
    const int num_kb = p.num_kb;
    const uint32_t a_bytes = kBM * 128u;
    const uint32_t b_bytes = static_cast<uint32_t>(p.half_rows) * 128u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(bar_sfull + 8 * s, 1);
            mbar_init(bar_sempty + 8 * s, kEpiWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 2 * kEpiWarps);  // both CTAs' warps
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_as);
        // (tm_u is left to its first use: naming it here by rank made the
        // compiler keep the loop's uniform values in spilled registers)
        tma_prefetch_desc(&tm_b);
        if (kMode == kRowScales) tma_prefetch_desc(&tm_bs);
        tma_prefetch_desc(&tm_y);
    }
    if (warp == kEpiWarps + 1) {
        tmem_alloc_pair(smem_u32(tmem_ptr), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    // both CTAs' barriers initialised and TMEM allocated before any copy,
    // arrive or MMA that reaches the other CTA
    cluster_sync_all();
    tc_fence_after();
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_ptr);

    // tile t: the CTA's rows m0 .., the tile's groups g0 .. g0 + cnt of 32 columns
    auto tile_of = [&](int t, int &m0, int &g0, int &cnt) {
        int mt, nt;
        tile_coords<kGroupM>(t, p.tiles_m, p.tiles_n, mt, nt);
        m0 = mt * 2 * kBM + static_cast<int>(rank) * kBM;
        g0 = static_cast<int>(static_cast<long long>(p.groups) * nt / p.tiles_n);
        cnt = static_cast<int>(static_cast<long long>(p.groups) * (nt + 1) / p.tiles_n) - g0;
    };

    bool failed = false;

    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if ((warp == kEpiWarps || warp == kEpiWarps + 2) && lane == 0) {
            // ----------------------- TMA producers: B (and the bytes of all), A
            const bool is_b = warp == kEpiWarps;
            const uint32_t full_r0 = map_to_rank(bar_full, 0);
            const CUtensorMap *tm = !is_b ? &tm_a : (kMode == kGated && rank == 1 ? &tm_u : &tm_b);
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            for (int t = pair; t < num_tiles && !failed; t += num_pairs) {
                int m0, g0, cnt;
                tile_of(t, m0, g0, cnt);
                const int row = !is_b ? m0 : 32 * g0 + (kMode == kGated ? 0 : static_cast<int>(rank) * p.half_rows);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait_long(bar_empty + 8 * stage, phase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    }
                    // every copy of both CTAs is counted on the even CTA's barrier
                    if (is_b && rank == 0) mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * (a_bytes + b_bytes));
                    tma_load_2d_pair(tm, full_r0 + 8 * stage,
                                     base + stage * kPairStageBytes + (is_b ? a_bytes : 0u), kb * kBlockK, row);
                    ++issued;
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Never leave while a load may still write shared memory: the even
            // CTA's barriers count both CTAs' copies, and every block of the
            // odd CTA is consumed by the pair's MMAs before the last barrier.
            for (int s = 0; s < kPairStages && rank == 0; ++s)
                if (issued > s)
                    mbar_wait_drain(bar_full + 8 * s,
                                    static_cast<uint32_t>(((issued - 1 - s) / kPairStages) & 1));
        }
        if (warp == kEpiWarps + 3) {
            // ------------------------------------------------------ scales
            int slot = 0;
            uint32_t phase = 0;
            long long issued = 0;
            for (int t = pair; t < num_tiles && !failed; t += num_pairs) {
                int m0, g0, cnt;
                tile_of(t, m0, g0, cnt);
                // tile scales: lane = (block, half of the tile, group of the
                // half), the value its accumulating warps multiply by
                const float *src = nullptr;
                if (kMode != kRowScales) {
                    const int j = lane & 3;
                    const int group = g0 + ((lane & 4) ? (cnt + 1) / 2 : 0) + (kMode == kGated ? (j & 1) : j);
                    const float *table = (kMode == kGated && (j & 2)) ? bs1 : bs0;
                    src = table + static_cast<int64_t>(min(group / 4, (N + 127) / 128 - 1)) * num_kb;
                }
                for (int kb = 0; kb < num_kb; kb += kSlotBlocks) {
                    float v = 0.0f;
                    if (kMode != kRowScales) v = ld_plain(src + min(kb + lane / 8, num_kb - 1));
                    if (!mbar_wait_long(bar_sempty + 8 * slot, phase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    }
                    const uint32_t sb = bar_sfull + 8 * slot;
                    const uint32_t dst = base + L::kOffSlots + slot * L::kSlotBytes;
                    if (kMode != kRowScales) {
                        sts_f32(dst + L::kOffB + 4u * lane, v);
                        __syncwarp();
                    }
                    if (lane == 0) {
                        // (blocks past the last arrive as zeros)
                        mbar_arrive_expect_tx(sb, kSlotBlocks * (512u + (kMode == kRowScales ? 4u * p.s_cols : 0u)));
                        tma_load_2d(&tm_as, sb, dst, m0, kb);
                        if (kMode == kRowScales) tma_load_2d(&tm_bs, sb, dst + L::kOffB, 32 * g0, kb);
                    }
                    ++issued;
                    if (++slot == L::kSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < L::kSlots; ++s)
                if (issued > s)
                    mbar_wait_drain(bar_sfull + 8 * s,
                                    static_cast<uint32_t>(((issued - 1 - s) / L::kSlots) & 1));
        }
        if (warp == kEpiWarps + 1 && rank == 0) {
            // ----------------------------- MMA issuer for the pair (whole warp)
            const uint32_t idesc = make_idesc(0u, 2 * kBM, static_cast<uint32_t>(2 * p.half_rows));
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            for (int t = pair; t < num_tiles && !failed; t += num_pairs) {
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait_long(bar_full + 8 * stage, phase, abort_flag) ||
                        !mbar_wait_long(bar_tempty + 8 * buf, bphase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = base + stage * kPairStageBytes;
                    const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(a + a_bytes);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kPairBufCols);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8_pair(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                    mma_commit_both(bar_empty + 8 * stage);
                    mma_commit_both(bar_tfull + 8 * buf);
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
            // Every MMA issued here must finish before TMEM is released.
            mma_commit_own(bar_drain);
            mbar_wait_drain(bar_drain, 0);
        }
    } else {
        // ------------------------------------------ accumulation + epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t obuf = base + L::kOffOut + static_cast<uint32_t>(warp) * kOutBytes;
        int onext = 0;  // next staging box
        const uint32_t tempty_r0 = map_to_rank(bar_tempty, 0);
        int slot = 0;
        uint32_t buf8 = 0;            // 8 x the TMEM buffer in turn
        uint32_t pa = 0, pb = 0;      // the next block's scales of A (this row's) and of B
        uint32_t sphase = 0, bphase = 0;
        for (int t = pair; t < num_tiles && !failed; t += num_pairs) {
            int m0, g0, cnt;
            tile_of(t, m0, g0, cnt);
            // this warp's groups of 32 columns: the lower or upper half of the
            // tile's (gated: of both products)
            const int first = half ? (cnt + 1) / 2 : 0;
            const int mine = half ? cnt / 2 : (cnt + 1) / 2;
            const int rows = min(32, M - m0 - 32 * quad);  // <= 0: none
            const uint32_t col0 = 32u * static_cast<uint32_t>(first);
            const uint32_t col2 = kMode == kGated ? col0 + static_cast<uint32_t>(p.half_rows) : col0 + 64u;
            // groups are read in pairs (an odd count reads one more, gated always
            // all four; sums of columns beyond the tile are not stored)
            const int groups = rows <= 0 || mine == 0 ? 0 : (kMode == kGated ? 4 : (mine + 1) / 2 * 2);
            unsigned long long acc[4][16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][i] = 0ull;
            constexpr bool kFrag = kMode == kRowScales;
            float sa[kFrag ? 4 : 1] = {}, sb[4] = {};
            uint32_t srow = 0;        // this block's row scales of B
            uint32_t v[2][32];
            auto read_group = [&](uint32_t at, uint32_t (&r)[32]) {
                if constexpr (kFrag) {
                    tmem_ld_16x256b_x4<0>(at, r);
                    tmem_ld_16x256b_x4<16>(at + (16u << 16), r);
                } else {
                    tmem_ld_32x32b_x32(at, r);
                }
            };
            // One block ahead: wait for its accumulators, start reading them,
            // and fetch its scales.
            auto open_block = [&](bool new_slot) -> bool {
                if (new_slot) {
                    if (!mbar_wait_long(bar_sfull + 8 * slot, sphase, abort_flag)) return false;
                    pa = base + L::kOffSlots + slot * L::kSlotBytes + 4u * (quad * 32 + (kFrag ? lane >> 2 : lane));
                    pb = base + L::kOffSlots + slot * L::kSlotBytes + L::kOffB + (kFrag ? 8u * (lane & 3) : 16u * half);
                }
                if (!mbar_wait_long(bar_tfull + buf8, bphase, abort_flag)) return false;
                tc_fence_after();
                if (groups == 0) return true;
                read_group(lanes + 32u * buf8 + col0, v[0]);
#pragma unroll
                for (int i = 0; i < (kFrag ? 4 : 1); ++i) sa[i] = lds_f32(pa + 32u * i);
                pa += 512u;
                if constexpr (!kFrag) {
                    const uint4 w = lds_v4(pb);
                    pb += 32u;
                    sb[0] = __uint_as_float(w.x);
                    sb[1] = __uint_as_float(w.y);
                    sb[2] = __uint_as_float(w.z);
                    sb[3] = __uint_as_float(w.w);
                } else {
                    srow = pb;
                    pb += 4u * static_cast<uint32_t>(p.s_cols);
                }
                return true;
            };
            if (!open_block(true)) {
                failed = true;
                break;
            }
            for (int kb = 0; kb < num_kb; ++kb) {
                const uint32_t d = lanes + 32u * buf8;
                float s[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = sa[0] * sb[j];
                float sa_now[kFrag ? 4 : 1];
#pragma unroll
                for (int i = 0; i < (kFrag ? 4 : 1); ++i) sa_now[i] = sa[i];
                const uint32_t srow_now = srow;
                auto read = [&](int o) { read_group(d + (o < 2 ? col0 : col2) + 32u * (o & 1), v[o & 1]); };
                auto add = [&](int o) {
                    if constexpr (kFrag)
                        add_fragments(acc[o], v[o & 1], sa_now, srow_now + 4u * ((o < 2 ? col0 : col2) + 32u * (o & 1)));
                    else
                        add_block(acc[o], v[o & 1], s[o]);
                };
                // the next 32 columns are on their way while these are added
                if (groups > 0) {
                    tmem_ld_wait(v[0]);
                    read(1);
                    add(0);
                    if (kMode == kGated || groups > 2) {
                        tmem_ld_wait(v[1]);
                        read(2);
                        add(1);
                        tmem_ld_wait(v[0]);
                        read(3);
                        add(2);
                    }
                    tmem_ld_wait(v[1]);
                }
                // every value of this buffer has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty_r0 + buf8);
                buf8 ^= 8u;
                if (buf8 == 0) bphase ^= 1u;
                const bool last = kb + 1 == num_kb;
                const bool slot_done = (kb & (kSlotBlocks - 1)) == kSlotBlocks - 1 || last;
                const uint32_t slot_bar = bar_sempty + 8 * slot;
                if (slot_done && ++slot == L::kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                if (!last && !open_block(slot_done)) {
                    failed = true;
                    break;
                }
                if (groups > 2) add(3);
                else if (kMode != kGated && groups > 0) add(1);
                if (slot_done) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(slot_bar);
                }
            }
            if (failed || groups == 0) continue;
            const int x0 = 32 * (g0 + first), y0 = m0 + 32 * quad;
            // lane = row writes its 64 (bf16) or 128 bytes (fp32) where the
            // TMA swizzle expects them; stores clip at N and M
            auto put_bf16 = [&](const CUtensorMap &map, int group, auto value) {
                const uint32_t box = obuf + static_cast<uint32_t>(onext) * 2048u;
                if (lane == 0) bulk_wait_read<3>();  // the store from this box four boxes ago
                __syncwarp();
                if constexpr (kFrag) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {   // sum i: see add_fragments
                        const int r = 16 * (i >> 3) + 8 * (i & 1) + (lane >> 2), j = (i >> 1) & 3;
                        sts_b32(box + r * 64 + ((j ^ ((r >> 1) & 3)) << 4) + 4 * (lane & 3), value(i));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        sts_v4(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4),
                               make_uint4(value(4 * c), value(4 * c + 1), value(4 * c + 2), value(4 * c + 3)));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&map, box, x0 + 32 * group, y0);
                    bulk_commit();
                }
                onext = (onext + 1) & 3;
            };
            if constexpr (kMode == kGated) {
                // (one copy of the code per activation: deciding inside, value
                // by value, cost the loop above its uniform registers)
                auto put_gated = [&](auto which) {
                    constexpr int kAct = decltype(which)::value;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (j < mine)
                            put_bf16(tm_y, j, [&](int i) {
                                return pack_bf16x2(
                                    act::gated<false>(kAct, out.alpha, lo2(acc[j][i]), lo2(acc[2 + j][i])),
                                    act::gated<false>(kAct, out.alpha, hi2(acc[j][i]), hi2(acc[2 + j][i])));
                            });
                };
                if (out.act == act::kSilu) put_gated(std::integral_constant<int, act::kSilu>());
                else put_gated(std::integral_constant<int, act::kGeluTanh>());
                if (out.g) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j < mine) {
                            put_bf16(tm_yg, j, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
                            put_bf16(tm_yu, j, [&](int i) { return pack_bf16x2(lo2(acc[2 + j][i]), hi2(acc[2 + j][i])); });
                        }
                    }
                }
            } else if (!out.f32) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < mine)
                        put_bf16(tm_y, j, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < mine) {
                        const uint32_t box = obuf + static_cast<uint32_t>(onext & 1) * 4096u;
                        if (lane == 0) bulk_wait_read<1>();  // the store from this box two boxes ago
                        __syncwarp();
                        if constexpr (kFrag) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int r = 16 * (i >> 3) + 8 * (i & 1) + (lane >> 2);
                                const int c = (i & 6) + ((lane >> 1) & 1);
                                sts_b64(box + r * 128 + ((c ^ (r & 7)) << 4) + 8 * (lane & 1), acc[j][i]);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const unsigned long long a0 = acc[j][2 * c], a1 = acc[j][2 * c + 1];
                                sts_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4),
                                       make_uint4(static_cast<uint32_t>(a0), static_cast<uint32_t>(a0 >> 32),
                                                  static_cast<uint32_t>(a1), static_cast<uint32_t>(a1 >> 32)));
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tm_y, box, x0 + 32 * j, y0);
                            bulk_commit();
                        }
                        onext = (onext + 1) & 3;
                    }
                }
            }
        }
        if (lane == 0) bulk_wait<0>();
    }

    if (failed) atomicOr(&g_gemm_b128_status, 1u);

    tc_fence_before();
    __syncthreads();
    // the pair's MMAs have completed (the issuer drained them) and both CTAs'
    // sums are stored before either frees TMEM or leaves
    cluster_sync_all();
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// Tiles of 256 rows over `pairs` pairs of SMs, their columns in groups of 32
// (a group has one tile scale, and the pair's MMA takes N in steps of 32) cut
// evenly into as many tiles as cost least: waves of tiles over the pairs, a
// tile its columns plus a constant (its rows of A whatever its width).
PairPlan make_pair_plan(int M, int N, int K, bool gated, bool row_scales, int pairs) {
    PairPlan p{};
    p.tiles_m = (M + 2 * kBM - 1) / (2 * kBM);
    p.groups = (N + 31) / 32;
    p.num_kb = (K + kBlockK - 1) / kBlockK;
    const int per_group = gated ? 64 : 32;
    const int max_groups = kPairBufCols / per_group;
    const int least = (p.groups + max_groups - 1) / max_groups;
    const int most = p.groups < least + pairs ? p.groups : least + pairs;
    long long best = -1;
    int widest = 0;
    for (int tn = least; tn <= most; ++tn) {
        const int cols = (p.groups + tn - 1) / tn * per_group;
        const long long waves = (static_cast<long long>(p.tiles_m) * tn + pairs - 1) / pairs;
        const long long cost = waves * (cols + 64);
        if (best < 0 || cost < best) {
            best = cost;
            p.tiles_n = tn;
            widest = cols;
        }
    }
    p.half_rows = widest / 2;
    p.s_cols = row_scales ? widest : 0;
    return p;
}

std::atomic<int> g_pair_clusters[3][32];   // per mode and device, 0: not asked yet

template <int kMode>
cudaError_t launch_pair(const void *A, const float *As, const void *B0, const float *Bs0,
                        const void *B1, const float *Bs1, const Out &out, int M, int N, int K,
                        const DeviceInfo &dev, cudaStream_t stream) {
    auto kernel = swiglu_gemm_b128_pair_kernel<kMode>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = PairLayout<kMode>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    int max_clusters = g_pair_clusters[kMode][dev.device & 31].load();
    if (max_clusters == 0) {
        e = prepare_kernel(kernel, PairLayout<kMode>::kSmem);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2);
        e = cudaOccupancyMaxActiveClusters(&max_clusters, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (max_clusters < 1) return cudaErrorInvalidConfiguration;
        g_pair_clusters[kMode][dev.device & 31].store(max_clusters);
    }
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    const PairPlan p = make_pair_plan(M, N, K, kMode == kGated, kMode == kRowScales, max_clusters);
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapDataType f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapSwizzle none = CU_TENSOR_MAP_SWIZZLE_NONE;
    const uint64_t k64 = static_cast<uint64_t>(K), n64 = static_cast<uint64_t>(N);
    const uint32_t half = static_cast<uint32_t>(p.half_rows);
    CUtensorMap ta, tas, tb, tu, tbs, ty, tyg, tyu;
    if (!encode_tmap_2d(&ta, A, u8, k64, M, k64, kBlockK, kBM, sw) ||
        !encode_tmap_2d(&tas, As, f32, M, p.num_kb, static_cast<uint64_t>((M + 3) / 4 * 4) * 4, 128,
                        kSlotBlocks, none) ||
        !encode_tmap_2d(&tb, B0, u8, k64, n64, k64, kBlockK, half, sw))
        return cudaErrorInvalidValue;
    tu = tb;
    tbs = tas;
    if (kMode == kGated && !encode_tmap_2d(&tu, B1, u8, k64, n64, k64, kBlockK, half, sw))
        return cudaErrorInvalidValue;
    if (kMode == kRowScales &&
        !encode_tmap_2d(&tbs, Bs0, f32, n64, p.num_kb, n64 * 4, static_cast<uint32_t>(p.s_cols),
                        kSlotBlocks, none))
        return cudaErrorInvalidValue;
    const bool ok = out.f32 ? encode_tmap_2d(&ty, out.y, f32, n64, M, n64 * 4, 32, 32, sw)
                            : encode_tmap_2d(&ty, out.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n64, M, n64 * 2, 32,
                                             32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return cudaErrorInvalidValue;
    tyg = tyu = ty;
    if (out.g && (!encode_tmap_2d(&tyg, out.g, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n64, M, n64 * 2, 32, 32,
                                  CU_TENSOR_MAP_SWIZZLE_64B) ||
                  !encode_tmap_2d(&tyu, out.u, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n64, M, n64 * 2, 32, 32,
                                  CU_TENSOR_MAP_SWIZZLE_64B)))
        return cudaErrorInvalidValue;
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    const long long pairs = tiles < max_clusters ? tiles : max_clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    e = cudaLaunchKernelEx(&cfg, kernel, ta, tas, tb, tu, tbs, ty, tyg, tyu, Bs0, Bs1, out, M, N, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_b128(const void *A, const float *As, const void *B, const float *Bs,
                             void *Y, int M, int N, int K, bool row_scales, int f32_out,
                             const DeviceInfo &dev, cudaStream_t stream) {
    if (b128_few_rows(M, K))
        return launch_gemm_b128_stream(A, As, B, Bs, Y, M, N, K, row_scales, f32_out, dev, stream);
    Out out{};
    out.y = Y;
    out.f32 = f32_out;
    return row_scales ? launch_pair<kRowScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream)
                      : launch_pair<kTileScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream);
}

cudaError_t launch_fwd_b128(const void *X, const float *Xs, const void *Wg, const float *Gs,
                            const void *Wu, const float *Us, void *H, int M, int N, int K,
                            const Epilogue &epi, const DeviceInfo &dev, cudaStream_t stream) {
    if (b128_few_rows(M, K))
        return launch_fwd_b128_stream(X, Xs, Wg, Gs, Wu, Us, H, M, N, K, epi, dev, stream);
    Out out{};
    out.y = H;
    out.g = static_cast<__nv_bfloat16 *>(epi.G);
    out.u = static_cast<__nv_bfloat16 *>(epi.U);
    out.act = epi.activation;
    out.alpha = epi.gate_multiplier;
    return launch_pair<kGated>(X, Xs, Wg, Gs, Wu, Us, out, M, N, K, dev, stream);
}

cudaError_t gemm_b128_status_fetch_and_clear(unsigned int *host_out, cudaStream_t stream) {
    return fetch_and_clear(g_gemm_b128_status, host_out, stream);
}

}  // namespace swiglu
