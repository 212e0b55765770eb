// gemm_b128_stream.cu -- the block-scaled e4m3 products (gemm_b128.cu) for
// M <= 64 rows of A (b128_few_rows): a read of the weights from HBM once, on the fp8 tensor
// cores.
//
// The operands are swapped against the large products: the weights are the
// MMA's M operand (up to 128 of their rows per MMA, the gated form half of
// them rows of Wg and half of Wu), the few rows of A its N operand.  An MMA
// reads its whole M operand from shared memory and takes some 70 cycles
// however few columns it has: here those reads are the weights themselves, four
// MMAs (K = 32) per block whatever M is, and lane n of the accumulator holds
// output column n for all rows of A.  (B200, M = 8, N = 4096, K = 14336, 58.7 MB
// of weights: A as the M operand 29.8 us; warp-level mma.sync, which unpacks
// e4m3 to fp16 first, 22.3 us; this form 16.9 us, of 13 us that the copies alone
// take.)
//
// A tile is R rows of weights (a multiple of 8, at most 256: two MMAs per
// step), spread evenly over the SMs; where that would leave few rows per SM,
// the blocks of the reduction are split over a cluster of 2, 4 or 8 CTAs and
// their sums meet in the leader's shared memory, added in a fixed order.
//
// As in gemm_b128.cu a block's MMAs fill columns of TMEM of their own, which
// eight warps read back, scale and add to sums in registers.  Copies take
// `kbs` blocks at once -- a 3-D box [block][row][128] (gated, 4-D: [block]
// [matrix][row][128], where the two weights' distance allows it) lands as one
// 128-byte-swizzled operand tile per block --, barriers go by stages and by
// groups of `g` blocks, as many as half of TMEM holds.
//
// A last block shorter than 128 is a step of its own: the views of whole
// blocks end before it, a 2-D one fills it up with zeros.
//
//  * warps 0..7 accumulate: rows 32 (w mod 4) .. +31 of each 128; the two
//    warps of a row take every other block (M <= 32) or half of A's rows;
//  * warps 8 and 10 (one thread each) copy the weights and A, warp 11 the
//    scales; warp 9 (one thread) issues the MMAs.
// Waits are bounded; a stuck pipeline sets the status word, the MMAs and
// copies in flight are drained and TMEM is freed before the kernel returns.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "b128.cuh"
#include "kernels.cuh"
#include "status.cuh"
#include "tmap.cuh"

namespace swiglu {

// Status word of this translation unit's kernel (bit 0 = a wait gave up).
__device__ unsigned int g_gemm_b128_stream_status;

namespace {

using namespace b128;

constexpr int kMaxStages = 8;
constexpr int kMaxSlots = kMaxStages + 2;
constexpr uint32_t kBufCols = kTmemCols / 2;
constexpr uint32_t kNumBars = 2 * kMaxStages + 2 * kMaxSlots + 2 * 2 + 1;
constexpr uint32_t kTailBytes = 8 * kNumBars + 32 + 1024;  // + TMEM slot, abort flag, alignment
constexpr int kMaxCluster = 8;

struct StreamPlan {
    int units, tiles;  // units of 8 output columns, cut into tiles of q or q + 1
    int q;
    int cluster;       // CTAs that share a tile's reduction
    int rows;          // weight rows of the widest tile (gated: of both)
    int mma_m;         // rows per MMA: 64 where a tile has no more, else 128
    int nrt;           // MMAs per step: groups of mma_m rows of them
    int a_rows;        // rows of an A box
    int mma_n;
    int tok;           // rows of A per accumulating warp: 8 or 32
    int parity;        // the two warps of a row take every other block
    int kbs, g;        // blocks per stage, per TMEM buffer
    int acc_cols;      // TMEM columns of a block and group of 128 rows
    int full;          // whole blocks of K
    int stages, slots;
    int part_m;        // rows of A in the exchange of sums
    uint32_t stage_bytes, slot_bytes, slot_b;
    uint32_t off_slots, off_bar, smem;
};

// w3 (gated: the 4-D view of both weights): whole blocks, boxes of kbs blocks;
// w2, u2: rows of 128 bytes of either weight, for the short last block.  _lo: boxes of 8 q rows, _hi: 8 (q + 1).
struct StreamMaps {
    CUtensorMap a3, a2, as, bs, w3_lo, w3_hi, w2_lo, w2_hi, u2_lo, u2_hi;
};

template <int kMode, int kTok>
__global__ void __launch_bounds__(kThreads, 1)
    swiglu_gemm_b128_stream_kernel(const __grid_constant__ StreamMaps maps,
                                   const float *bs0, const float *bs1,
                                   const Out out, int M, int N, int num_kb, int joined, int swapped,
                                   const StreamPlan p) {
    constexpr int kRt = 2;   // groups of 128 rows a warp can hold
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar_full = base + p.off_bar;
    const uint32_t bar_empty = bar_full + 8 * kMaxStages;
    const uint32_t bar_sfull = bar_empty + 8 * kMaxStages;
    const uint32_t bar_sempty = bar_sfull + 8 * kMaxSlots;
    const uint32_t bar_tfull = bar_sempty + 8 * kMaxSlots;
    const uint32_t bar_tempty = bar_tfull + 16;
    const uint32_t bar_drain = bar_tempty + 16;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(gbase + p.off_bar + 8 * kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + p.off_bar + 8 * kNumBars + 16);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (known uniform)
    const int lane = threadIdx.x % 32;
    const int rank = p.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;

    auto tile_of = [&](int t, int &u0, int &cnt) {
        u0 = static_cast<int>(static_cast<long long>(p.units) * t / p.tiles);
        cnt = static_cast<int>(static_cast<long long>(p.units) * (t + 1) / p.tiles) - u0;
    };
    // this CTA's blocks, in steps of kbs whole ones; a short last block is a
    // step of its own
    const int kb_begin = static_cast<int>(static_cast<long long>(num_kb) * rank / p.cluster);
    const int kb_end = static_cast<int>(static_cast<long long>(num_kb) * (rank + 1) / p.cluster);
    auto step_of = [&](int kb, int &nb) {  // blocks of the step that begins with kb
        nb = kb < p.full ? min(p.kbs, min(kb_end, p.full) - kb) : 1;
        return kb < p.full;
    };
    const int first_tile = static_cast<int>(blockIdx.x) / p.cluster;
    const int tile_step = static_cast<int>(gridDim.x) / p.cluster;
    constexpr int kSides = kMode == kGated ? 2 : 1;

    // One step's weights (and the bytes of the step's A) into a stage.
    auto copy_weights = [&](int kb, int u0, int cnt, int at_stage) {
        int nb;
        const bool whole = step_of(kb, nb);
        const bool hi = cnt > p.q;
        const int R = kSides * 8 * cnt;
        const uint32_t fb = bar_full + 8 * at_stage;
        const uint32_t st = base + at_stage * p.stage_bytes;
        // (a box always holds kbs blocks: what lies past the view arrives as
        // zeros, what the next CTA's is not multiplied)
        const uint32_t boxes = whole ? static_cast<uint32_t>(p.kbs) : 1u;
        mbar_arrive_expect_tx(fb, boxes * 128u * static_cast<uint32_t>(R + p.a_rows));
        if (whole && joined) {
            tma_load_4d(hi ? &maps.w3_hi : &maps.w3_lo, fb, st, 0, 8 * u0, 0, kb);
        } else if (whole && kMode != kGated) {
            tma_load_3d(hi ? &maps.w3_hi : &maps.w3_lo, fb, st, 0, 8 * u0, kb);
        } else {
            // block by block: a short one, or two weights that no view joins
            // (their rows side by side)
            for (uint32_t b = 0; b < boxes; ++b) {
                const uint32_t dst = st + b * static_cast<uint32_t>(R) * 128u;
                const int x = (kb + static_cast<int>(b)) * kBlockK;
                tma_load_2d(hi ? &maps.w2_hi : &maps.w2_lo, fb, dst, x, 8 * u0);
                if (kMode == kGated)
                    tma_load_2d(hi ? &maps.u2_hi : &maps.u2_lo, fb, dst + static_cast<uint32_t>(8 * cnt) * 128u, x,
                                8 * u0);
            }
        }
    };

    // Setup runs while the kernel before this one ends (programmatic dependent
    // launch); nothing is read or written before it has.  The weights' thread
    // fills the ring before the rest of the CTA is ready.
    griddep_launch_dependents();
    int ahead = 0;   // steps of the first tile copied here
    if (warp == kEpiWarps && lane == 0) {
        tma_prefetch_desc(&maps.w3_lo);
        tma_prefetch_desc(&maps.w3_hi);
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        fence_mbar_init();
        griddep_wait();
        int u0, cnt, nb;
        tile_of(first_tile, u0, cnt);
        for (int kb = kb_begin; kb < kb_end && ahead < p.stages; kb += nb) {
            step_of(kb, nb);
            copy_weights(kb, u0, cnt, ahead);
            ++ahead;
        }
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.a3);
        tma_prefetch_desc(&maps.as);
        for (int s = 0; s < p.slots; ++s) {
            mbar_init(bar_sfull + 8 * s, 1);
            mbar_init(bar_sempty + 8 * s, kEpiWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, kEpiWarps);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == kEpiWarps + 1) {
        tmem_alloc(smem_u32(tmem_ptr), kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_ptr);

    bool failed = false;
    // state of the roles across tiles
    int stage = 0, slot = 0, buf = 0;
    uint32_t phase = 0, sphase = 0, bphase = 0;
    long long issued = 0;

    for (int t = first_tile; t < p.tiles; t += tile_step) {
        int u0, cnt;
        tile_of(t, u0, cnt);
        const int side = 8 * cnt;            // rows of one weight
        const int R = kSides * side;
        unsigned long long acc[kRt][kTok / 2];
        if (warp >= kEpiWarps) {
            if ((warp == kEpiWarps || warp == kEpiWarps + 2) && lane == 0) {
                // ------------ TMA producers: weights (and the bytes of both), A
                const bool is_w = warp == kEpiWarps;
                int nb, done = 0;
                for (int kb = kb_begin; kb < kb_end && !failed; kb += nb, ++done) {
                    const bool whole = step_of(kb, nb);
                    if (is_w && t == first_tile && done < ahead) {
                        // copied above
                    } else if (!mbar_wait_long(bar_empty + 8 * stage, phase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    } else if (is_w) {
                        copy_weights(kb, u0, cnt, stage);
                    } else {
                        const uint32_t xst =
                            base + stage * p.stage_bytes + static_cast<uint32_t>(p.kbs * p.rows) * 128u;
                        if (whole) tma_load_3d(&maps.a3, bar_full + 8 * stage, xst, 0, 0, kb);
                        else tma_load_2d(&maps.a2, bar_full + 8 * stage, xst, kb * kBlockK, 0);
                    }
                    ++issued;
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (warp == kEpiWarps + 3) {
                // -------------------------------------------------- scales
                // slot: A's [kbs][a_rows], then the weights' [kbs][side] (row
                // scales), or of each block four tile scales: plain, of column
                // blocks b0 .. b0 + 3 (the last one repeated), gated, of b0,
                // b0 + 1 of Wg and of Wu.  (Rows past the last block: zeros.)
                const float *src = nullptr;
                if (kMode != kRowScales) {
                    const int i = kMode == kGated ? (lane & 1) : (lane & 3);
                    const float *table = (kMode == kGated && (lane & 2)) ? bs1 : bs0;
                    src = table + static_cast<int64_t>(min(u0 / 16 + i, (N + 127) / 128 - 1)) * num_kb;
                }
                int nb;
                for (int kb = kb_begin; kb < kb_end && !failed; kb += nb) {
                    step_of(kb, nb);
                    float v = 0.0f;
                    if (kMode != kRowScales && lane < 4 * p.kbs) v = ld_plain(src + min(kb + lane / 4, num_kb - 1));
                    if (!mbar_wait_long(bar_sempty + 8 * slot, sphase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    }
                    const uint32_t sb = bar_sfull + 8 * slot;
                    const uint32_t dst = base + p.off_slots + slot * p.slot_bytes;
                    if (kMode != kRowScales) {
                        if (lane < 4 * p.kbs) sts_f32(dst + p.slot_b + 4u * lane, v);
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const uint32_t rows = static_cast<uint32_t>(p.a_rows + (kMode == kRowScales ? p.rows : 0));
                        mbar_arrive_expect_tx(sb, static_cast<uint32_t>(p.kbs) * 4u * rows);
                        tma_load_2d(&maps.as, sb, dst, 0, kb);
                        if (kMode == kRowScales) tma_load_2d(&maps.bs, sb, dst + p.slot_b, 8 * u0, kb);
                    }
                    ++issued;
                    if (++slot == p.slots) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (warp == kEpiWarps + 1) {
                // -------------------------------------- MMA issuer (whole warp)
                // (rows beyond the tile's are whatever lies behind it in shared
                // memory: lanes never read)
                const uint32_t idesc = make_idesc(0u, static_cast<uint32_t>(p.mma_m), static_cast<uint32_t>(p.mma_n));
                const int nrt = (R + p.mma_m - 1) / p.mma_m;
                int nb;
                for (int kb = kb_begin; kb < kb_end && !failed; kb += nb) {
                    step_of(kb, nb);
                    if (!mbar_wait_long(bar_full + 8 * stage, phase, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = base + stage * p.stage_bytes;
                    const uint32_t xst = st + static_cast<uint32_t>(p.kbs * p.rows) * 128u;
                    for (int b0 = 0; b0 < nb; b0 += p.g) {
                        if (!mbar_wait_long(bar_tempty + 8 * buf, bphase ^ 1u, abort_flag)) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        const int b1 = min(nb, b0 + p.g);
                        uint32_t d = tmem_base + static_cast<uint32_t>(buf) * kBufCols;
                        uint64_t xd = sw128_kmajor_desc(xst + static_cast<uint32_t>(b0 * p.a_rows) * 128u);
                        uint64_t wd = sw128_kmajor_desc(st + static_cast<uint32_t>(b0 * R) * 128u);
                        for (int b = b0; b < b1; ++b) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) mma_f8(d, wd + 2u * kk, xd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                            d += static_cast<uint32_t>(p.acc_cols);
                            if (nrt > 1) {  // rows 128 .. of the tile, 16 KB further on
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    mma_f8(d, wd + 1024u + 2u * kk, xd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                            }
                            if (p.nrt > 1) d += static_cast<uint32_t>(p.acc_cols);
                            xd += static_cast<uint32_t>(p.a_rows) * 8u;  // (addresses count 16 bytes)
                            wd += static_cast<uint32_t>(R) * 8u;
                        }
                        commit_elect(bar_tfull + 8 * buf);
                        if (++buf == 2) {
                            buf = 0;
                            bphase ^= 1u;
                        }
                    }
                    if (failed) break;
                    commit_elect(bar_empty + 8 * stage);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else {
            // ------------------------------------------------ accumulation
            const int quad = warp & 3, half = warp >> 2;
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
            const int tok0 = p.parity ? 0 : kTok * half;    // first row of A
            // (an M = 64 MMA leaves row 16 q + l in lane l < 16 of quadrant q)
            const int per_quad = p.mma_m / 4;
            const bool work = tok0 < M;
            const int nrt = min(kRt, (R + p.mma_m - 1) / p.mma_m);
            // byte offset of a lane's weight scale within a block's
            uint32_t at[kRt];
#pragma unroll
            for (int rt = 0; rt < kRt; ++rt) {
                const int r = min(rt * 128 + quad * per_quad + lane, R - 1);
                const int r1 = r < side ? r : r - side;     // (gated: of Wu)
                at[rt] = kMode == kRowScales
                             ? 4u * static_cast<uint32_t>(r)
                             : 4u * static_cast<uint32_t>((8 * u0 + r1) / 128 - u0 / 16 + (r < side ? 0 : 2));
            }
            const uint32_t b_step = kMode == kRowScales ? 4u * static_cast<uint32_t>(p.rows) : 16u;
#pragma unroll
            for (int rt = 0; rt < kRt; ++rt)
#pragma unroll
                for (int i = 0; i < kTok / 2; ++i) acc[rt][i] = 0ull;
            int nb;
            for (int kb = kb_begin; kb < kb_end && !failed; kb += nb) {
                step_of(kb, nb);
                if (!mbar_wait_long(bar_sfull + 8 * slot, sphase, abort_flag)) {
                    failed = true;
                    break;
                }
                const uint32_t sa_src = base + p.off_slots + slot * p.slot_bytes;
                const uint32_t sb_src = sa_src + p.slot_b;
                for (int b0 = 0; b0 < nb; b0 += p.g) {
                    if (!mbar_wait_long(bar_tfull + 8 * buf, bphase, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const int b1 = work ? min(nb, b0 + p.g) : 0;
                    // kBatch blocks' reads are in flight together
                    constexpr int kBatch = kTok == 8 ? 4 : 2;
                    const int next = p.parity ? 2 : 1;
                    for (int b = b0 + (p.parity ? half : 0); b < b1; b += kBatch * next) {
#pragma unroll
                        for (int rt = 0; rt < kRt; ++rt) {
                            if (rt < nrt) {
                                uint32_t v[kBatch][kTok];
                                float f[kBatch];
#pragma unroll
                                for (int q = 0; q < kBatch; ++q) {
                                    const int bq = b + q * next;
                                    if (q > 0 && bq >= b1) continue;
                                    const uint32_t d = lanes + static_cast<uint32_t>(buf) * kBufCols +
                                                       static_cast<uint32_t>(((bq - b0) * p.nrt + rt) * p.acc_cols + tok0);
                                    if constexpr (kTok == 8) {
                                        tmem_ld_32x32b_x8(d, v[q]);
                                    } else {
                                        tmem_ld_32x32b_x32(d, v[q]);
                                    }
                                    f[q] = lds_f32(sb_src + static_cast<uint32_t>(bq) * b_step + at[rt]);
                                }
#pragma unroll
                                for (int q = 0; q < kBatch; ++q) {
                                    const int bq = b + q * next;
                                    if (q > 0 && bq >= b1) continue;
                                    const uint32_t sa = sa_src + 4u * static_cast<uint32_t>(bq * p.a_rows + tok0);
                                    if constexpr (kTok == 8) {
                                        tmem_ld_wait8(v[q]);
                                        const uint4 w0 = lds_v4(sa), w1 = lds_v4(sa + 16u);
                                        const unsigned long long s2 = pair2(f[q], f[q]);
                                        fma2(acc[rt][0], v[q][0], v[q][1], mul2(pair2(__uint_as_float(w0.x), __uint_as_float(w0.y)), s2));
                                        fma2(acc[rt][1], v[q][2], v[q][3], mul2(pair2(__uint_as_float(w0.z), __uint_as_float(w0.w)), s2));
                                        fma2(acc[rt][2], v[q][4], v[q][5], mul2(pair2(__uint_as_float(w1.x), __uint_as_float(w1.y)), s2));
                                        fma2(acc[rt][3], v[q][6], v[q][7], mul2(pair2(__uint_as_float(w1.z), __uint_as_float(w1.w)), s2));
                                    } else {
                                        tmem_ld_wait(v[q]);
                                        add_rows(acc[rt], v[q], f[q], sa);
                                    }
                                }
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_tempty + 8 * buf);
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
                if (lane == 0) mbar_arrive(bar_sempty + 8 * slot);  // (read before the last __syncwarp)
                if (++slot == p.slots) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
        }
        __syncwarp();

        // ---------------------------------------------------- sum and store
        // Every CTA of the cluster has multiplied all it copied: the leader's
        // stages take the sums [slice][row of A][weight row], a slice per CTA
        // and (parity) warp of a row.
        const int slices = p.cluster * (p.parity ? 2 : 1);
        if (p.cluster > 1) cluster_sync_all();
        else __syncthreads();
        if (warp < kEpiWarps) {
            const int quad = warp & 3, half = warp >> 2;
            const int tok0 = p.parity ? 0 : kTok * half;
            const int slice = p.parity ? 2 * rank + half : rank;
            const int per_quad = p.mma_m / 4;
            const int row = quad * per_quad + lane;
            const uint32_t to = map_to_rank(base, 0) +
                                4u * static_cast<uint32_t>((slice * p.part_m + tok0) * p.rows + row);
#pragma unroll
            for (int rt = 0; rt < kRt; ++rt) {
                if (lane < per_quad && rt * 128 + row < R) {
#pragma unroll
                    for (int i = 0; i < kTok; ++i) {
                        if (tok0 + i < M) {
                            const float v = (i & 1) ? hi2(acc[rt][i / 2]) : lo2(acc[rt][i / 2]);
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                                             to + 4u * static_cast<uint32_t>(i * p.rows + rt * 128)),
                                         "f"(v)
                                         : "memory");
                        }
                    }
                }
            }
        }
        if (p.cluster > 1) cluster_sync_all();
        else __syncthreads();
        if (rank == 0 && !*abort_flag) {
            const float *part = reinterpret_cast<const float *>(gbase);
            const int plane = p.part_m * p.rows;
            auto total = [&](int m, int r) {
                float v = part[m * p.rows + r];
                for (int s = 1; s < slices; ++s) v += part[s * plane + m * p.rows + r];
                return v;
            };
            for (int i = threadIdx.x; i < M * side; i += kThreads) {
                const int m = i / side, r = i - m * side;
                const int64_t o = static_cast<int64_t>(m) * N + 8 * u0 + r;
                const float v = total(m, r);
                if constexpr (kMode == kGated) {
                    // (the view that joins the weights starts with the one at
                    // the lower address)
                    const float w = total(m, side + r);
                    const float g = joined && swapped ? w : v, u = joined && swapped ? v : w;
                    static_cast<__nv_bfloat16 *>(out.y)[o] =
                        __float2bfloat16_rn(act::gated<false>(out.act, out.alpha, g, u));
                    if (out.g) {
                        out.g[o] = __float2bfloat16_rn(g);
                        out.u[o] = __float2bfloat16_rn(u);
                    }
                } else if (out.f32) {
                    static_cast<float *>(out.y)[o] = v;
                } else {
                    static_cast<__nv_bfloat16 *>(out.y)[o] = __float2bfloat16_rn(v);
                }
            }
        }
        if (t + tile_step < p.tiles) {  // the stages are free for the next tile's copies
            fence_proxy_async_smem();
            if (p.cluster > 1) cluster_sync_all();
            else __syncthreads();
        }
    }

    // Never leave while a load issued here may still write shared memory, or
    // an MMA may still run.
    if ((warp == kEpiWarps || warp == kEpiWarps + 2) && lane == 0) {
        for (int s = 0; s < p.stages; ++s)
            if (issued > s)
                mbar_wait_drain(bar_full + 8 * s, static_cast<uint32_t>(((issued - 1 - s) / p.stages) & 1));
    }
    if (warp == kEpiWarps + 3) {
        for (int s = 0; s < p.slots; ++s)
            if (issued > s)
                mbar_wait_drain(bar_sfull + 8 * s, static_cast<uint32_t>(((issued - 1 - s) / p.slots) & 1));
    }
    if (warp == kEpiWarps + 1) {
        commit_elect(bar_drain);
        mbar_wait_drain(bar_drain, 0);
    }
    if (failed) atomicOr(&g_gemm_b128_stream_status, 1u);

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (p.cluster > 1) cluster_sync_all();  // no CTA leaves before its sums have been read
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// Tile height, cluster and ring for `max_clusters[i]` resident clusters of
// 2^i CTAs.  A CTA's time per block is the larger of its weights' share of the
// HBM bandwidth (about 24 bytes per cycle and SM of the device on a B200, at
// most 48 for one SM) and of its MMAs and
// their accumulation (measured: 250 cycles for up to 8 rows of A, 340 up to
// 32, 520 up to 64, per 128 rows of weights), plus some of the smaller, as they
// do not overlap fully; a cluster costs two barriers and the exchange.  The
// cheapest (cluster, tiles) wins.  B200, clusters of 1, 2, 4, us: M = 8, 4096 x
// 14336 25.2, 17.7, 16.8; 512 x 4096 10.6, 8.9, 7.8; 1024 x 1024 6.5, 7.2, 6.9;
// 11008 x 14336 31.8, 35.0, 44.5.
StreamPlan make_stream_plan(int M, int N, int K, bool gated, bool row_scales, const int max_clusters[4]) {
    StreamPlan best{};
    long long best_cost = -1;
    const int num_kb = (K + kBlockK - 1) / kBlockK;
    const int sides = gated ? 2 : 1;
    for (int ci = 0; ci < 4; ++ci) {
        const int c = 1 << ci;
        if (max_clusters[ci] < 1 || c > num_kb) continue;
        StreamPlan p{};
        p.units = N / 8;
        p.cluster = c;
        p.full = K / kBlockK;
        p.a_rows = (M + 7) / 8 * 8;
        p.mma_n = (M + 15) / 16 * 16;
        p.tok = M <= 8 ? 8 : 32;
        p.parity = M <= 32 ? 1 : 0;
        p.part_m = p.parity ? p.a_rows : 2 * p.tok;
        const int max_units = 256 / (8 * sides);
        const int least = (p.units + max_units - 1) / max_units;
        p.tiles = p.units < max_clusters[ci] ? p.units : max_clusters[ci];
        if (p.tiles < least) p.tiles = least;
        p.q = p.units / p.tiles;
        const int cnt = (p.units + p.tiles - 1) / p.tiles;
        p.rows = 8 * sides * cnt;
        p.mma_m = p.rows <= 64 ? 64 : 128;
        p.nrt = (p.rows + p.mma_m - 1) / p.mma_m;
        p.acc_cols = p.tok == 8 ? 16 : (M <= 32 ? 32 : 64);
        p.g = 8;
        while (p.g > 1 && p.g * p.nrt * p.acc_cols > static_cast<int>(kBufCols)) p.g /= 2;
        const uint32_t exchange = 4u * static_cast<uint32_t>(c * (p.parity ? 2 : 1) * p.part_m * p.rows);
        const uint32_t slack = 16u * 1024u;  // the MMA's rows beyond the last tile of a stage
        const int per_cta = (num_kb + c - 1) / c;
        for (int want = 3; want >= 2 && p.stages == 0; --want) {
            for (int kbs = 8; kbs >= 1; kbs /= 2) {
                // (no more than an eighth of the copies past the CTA's blocks)
                if (kbs > 1 && ((per_cta + kbs - 1) / kbs * kbs - per_cta) * 8 > per_cta) continue;
                p.kbs = kbs;
                p.stage_bytes = static_cast<uint32_t>(kbs * (p.rows + p.a_rows)) * 128u;
                p.slot_b = (static_cast<uint32_t>(kbs * p.a_rows) * 4u + 128u + 127u) / 128u * 128u;
                p.slot_bytes = p.slot_b + (row_scales ? (static_cast<uint32_t>(kbs * p.rows) * 4u + 127u) / 128u * 128u : 128u);
                const uint32_t fixed = slack + kTailBytes;
                int stages = kMaxStages;
                while (stages > 0 && fixed + stages * p.stage_bytes + (stages + 2) * p.slot_bytes > kMaxSmem) --stages;
                if (stages >= want && stages * p.stage_bytes + slack >= exchange) {
                    p.stages = stages;
                    break;
                }
            }
        }
        if (p.stages == 0) continue;
        if (p.g > p.kbs) p.g = p.kbs;
        p.slots = p.stages + 2;
        p.off_slots = p.stages * p.stage_bytes + slack;
        p.off_bar = p.off_slots + p.slots * p.slot_bytes;
        p.smem = p.off_bar + kTailBytes;
        const long long waves = (p.tiles + max_clusters[ci] - 1) / max_clusters[ci];
        const long long busy = static_cast<long long>(p.tiles < max_clusters[ci] ? p.tiles : max_clusters[ci]) * c;
        const long long share = p.rows * 128 * busy / (24 * max_clusters[0]), alone = p.rows * 128 / 48;
        const long long bytes = share > alone ? share : alone;
        const long long work = p.nrt * (p.tok == 8 ? 250ll : (p.parity ? 340ll : 520ll));
        const long long more = bytes > work ? bytes : work, less = bytes + work - more;
        const long long cost = waves * (per_cta * (more + less * (p.nrt == 1 ? 5 : 8) / 20) +
                                        (c > 1 ? 1200 + c * (150 + 8 * p.a_rows) : 0));
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = p;
        }
    }
    return best;
}

struct DeviceState {
    bool ready = false;
    int max_clusters[4] = {};
};

std::mutex g_state_mutex;
DeviceState g_state[3][2][64];   // mode, tok, device

template <int kMode, int kTok>
cudaError_t device_state(const DeviceInfo &dev, int slot, DeviceState &out) {
    std::lock_guard<std::mutex> lock(g_state_mutex);
    DeviceState &s = g_state[kMode][slot][dev.device & 63];
    if (!s.ready) {
        auto kernel = swiglu_gemm_b128_stream_kernel<kMode, kTok>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMaxSmem));
        if (e != cudaSuccess) return e;
        s.max_clusters[0] = dev.sm_count;
        for (int ci = 1; ci < 4; ++ci) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << ci);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kMaxSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << ci;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&s.max_clusters[ci], kernel, &cfg);
            if (e != cudaSuccess) return e;
        }
        s.ready = true;
    }
    out = s;
    return cudaSuccess;
}

template <int kMode, int kTok>
cudaError_t launch_stream(const void *A, const float *As, const void *B0, const float *Bs0,
                          const void *B1, const float *Bs1, const Out &out, int M, int N, int K,
                          const DeviceInfo &dev, cudaStream_t stream) {
    DeviceState state;
    cudaError_t e = device_state<kMode, kTok>(dev, kTok == 8 ? 0 : 1, state);
    if (e != cudaSuccess) return e;
    const StreamPlan p = make_stream_plan(M, N, K, kMode == kGated, kMode == kRowScales, state.max_clusters);
    if (p.stages < 2 || p.smem > kMaxSmem) return cudaErrorInvalidValue;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapDataType f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapSwizzle none = CU_TENSOR_MAP_SWIZZLE_NONE;
    const uint64_t k64 = static_cast<uint64_t>(K), full = static_cast<uint64_t>(p.full);
    const uint64_t n64 = static_cast<uint64_t>(N);
    const uint32_t lo = 8u * p.q;
    const uint32_t hi = p.units % p.tiles ? lo + 8u : lo;  // (no tile holds more: same box)
    const uint32_t arows = static_cast<uint32_t>(p.a_rows), kbs = static_cast<uint32_t>(p.kbs);
    const int num_kb = (K + kBlockK - 1) / kBlockK;
    const bool tail = num_kb > p.full;
    StreamMaps m;
    if (p.full > 0 && !encode_tmap_3d(&m.a3, A, u8, 128, static_cast<uint64_t>(M), full, k64, 128, 128, arows, kbs, sw))
        return cudaErrorInvalidValue;
    if ((tail || p.full == 0) &&
        !encode_tmap_2d(&m.a2, A, u8, k64, static_cast<uint64_t>(M), k64, kBlockK, arows, sw))
        return cudaErrorInvalidValue;
    if (p.full == 0) m.a3 = m.a2;
    if (!tail) m.a2 = m.a3;
    // gated: one view of both weights, from the lower address
    int joined = 0, swapped = 0;
    if (kMode == kGated && p.full > 0) {
        const uintptr_t pg = reinterpret_cast<uintptr_t>(B0), pu = reinterpret_cast<uintptr_t>(B1);
        swapped = pu < pg ? 1 : 0;
        const uint64_t dist = swapped ? pg - pu : pu - pg;
        if (dist != 0 && dist % 16 == 0 && dist < (1ull << 40)) {
            const uint64_t dims[4] = {128, n64, 2, full};
            const uint64_t strides[3] = {k64, dist, 128};
            const uint32_t box_lo[4] = {128, lo, 2, kbs}, box_hi[4] = {128, hi, 2, kbs};
            const void *w0 = swapped ? B1 : B0;
            joined = encode_tmap_4d(&m.w3_lo, w0, u8, dims, strides, box_lo, sw);
            m.w3_hi = m.w3_lo;
            if (joined && hi != lo) joined = encode_tmap_4d(&m.w3_hi, w0, u8, dims, strides, box_hi, sw);
        }
        if (!joined) swapped = 0;
    }
    // (joined, the sides of a tile are in address order: so are its short last
    // block's copies and its scales)
    const void *s0 = swapped ? B1 : B0, *s1 = swapped ? B0 : B1;
    const float *t0 = swapped ? Bs1 : Bs0, *t1 = swapped ? Bs0 : Bs1;
    if (kMode != kGated && p.full > 0) {
        if (!encode_tmap_3d(&m.w3_lo, s0, u8, 128, n64, full, k64, 128, 128, lo, kbs, sw)) return cudaErrorInvalidValue;
        m.w3_hi = m.w3_lo;
        if (hi != lo && !encode_tmap_3d(&m.w3_hi, s0, u8, 128, n64, full, k64, 128, 128, hi, kbs, sw))
            return cudaErrorInvalidValue;
    }
    const bool by_block = tail || p.full == 0 || (kMode == kGated && !joined);
    if (by_block) {
        if (!encode_tmap_2d(&m.w2_lo, s0, u8, k64, n64, k64, kBlockK, lo, sw)) return cudaErrorInvalidValue;
        m.w2_hi = m.w2_lo;
        if (hi != lo && !encode_tmap_2d(&m.w2_hi, s0, u8, k64, n64, k64, kBlockK, hi, sw)) return cudaErrorInvalidValue;
        if (kMode == kGated) {
            if (!encode_tmap_2d(&m.u2_lo, s1, u8, k64, n64, k64, kBlockK, lo, sw)) return cudaErrorInvalidValue;
            m.u2_hi = m.u2_lo;
            if (hi != lo && !encode_tmap_2d(&m.u2_hi, s1, u8, k64, n64, k64, kBlockK, hi, sw))
                return cudaErrorInvalidValue;
        }
        if (!joined && (kMode == kGated || p.full == 0)) m.w3_lo = m.w3_hi = m.w2_lo;
    } else {
        m.w2_lo = m.w2_hi = m.w3_lo;
    }
    if (!(by_block && kMode == kGated)) m.u2_lo = m.u2_hi = m.w2_lo;
    if (!encode_tmap_2d(&m.as, As, f32, static_cast<uint64_t>(M), static_cast<uint64_t>(num_kb),
                        static_cast<uint64_t>((M + 3) / 4 * 4) * 4, arows, kbs, none))
        return cudaErrorInvalidValue;
    m.bs = m.as;
    if (kMode == kRowScales &&
        !encode_tmap_2d(&m.bs, Bs0, f32, n64, static_cast<uint64_t>(num_kb), n64 * 4,
                        static_cast<uint32_t>(p.rows), kbs, none))
        return cudaErrorInvalidValue;
    const int ci = p.cluster == 1 ? 0 : (p.cluster == 2 ? 1 : (p.cluster == 4 ? 2 : 3));
    const int clusters = p.tiles < state.max_clusters[ci] ? p.tiles : state.max_clusters[ci];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, swiglu_gemm_b128_stream_kernel<kMode, kTok>, m, t0, t1, out, M, N, num_kb, joined,
                           swapped, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int kMode>
cudaError_t launch_tok(const void *A, const float *As, const void *B0, const float *Bs0, const void *B1,
                       const float *Bs1, const Out &out, int M, int N, int K, const DeviceInfo &dev,
                       cudaStream_t stream) {
    if (M <= 8) return launch_stream<kMode, 8>(A, As, B0, Bs0, B1, Bs1, out, M, N, K, dev, stream);
    return launch_stream<kMode, 32>(A, As, B0, Bs0, B1, Bs1, out, M, N, K, dev, stream);
}

}  // namespace

cudaError_t launch_gemm_b128_stream(const void *A, const float *As, const void *B, const float *Bs,
                                    void *Y, int M, int N, int K, bool row_scales, int f32_out,
                                    const DeviceInfo &dev, cudaStream_t stream) {
    Out out{};
    out.y = Y;
    out.f32 = f32_out;
    return row_scales ? launch_tok<kRowScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream)
                      : launch_tok<kTileScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream);
}

cudaError_t launch_fwd_b128_stream(const void *X, const float *Xs, const void *Wg, const float *Gs,
                                   const void *Wu, const float *Us, void *H, int M, int N, int K,
                                   const Epilogue &epi, const DeviceInfo &dev, cudaStream_t stream) {
    Out out{};
    out.y = H;
    out.g = static_cast<__nv_bfloat16 *>(epi.G);
    out.u = static_cast<__nv_bfloat16 *>(epi.U);
    out.act = epi.activation;
    out.alpha = epi.gate_multiplier;
    return launch_tok<kGated>(X, Xs, Wg, Gs, Wu, Us, out, M, N, K, dev, stream);
}

cudaError_t gemm_b128_stream_status_fetch_and_clear(unsigned int *host_out, cudaStream_t stream) {
    return fetch_and_clear(g_gemm_b128_stream_status, host_out, stream);
}

}  // namespace swiglu
