// gemm_b128.cu -- products of e4m3 operands with one fp32 scale per block of
// 128 along the reduction, on the fp8 tensor cores (tcgen05 kind::f8f6f4):
//
//   Y[m, n] = sum_b As[m, b] Bs[n, b] sum_{k in block b} A[m, k] B[n, k]
//
// with Bs one value per row of B ("row") or per 128 rows ("tile"); and the
// gated pair, H = act(alpha G) * U with G and U such products of one A.
//
// The scales differ from block to block, so the tensor cores accumulate one
// 128-deep block only: four MMAs (K = 32) into a buffer of tensor memory,
// which eight warps read back, multiply by the block's scales and add to the
// running sums in their registers (fp32, round to nearest: 128 x 256 sums are
// 128 registers of 256 threads), while the next block's MMAs fill another
// buffer.  That read (128 x 256 x 4 bytes per 512 cycles of MMA) and its
// multiply-adds (packed in pairs) fit beside the MMAs.
//
//  * warps 0..7: accumulation and epilogue: warp w holds rows 32 (w mod 4)
//    .. +31, columns of one half of the tile;
//  * warp 8 (one thread): TMA producer of the codes' ring and of a second
//    ring with the blocks' scales (which are freed by other warps, later);
//  * warp 9 (one thread): MMA issuer (warps 10, 11 only give up registers).
//
// A tile is 128 rows of A by up to 256 columns (gated: 128 + 128, the rows of
// both weights stacked into one operand, one MMA per k step).  The columns are
// cut into units of 8 spread evenly over as many tiles as fill the SMs, so the
// same kernel streams the weights of a small batch (one tile of N / 148
// columns per SM) and runs the large products.
//
// Waits are bounded; a stuck pipeline sets the status word, the MMAs and
// copies in flight are drained and TMEM is freed before the kernel returns.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "gemm_common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tmap.cuh"

namespace swiglu {

// Status word of this translation unit's kernel (bit 0 = a wait gave up).
__device__ unsigned int g_gemm_b128_status;

namespace {

using namespace dev;
using gemm::mbar_wait_drain;
using gemm::tile_coords;

constexpr int kBM = 128;
constexpr int kBlockK = 128;                 // bytes = e4m3 values per block and stage row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 4);  // (register shares go by groups of 4 warps)
// 384 threads start with 168 registers each; the accumulating warps take
// what the third group of warps gives back: 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kRegsLaunch = 168, kRegsEpi = 224, kRegsRest = 56;
static_assert(256 * kRegsEpi + 128 * kRegsRest <= kThreads * kRegsLaunch, "register split");
constexpr int kMaxUnits = 32;                // units of 8 columns per tile
constexpr int kMaxStages = 24;
constexpr int kMaxBufs = 8;
constexpr int kMaxSlots = kMaxStages + kMaxBufs;
constexpr int kTmemCols = 512;
constexpr int kGroupM = 16;
constexpr uint32_t kStageOutBytes = 32 * 64;  // per epilogue warp: 32 rows x 64 bytes
constexpr uint32_t kNumBars = 2 * kMaxStages + 2 * kMaxSlots + 2 * kMaxBufs + 1;
constexpr uint32_t kTailBytes = 8 * kNumBars + 32 + 1024;  // + abort, TMEM slot, alignment
constexpr uint32_t kMaxSmem = 227 * 1024;

enum : int { kTileScales = 0, kRowScales = 1, kGated = 2 };

struct Plan {
    int tiles_m, tiles_n;
    int units;         // units of 8 output columns
    int q;             // tiles hold q or q + 1 units
    int a_rows;        // rows of an A box
    int b_rows;        // rows of the B part of a stage (a multiple of 16)
    int s_cols;        // row scales of B per block (columns of the widest tile)
    int stages, slots, bufs;
    int buf_cols;      // TMEM columns of a buffer
    uint32_t stage_bytes, slot_bytes;
    uint32_t off_slots, off_out, off_bar, smem;
    int num_kb;
};

struct Out {
    void *y;                 // Y or H
    __nv_bfloat16 *g, *u;    // gated: null or the two products
    int f32;
    int act;
    float alpha;
};

// mbar_wait for waits that are long by design: after one test the thread
// sleeps until the phase completes (or 20 us have passed) instead of polling,
// which leaves the issue slots to the accumulating warps.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            *abort_flag = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// acc += s * d on a pair of columns.
__device__ __forceinline__ void fma2(unsigned long long &acc, uint32_t d0, uint32_t d1,
                                     unsigned long long s) {
    asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(d0), "r"(d1), "l"(s));
}

__device__ __forceinline__ unsigned long long pair2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float lo2(unsigned long long v) {
    return __uint_as_float(static_cast<uint32_t>(v));
}
__device__ __forceinline__ float hi2(unsigned long long v) {
    return __uint_as_float(static_cast<uint32_t>(v >> 32));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A warp's 32 rows x 64 bytes to global memory through its staging buffer:
// lane = row writes its four 16-byte chunks (swizzled over the banks), then
// every four lanes store 64 consecutive bytes of a row.  `cols16` of the four
// chunks belong to the tile.
__device__ __forceinline__ void store_rows(uint32_t buf, int lane, const uint4 (&v)[4], char *dst,
                                           int64_t row_bytes, int rows, int cols16) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts_v4(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), v[j]);
    __syncwarp();
    const int j = lane & 3;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 8 + (lane >> 2);
        const uint4 w = lds_v4(buf + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
        if (r < rows && j < cols16) *reinterpret_cast<uint4 *>(dst + r * row_bytes + j * 16) = w;
    }
    __syncwarp();
}

// One block's 32 accumulator columns of a warp, times their scales, into the
// running sums.  Tile scales: the four units of 8 columns take slo below
// unit `cut` (counted from these columns) and shi from there on.
__device__ __forceinline__ void add_tile(unsigned long long (&acc)[16], const uint32_t (&v)[32],
                                         float slo, float shi, int cut) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float s = u < cut ? slo : shi;
        const unsigned long long s2 = pair2(s, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) fma2(acc[4 * u + i], v[8 * u + 2 * i], v[8 * u + 2 * i + 1], s2);
    }
}

// The same with one scale for all 32 columns.
__device__ __forceinline__ void add_block(unsigned long long (&acc)[16], const uint32_t (&v)[32], float s) {
    const unsigned long long s2 = pair2(s, s);
#pragma unroll
    for (int i = 0; i < 16; ++i) fma2(acc[i], v[2 * i], v[2 * i + 1], s2);
}

// Row scales: one per column, in shared memory at sb.
__device__ __forceinline__ void add_rows(unsigned long long (&acc)[16], const uint32_t (&v)[32],
                                         float sa, uint32_t sb) {
    const unsigned long long sa2 = pair2(sa, sa);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 w = lds_v4(sb + 16u * i);
        const unsigned long long s0 = pair2(__uint_as_float(w.x), __uint_as_float(w.y));
        const unsigned long long s1 = pair2(__uint_as_float(w.z), __uint_as_float(w.w));
        fma2(acc[2 * i], v[4 * i], v[4 * i + 1], mul2(s0, sa2));
        fma2(acc[2 * i + 1], v[4 * i + 2], v[4 * i + 3], mul2(s1, sa2));
    }
}

// A warp's share of a tile, from its sums to global memory: rows row0 .. (at
// most 32, `rows` of them), columns colg .. of `mine` units of 8.  acc[0..3]:
// groups of 32 columns (gated: 0, 1 of G and 2, 3 of U).
template <int kMode>
__device__ __forceinline__ void store_tile(const unsigned long long (&acc)[4][16], const Out &out,
                                           uint32_t buf, int lane, int64_t row0, int64_t colg, int N,
                                           int rows, int mine) {
    auto put_bf16 = [&](void *y, int group, int units_left, auto value) {
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = make_uint4(value(4 * c), value(4 * c + 1), value(4 * c + 2), value(4 * c + 3));
        store_rows(buf, lane, v, static_cast<char *>(y) + 2 * (row0 * N + colg + 32 * group), 2ll * N,
                   rows, units_left);
    };
    if constexpr (kMode == kGated) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int left = mine - 4 * j;
            if (left > 0) {
                put_bf16(out.y, j, left, [&](int i) {
                    return pack_bf16x2(
                        act::gated<false>(out.act, out.alpha, lo2(acc[j][i]), lo2(acc[2 + j][i])),
                        act::gated<false>(out.act, out.alpha, hi2(acc[j][i]), hi2(acc[2 + j][i])));
                });
                if (out.g) {
                    put_bf16(out.g, j, left, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
                    put_bf16(out.u, j, left,
                             [&](int i) { return pack_bf16x2(lo2(acc[2 + j][i]), hi2(acc[2 + j][i])); });
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = mine - 4 * j;
            if (left > 0) {
                if (!out.f32) {
                    put_bf16(out.y, j, left, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 columns = 64 bytes each
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const unsigned long long a0 = acc[j][8 * h + 2 * c], a1 = acc[j][8 * h + 2 * c + 1];
                            v[c] = make_uint4(static_cast<uint32_t>(a0), static_cast<uint32_t>(a0 >> 32),
                                              static_cast<uint32_t>(a1), static_cast<uint32_t>(a1 >> 32));
                        }
                        store_rows(buf, lane, v,
                                   static_cast<char *>(out.y) + 4 * (row0 * N + colg + 32 * j + 16 * h),
                                   4ll * N, rows, 2 * (left - 2 * h));
                    }
                }
            }
        }
    }
}

// tm_b*: rows of B (gated: of Wg and Wu), boxes of 8 q (lo) and 8 (q + 1)
// (hi) rows.  tm_as: As [blocks][M], boxes of 128 values; tm_bs: Bs
// [blocks][N] of the row form, boxes of the widest tile's columns.  bs0, bs1: [N/128][blocks]
// scales of the tile forms.
template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    swiglu_gemm_b128_kernel(const __grid_constant__ CUtensorMap tm_a,
                            const __grid_constant__ CUtensorMap tm_as,
                            const __grid_constant__ CUtensorMap tm_b_lo,
                            const __grid_constant__ CUtensorMap tm_b_hi,
                            const __grid_constant__ CUtensorMap tm_u_lo,
                            const __grid_constant__ CUtensorMap tm_u_hi,
                            const __grid_constant__ CUtensorMap tm_bs,
                            const float *__restrict__ bs0, const float *__restrict__ bs1,
                            const Out out, int M, int N, const Plan p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar_full = base + p.off_bar;
    const uint32_t bar_empty = bar_full + 8 * kMaxStages;
    const uint32_t bar_sfull = bar_empty + 8 * kMaxStages;
    const uint32_t bar_sempty = bar_sfull + 8 * kMaxSlots;
    const uint32_t bar_tfull = bar_sempty + 8 * kMaxSlots;
    const uint32_t bar_tempty = bar_tfull + 8 * kMaxBufs;
    const uint32_t bar_drain = bar_tempty + 8 * kMaxBufs;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(gbase + p.off_bar + 8 * kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + p.off_bar + 8 * kNumBars + 16);

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const int num_tiles = p.tiles_m * p.tiles_n;
    const int num_kb = p.num_kb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < p.slots; ++s) {
            mbar_init(bar_sfull + 8 * s, 1);
            mbar_init(bar_sempty + 8 * s, kEpiWarps);
        }
        for (int b = 0; b < p.bufs; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, kEpiWarps);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_as);
        tma_prefetch_desc(&tm_b_lo);
        tma_prefetch_desc(&tm_b_hi);
        if (kMode == kGated) {
            tma_prefetch_desc(&tm_u_lo);
            tma_prefetch_desc(&tm_u_hi);
        }
        if (kMode == kRowScales) tma_prefetch_desc(&tm_bs);
    }
    if (warp == kEpiWarps + 1) {
        tmem_alloc(smem_u32(tmem_ptr), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_ptr);

    // tile t: rows m0 .., units u0 .. u0 + cnt of 8 columns
    auto tile_of = [&](int t, int &m0, int &u0, int &cnt) {
        int mt, nt;
        tile_coords<kGroupM>(t, p.tiles_m, p.tiles_n, mt, nt);
        m0 = mt * kBM;
        u0 = static_cast<int>(static_cast<long long>(p.units) * nt / p.tiles_n);
        cnt = static_cast<int>(static_cast<long long>(p.units) * (nt + 1) / p.tiles_n) - u0;
    };

    bool failed = false;

    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kEpiWarps && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, slot = 0;
            uint32_t phase = 0, sphase = 0;
            long long issued = 0;
            for (int t = blockIdx.x; t < num_tiles && !failed; t += gridDim.x) {
                int m0, u0, cnt;
                tile_of(t, m0, u0, cnt);
                const CUtensorMap *tb = cnt > p.q ? &tm_b_hi : &tm_b_lo;
                const CUtensorMap *tu = cnt > p.q ? &tm_u_hi : &tm_u_lo;
                const uint32_t weights = static_cast<uint32_t>(cnt) * 1024u;
                const uint32_t bytes = static_cast<uint32_t>(p.a_rows) * 128u +
                                       (kMode == kGated ? 2u : 1u) * weights;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag) ||
                        !mbar_wait(bar_sempty + 8 * slot, sphase ^ 1u, abort_flag)) {
                        failed = true;
                        break;
                    }
                    const uint32_t fb = bar_full + 8 * stage;
                    const uint32_t a_dst = base + stage * p.stage_bytes;
                    const uint32_t b_dst = a_dst + static_cast<uint32_t>(p.a_rows) * 128u;
                    mbar_arrive_expect_tx(fb, bytes);
                    tma_load_2d(tb, fb, b_dst, kb * kBlockK, 8 * u0);
                    if (kMode == kGated) tma_load_2d(tu, fb, b_dst + weights, kb * kBlockK, 8 * u0);
                    tma_load_2d(&tm_a, fb, a_dst, kb * kBlockK, m0);
                    const uint32_t sb = bar_sfull + 8 * slot;
                    const uint32_t s_dst = base + p.off_slots + slot * p.slot_bytes;
                    mbar_arrive_expect_tx(sb, 512u + (kMode == kRowScales ? 4u * p.s_cols : 0u));
                    tma_load_2d(&tm_as, sb, s_dst, m0, kb);
                    if (kMode == kRowScales) tma_load_2d(&tm_bs, sb, s_dst + 512u, 8 * u0, kb);
                    ++issued;
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++slot == p.slots) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            // Never leave while a load issued here may still write shared memory.
            for (int s = 0; s < p.stages; ++s)
                if (issued > s)
                    mbar_wait_drain(bar_full + 8 * s,
                                    static_cast<uint32_t>(((issued - 1 - s) / p.stages) & 1));
            for (int s = 0; s < p.slots; ++s)
                if (issued > s)
                    mbar_wait_drain(bar_sfull + 8 * s,
                                    static_cast<uint32_t>(((issued - 1 - s) / p.slots) & 1));
        }
        if (warp == kEpiWarps + 1 && lane == 0) {
            // ------------------------------------------------- MMA issuer
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            for (int t = blockIdx.x; t < num_tiles && !failed; t += gridDim.x) {
                int m0, u0, cnt;
                tile_of(t, m0, u0, cnt);
                const uint32_t cols = static_cast<uint32_t>((kMode == kGated ? 16 : 8) * cnt);
                // (an odd unit count reads 8 rows past its box: columns never read)
                const uint32_t idesc = make_idesc(0u, kBM, (cols + 15u) / 16u * 16u);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(bar_tempty + 8 * buf, bphase ^ 1u, abort_flag) ||
                        !mbar_wait(bar_full + 8 * stage, phase, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = base + stage * p.stage_bytes;
                    const uint64_t ad = sw128_kmajor_desc(a);
                    const uint64_t bd = sw128_kmajor_desc(a + static_cast<uint32_t>(p.a_rows) * 128u);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * p.buf_cols);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                    mma_commit(bar_empty + 8 * stage);
                    mma_commit(bar_tfull + 8 * buf);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == p.bufs) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
            // Every MMA issued here must finish before TMEM is released.
            mma_commit(bar_drain);
            mbar_wait_drain(bar_drain, 0);
        }
    } else {
        // ------------------------------------------ accumulation + epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t row_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t obuf = base + p.off_out + static_cast<uint32_t>(warp) * kStageOutBytes;
        int slot = 0, buf = 0;
        uint32_t sphase = 0, bphase = 0;
        for (int t = blockIdx.x; t < num_tiles && !failed; t += gridDim.x) {
            int m0, u0, cnt;
            tile_of(t, m0, u0, cnt);
            // this warp's units of the tile: whole groups of 32 columns below,
            // the rest above (gated: of both products)
            const int split = min(cnt, ((cnt + 1) / 2 + 3) / 4 * 4);
            const int first = half ? split : 0;
            const int mine = half ? cnt - split : split;
            const int rows = min(32, M - m0 - 32 * quad);  // <= 0: none
            const bool work = rows > 0 && mine > 0;
            // columns of the accumulator groups 0,1 (plain: the first 64 of
            // this warp, gated: G) and 2,3 (the next 64, or U)
            const uint32_t col0 = static_cast<uint32_t>(8 * first);
            const uint32_t col2 = kMode == kGated ? col0 + static_cast<uint32_t>(8 * cnt) : col0 + 64u;
            // tile scales: 64 columns span at most two blocks of 128, the
            // second from unit `cut` of the 64 on
            const float *sc[2][2] = {};
            int cut[2] = {8, 8};
            float cur[2][2] = {};
            if (kMode != kRowScales && work) {
                const int blocks = (N + 127) / 128;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int unit = u0 + first + (kMode == kGated ? 0 : 8 * g);
                    const int b = min(unit / 16, blocks - 1);
                    cut[g] = 16 * (b + 1) - unit;
                    const float *table = (kMode == kGated && g == 1) ? bs1 : bs0;
                    sc[g][0] = table + static_cast<int64_t>(b) * num_kb;
                    sc[g][1] = table + static_cast<int64_t>(min(b + 1, blocks - 1)) * num_kb;
                    cur[g][0] = __ldg(sc[g][0]);
                    cur[g][1] = __ldg(sc[g][1]);
                }
            }
            unsigned long long acc[4][16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][i] = 0ull;

            for (int kb = 0; kb < num_kb; ++kb) {
                // the next block's tile scales, one block ahead of their use
                float nxt[2][2] = {};
                if (kMode != kRowScales && work && kb + 1 < num_kb) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        nxt[g][0] = __ldg(sc[g][0] + kb + 1);
                        nxt[g][1] = __ldg(sc[g][1] + kb + 1);
                    }
                }
                if (!mbar_wait(bar_sfull + 8 * slot, sphase, abort_flag)) {
                    failed = true;
                    break;
                }
                const uint32_t s_src = base + p.off_slots + slot * p.slot_bytes;
                const float sa = lds_f32(s_src + 4u * (quad * 32 + lane));
                if (!mbar_wait(bar_tfull + 8 * buf, bphase, abort_flag)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (work) {
                    const uint32_t d = tmem_base + row_off + static_cast<uint32_t>(buf * p.buf_cols);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int unit = 4 * (kMode == kGated ? (j & 1) : j);  // of this warp
                        if (unit < mine) {
                            uint32_t v[32];
                            const uint32_t col = (j < 2 ? col0 : col2) + 32u * (j & 1);
                            tmem_ld_32x32b_x32(d + col, v);
                            if (kMode == kRowScales) {
                                const unsigned long long sa2 = pair2(sa, sa);
                                const uint32_t sb = s_src + 512u + 4u * col;
                                tmem_ld_wait(v);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint4 w = lds_v4(sb + 16u * i);
                                    const unsigned long long s0 =
                                        pair2(__uint_as_float(w.x), __uint_as_float(w.y));
                                    const unsigned long long s1 =
                                        pair2(__uint_as_float(w.z), __uint_as_float(w.w));
                                    fma2(acc[j][2 * i], v[4 * i], v[4 * i + 1], mul2(s0, sa2));
                                    fma2(acc[j][2 * i + 1], v[4 * i + 2], v[4 * i + 3], mul2(s1, sa2));
                                }
                            } else {
                                const int g = j >> 1;
                                const float slo = sa * cur[g][0], shi = sa * cur[g][1];
                                tmem_ld_wait(v);
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const float s = 4 * (j & 1) + u < cut[g] ? slo : shi;
                                    const unsigned long long s2 = pair2(s, s);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        fma2(acc[j][4 * u + i], v[8 * u + 2 * i], v[8 * u + 2 * i + 1], s2);
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_tempty + 8 * buf);
                    mbar_arrive(bar_sempty + 8 * slot);
                }
                if (kMode != kRowScales) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        cur[g][0] = nxt[g][0];
                        cur[g][1] = nxt[g][1];
                    }
                }
                if (++slot == p.slots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                if (++buf == p.bufs) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            if (failed || !work) continue;
            // ------------------------------------------------------ store
            const int64_t row0 = m0 + 32 * quad;
            const int64_t colg = 8 * (static_cast<int64_t>(u0) + first);
            auto put_bf16 = [&](void *y, int group, int units_left, auto value) {
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] = make_uint4(value(4 * c), value(4 * c + 1), value(4 * c + 2), value(4 * c + 3));
                store_rows(obuf, lane, v,
                           static_cast<char *>(y) + 2 * (row0 * N + colg + 32 * group), 2ll * N, rows,
                           units_left);
            };
            if constexpr (kMode == kGated) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int left = mine - 4 * j;
                    if (left > 0) {
                        put_bf16(out.y, j, left, [&](int i) {
                            return pack_bf16x2(
                                act::gated<false>(out.act, out.alpha, lo2(acc[j][i]), lo2(acc[2 + j][i])),
                                act::gated<false>(out.act, out.alpha, hi2(acc[j][i]), hi2(acc[2 + j][i])));
                        });
                        if (out.g) {
                            put_bf16(out.g, j, left, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
                            put_bf16(out.u, j, left, [&](int i) { return pack_bf16x2(lo2(acc[2 + j][i]), hi2(acc[2 + j][i])); });
                        }
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int left = mine - 4 * j;
                    if (left > 0) {
                        if (!out.f32) {
                            put_bf16(out.y, j, left, [&](int i) { return pack_bf16x2(lo2(acc[j][i]), hi2(acc[j][i])); });
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {  // 16 columns = 64 bytes each
                                uint4 v[4];
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const unsigned long long a0 = acc[j][8 * h + 2 * c], a1 = acc[j][8 * h + 2 * c + 1];
                                    v[c] = make_uint4(static_cast<uint32_t>(a0), static_cast<uint32_t>(a0 >> 32),
                                                      static_cast<uint32_t>(a1), static_cast<uint32_t>(a1 >> 32));
                                }
                                store_rows(obuf, lane, v,
                                           static_cast<char *>(out.y) + 4 * (row0 * N + colg + 32 * j + 16 * h),
                                           4ll * N, rows, 2 * (left - 2 * h));
                            }
                        }
                    }
                }
            }
        }
    }

    if (failed) atomicOr(&g_gemm_b128_status, 1u);

    tc_fence_before();
    __syncthreads();
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// Pairs of SMs (M > 128): each MMA covers 256 rows over the two CTAs of a
// cluster (tcgen05 cta_group::2).  A CTA holds its own 128 rows of A and half
// of the tile's rows of B (gated: the even CTA the rows of Wg, the odd one
// those of Wu), so a stage is 32 KB instead of 48 and both the copies' writes
// and the MMAs' reads of shared memory shrink by a third; each CTA accumulates
// its own 128 rows.  The even CTA issues the MMAs; three threads of each CTA
// issue its copies (B; A; the scales), one copy per block each, since one
// thread issuing all of them took longer than a block's MMAs.

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
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;"
        "\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(z)
        : "memory");
}

// Arrive on the barrier at this offset of both CTAs' shared memory when every
// MMA issued so far by this thread has completed (one commit for the pair:
// B200, M = 8192 N = 4096 K = 14336, the MMAs alone: 2.5 PFLOP/s with a commit
// per CTA, PLACEHOLDER with this).
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
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
                                 const float *__restrict__ bs0, const float *__restrict__ bs1,
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
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_ptr);

    // tile t: the CTA's rows m0 .., the tile's groups g0 .. g0 + cnt of 32 columns
    auto tile_of = [&](int t, int &m0, int &g0, int &cnt) {
        int mt, nt;
        tile_coords<kGroupM / 2>(t, p.tiles_m, p.tiles_n, mt, nt);
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
                    if (kMode != kRowScales) v = __ldg(src + min(kb + lane / 8, num_kb - 1));
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
        if (warp == kEpiWarps + 1 && lane == 0 && rank == 0) {
            // ------------------------------------------ MMA issuer (pair)
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
            mma_commit_pair(bar_drain);
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
            float sa = 0.0f, sb[4] = {};
            uint32_t srow = 0;        // this block's row scales of B
            uint32_t v[2][32];
            // One block ahead: wait for its accumulators, start reading them,
            // and fetch its scales.
            auto open_block = [&](bool new_slot) -> bool {
                if (new_slot) {
                    if (!mbar_wait_long(bar_sfull + 8 * slot, sphase, abort_flag)) return false;
                    pa = base + L::kOffSlots + slot * L::kSlotBytes + 4u * (quad * 32 + lane);
                    pb = base + L::kOffSlots + slot * L::kSlotBytes + L::kOffB + (kMode == kRowScales ? 0u : 16u * half);
                }
                if (!mbar_wait_long(bar_tfull + buf8, bphase, abort_flag)) return false;
                tc_fence_after();
                if (groups == 0) return true;
                tmem_ld_32x32b_x32(lanes + 32u * buf8 + col0, v[0]);
                sa = lds_f32(pa);
                pa += 512u;
                if constexpr (kMode != kRowScales) {
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
                for (int j = 0; j < 4; ++j) s[j] = sa * sb[j];
                const float sa_now = sa;
                const uint32_t srow_now = srow;
                auto read = [&](int o) {
                    tmem_ld_32x32b_x32(d + (o < 2 ? col0 : col2) + 32u * (o & 1), v[o & 1]);
                };
                auto add = [&](int o) {
                    if constexpr (kMode == kRowScales)
                        add_rows(acc[o], v[o & 1], sa_now, srow_now + 4u * ((o < 2 ? col0 : col2) + 32u * (o & 1)));
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
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sts_v4(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4),
                           make_uint4(value(4 * c), value(4 * c + 1), value(4 * c + 2), value(4 * c + 3)));
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
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const unsigned long long a0 = acc[j][2 * c], a1 = acc[j][2 * c + 1];
                            sts_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4),
                                   make_uint4(static_cast<uint32_t>(a0), static_cast<uint32_t>(a0 >> 32),
                                              static_cast<uint32_t>(a1), static_cast<uint32_t>(a1 >> 32)));
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

// Tiles over the columns, as make_plan, for tiles of 256 rows over `pairs`
// pairs of SMs, in groups of 32 columns (a group has one tile scale, and the
// pair's MMA takes N in steps of 32).
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

std::atomic<unsigned> g_pair_attr_set_mask[3];

template <int kMode>
cudaError_t launch_pair(const void *A, const float *As, const void *B0, const float *Bs0,
                        const void *B1, const float *Bs1, const Out &out, int M, int N, int K,
                        const DeviceInfo &dev, cudaStream_t stream) {
    auto kernel = swiglu_gemm_b128_pair_kernel<kMode>;
    const unsigned bit = 1u << (dev.device & 31);
    if (!(g_pair_attr_set_mask[kMode].load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(PairLayout<kMode>::kSmem));
        if (e != cudaSuccess) return e;
        // the register split needs the whole launch's registers
        cudaFuncAttributes fa{};
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
        g_pair_attr_set_mask[kMode].fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = PairLayout<kMode>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2);
    int max_clusters = 0;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&max_clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (max_clusters < 1) return cudaErrorInvalidConfiguration;
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

// Tiles over the columns and the ring.  A tile costs its columns plus a
// constant (its rows of A are loaded and read whatever its width), and the
// tiles of all rows run in waves over the SMs: the cheapest count wins.
Plan make_plan(int M, int N, int K, bool gated, bool row_scales, int sm_count) {
    Plan p{};
    p.tiles_m = (M + kBM - 1) / kBM;
    p.units = N / 8;
    p.num_kb = (K + kBlockK - 1) / kBlockK;
    const int per_unit = gated ? 16 : 8;               // accumulator columns
    const int max_units = kMaxUnits * 8 / per_unit;
    const int least = (p.units + max_units - 1) / max_units;
    const int most = p.units < least + sm_count ? p.units : least + sm_count;
    long long best = -1;
    for (int tn = least; tn <= most; ++tn) {
        const int cols = (p.units + tn - 1) / tn * per_unit;
        const long long waves = (static_cast<long long>(p.tiles_m) * tn + sm_count - 1) / sm_count;
        const long long cost = waves * (cols + 48);
        if (best < 0 || cost < best) {
            best = cost;
            p.tiles_n = tn;
        }
    }
    p.q = p.units / p.tiles_n;
    const int widest = (p.units + p.tiles_n - 1) / p.tiles_n * per_unit;
    p.a_rows = p.tiles_m == 1 ? (M + 7) / 8 * 8 : kBM;
    p.b_rows = (widest + 15) / 16 * 16;
    p.buf_cols = gated ? (widest / 2 + (widest / 2 + 31) / 32 * 32 + 31) / 32 * 32
                       : (widest + 31) / 32 * 32;
    p.bufs = kTmemCols / p.buf_cols < kMaxBufs ? kTmemCols / p.buf_cols : kMaxBufs;
    p.stage_bytes = static_cast<uint32_t>(p.a_rows + p.b_rows) * 128u;
    p.s_cols = row_scales ? widest : 0;
    p.slot_bytes = 512u + (row_scales ? 1024u : 0u);   // 128 + up to 256 values
    // behind the ring: slack for the A operand's rows beyond its box
    const uint32_t slack = static_cast<uint32_t>(kBM - p.a_rows) * 128u;
    const uint32_t fixed = slack + kEpiWarps * kStageOutBytes + kTailBytes;
    int stages = kMaxStages;
    for (; stages > 2; --stages) {
        p.slots = stages + p.bufs;
        if (fixed + stages * p.stage_bytes + p.slots * p.slot_bytes <= kMaxSmem) break;
    }
    p.stages = stages;
    p.slots = stages + p.bufs;
    p.off_slots = p.stages * p.stage_bytes + slack;
    p.off_out = (p.off_slots + p.slots * p.slot_bytes + 127u) / 128u * 128u;
    p.off_bar = p.off_out + kEpiWarps * kStageOutBytes;
    p.smem = p.off_bar + kTailBytes;
    return p;
}

std::atomic<unsigned> g_attr_set_mask[3];

template <int kMode>
cudaError_t launch(const void *A, const float *As, const void *B0, const float *Bs0, const void *B1,
                   const float *Bs1, const Out &out, int M, int N, int K, const DeviceInfo &dev,
                   cudaStream_t stream) {
    if (M > kBM) return launch_pair<kMode>(A, As, B0, Bs0, B1, Bs1, out, M, N, K, dev, stream);
    const Plan p = make_plan(M, N, K, kMode == kGated, kMode == kRowScales, dev.sm_count);
    if (p.smem > kMaxSmem || p.bufs < 2) return cudaErrorInvalidValue;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapDataType f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapSwizzle none = CU_TENSOR_MAP_SWIZZLE_NONE;
    const uint64_t k64 = static_cast<uint64_t>(K), n64 = static_cast<uint64_t>(N);
    const uint32_t lo = 8u * p.q;
    const uint32_t hi = p.units % p.tiles_n ? lo + 8u : lo;  // (no tile holds more: same box)
    CUtensorMap ta, tas, tb_lo, tb_hi, tu_lo, tu_hi, tbs;
    if (!encode_tmap_2d(&ta, A, u8, k64, M, k64, kBlockK, static_cast<uint32_t>(p.a_rows), sw) ||
        !encode_tmap_2d(&tas, As, f32, M, p.num_kb, static_cast<uint64_t>((M + 3) / 4 * 4) * 4, 128, 1,
                        none) ||
        !encode_tmap_2d(&tb_lo, B0, u8, k64, n64, k64, kBlockK, lo, sw) ||
        !encode_tmap_2d(&tb_hi, B0, u8, k64, n64, k64, kBlockK, hi, sw))
        return cudaErrorInvalidValue;
    tu_lo = tb_lo;
    tu_hi = tb_hi;
    tbs = tas;
    if (kMode == kGated && (!encode_tmap_2d(&tu_lo, B1, u8, k64, n64, k64, kBlockK, lo, sw) ||
                            !encode_tmap_2d(&tu_hi, B1, u8, k64, n64, k64, kBlockK, hi, sw)))
        return cudaErrorInvalidValue;
    if (kMode == kRowScales &&
        !encode_tmap_2d(&tbs, Bs0, f32, n64, p.num_kb, n64 * 4, static_cast<uint32_t>(p.s_cols), 1, none))
        return cudaErrorInvalidValue;
    const unsigned bit = 1u << (dev.device & 31);
    if (!(g_attr_set_mask[kMode].load() & bit)) {
        cudaError_t e = cudaFuncSetAttribute(swiglu_gemm_b128_kernel<kMode>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMaxSmem));
        if (e != cudaSuccess) return e;
        // the register split needs the whole launch's registers
        cudaFuncAttributes fa{};
        e = cudaFuncGetAttributes(&fa, swiglu_gemm_b128_kernel<kMode>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
        g_attr_set_mask[kMode].fetch_or(bit);
    }
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    const int grid = static_cast<int>(tiles < dev.sm_count ? tiles : dev.sm_count);
    swiglu_gemm_b128_kernel<kMode><<<grid, kThreads, p.smem, stream>>>(
        ta, tas, tb_lo, tb_hi, tu_lo, tu_hi, tbs, Bs0, Bs1, out, M, N, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_b128(const void *A, const float *As, const void *B, const float *Bs,
                             void *Y, int M, int N, int K, bool row_scales, int f32_out,
                             const DeviceInfo &dev, cudaStream_t stream) {
    Out out{};
    out.y = Y;
    out.f32 = f32_out;
    return row_scales ? launch<kRowScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream)
                      : launch<kTileScales>(A, As, B, Bs, nullptr, nullptr, out, M, N, K, dev, stream);
}

cudaError_t launch_fwd_b128(const void *X, const float *Xs, const void *Wg, const float *Gs,
                            const void *Wu, const float *Us, void *H, int M, int N, int K,
                            const Epilogue &epi, const DeviceInfo &dev, cudaStream_t stream) {
    Out out{};
    out.y = H;
    out.g = static_cast<__nv_bfloat16 *>(epi.G);
    out.u = static_cast<__nv_bfloat16 *>(epi.U);
    out.act = epi.activation;
    out.alpha = epi.gate_multiplier;
    return launch<kGated>(X, Xs, Wg, Gs, Wu, Us, out, M, N, K, dev, stream);
}

cudaError_t gemm_b128_status_fetch_and_clear(unsigned int *host_out, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(host_out, g_gemm_b128_status, sizeof(unsigned int), 0,
                                              cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_gemm_b128_status, &zero, sizeof(unsigned int), 0,
                                cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace swiglu
