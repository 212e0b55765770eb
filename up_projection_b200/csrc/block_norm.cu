// block_norm.cu -- the norms on either side of a block boundary, fused with
// the block's gate, residual scale and residual sum; forward and backward.
//
//   P  = W1 * Y * r1            r1 = 1 / sqrt(mean(Y^2) + eps)     (post-norm)
//   R' = R + s * g * P                                             (residual)
//   N  = W2 * R' * r2           r2 = 1 / sqrt(mean(R'^2) + eps)    (pre-norm)
//
// per row of D elements; without W1, P = Y; without W2 there is no N; without
// g, g = 1.  R' enters r2 and N before it is rounded to the storage type.
//
// Backward, from dR' and dN, with n = R' r2, y = Y r1, a = W2 dN:
//   dX  = dR' + r2 (a - n mean(a n))                    (= dR)
//   dY  = r1 (b - y mean(b y)),   b = W1 s g dX         (no W1: dY = s g dX)
//   dW2 = sum_m dN n,  dW1 = sum_m s g dX y,  dg = s W1 sum_m dX y.
// mean(b y) = (sum t e - r2 mean(a n) sum t n) / D with t = W1 s g y and
// e = dR' + r2 a, so one row needs ONE reduction (of three sums) and not two.
//
// All sums and statistics are fp32; each output is rounded once.
#include <cuda_bf16.h>

#include <atomic>

#include "kernels.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "status.cuh"

namespace swiglu {

// Status word of this translation unit's kernels (bit 0 = a wait gave up).
__device__ unsigned int g_block_norm_status;

namespace {

using namespace dev;

constexpr int kRowThreadsMax = 512;
constexpr int kBlockThreads = 256;  // row groups fill a block up to this

// Pairs of fp32 values: one instruction for two operations.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float lo2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(f2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

template <bool kBf16>
struct Vec {
    static constexpr int kE = kBf16 ? 8 : 4;  // elements per 16 bytes
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[kE]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBf16) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    }
    // four consecutive elements
    static __device__ __forceinline__ float4 load4(const uint4 *p, int64_t i) {
        if constexpr (kBf16) {
            const uint2 x = ld_plain(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i));
            return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                               __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
        } else {
            return ld_plain(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i));
        }
    }
    static __device__ __forceinline__ void store4(uint4 *p, int64_t i, const float4 &x) {
        if constexpr (kBf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
            *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p) + i) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        } else {
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i) = x;
        }
    }
    static __device__ __forceinline__ void unpack2(const uint4 &v, f2 (&f)[kE / 2]) {
        float x[kE];
        unpack(v, x);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) f[i] = pack2(x[2 * i], x[2 * i + 1]);
    }
    static __device__ __forceinline__ uint4 pack_pairs(const f2 (&f)[kE / 2]) {
        float x[kE];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            x[2 * i] = lo2(f[i]);
            x[2 * i + 1] = hi2(f[i]);
        }
        return pack(x);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[kE]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBf16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                w[i] = __float_as_uint(f[i]);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ void row_barrier(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

__device__ __forceinline__ void block_barrier(int threads) {
    asm volatile("bar.sync 15, %0;" ::"r"(threads) : "memory");
}

// Sum of K values over the T = 32 * warps threads (tid) of a row group.  `slots`
// is the group's shared memory, two sets of K * 16 floats used in turn, so
// one barrier per reduction is enough: a set is rewritten only after the
// barrier of the next reduction, which every reader of this one has reached.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *slots, int &turn, int group, int tid,
                                        int threads) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    const int warps = threads >> 5;
    if (warps == 1) return;
    float *s = slots + turn * (K * 16);
    turn ^= 1;
    const int w = tid >> 5;
    if ((tid & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k * 16 + w] = v[k];
    }
    row_barrier(group, threads);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float t = 0.0f;
        for (int i = 0; i < warps; ++i) t += s[k * 16 + i];
        v[k] = t;
    }
}

struct NormArgs {
    const uint4 *Y, *R;
    const uint4 *w1, *w2, *gate;   // any may be null
    uint4 *Rn, *N;
    float *rstd1, *rstd2;          // may be null
    int64_t M;
    int64_t rows_per_gate;
    int D;                         // elements
    float scale, eps;
};

// kV: 16-byte vectors per thread and row (vector v of a thread is column
// block v * blockDim.x + threadIdx.x).
template <bool kBf16, int kV>
__global__ void __launch_bounds__(kRowThreadsMax) block_norm_kernel(const NormArgs a) {
    using E = Vec<kBf16>;
    constexpr int kE = E::kE;
    __shared__ float slots[8][2 * 16];
    const int T = blockDim.x, tid = threadIdx.x, grp = threadIdx.y;
    const int nvec = a.D / kE;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    int turn = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + grp; row < a.M;
         row += stride) {
        const int64_t base = row * nvec;
        uint4 y[kV], r[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = v * T + tid;
            y[v] = r[v] = make_uint4(0, 0, 0, 0);
            if (c < nvec) {
                y[v] = ld_stream_v4(a.Y + base + c);
                r[v] = ld_stream_v4(a.R + base + c);
            }
        }
        float r1 = 1.0f;
        if (a.w1) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                float f[kE];
                E::unpack(y[v], f);
#pragma unroll
                for (int i = 0; i < kE; ++i) s[0] = fmaf(f[i], f[i], s[0]);
            }
            row_sum<1>(s, slots[grp], turn, grp, tid, T);
            r1 = 1.0f / sqrtf(s[0] * inv_d + a.eps);
            if (a.rstd1 && tid == 0) a.rstd1[row] = r1;
        }
        const float sr1 = a.scale * r1;
        const uint4 *gate = a.gate ? a.gate + (row / a.rows_per_gate) * nvec : nullptr;
        float rn[kV][kE];
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = v * T + tid;
            float f[kE], q[kE];
            E::unpack(y[v], f);
            E::unpack(r[v], q);
            if (c < nvec) {
                float w[kE];
#pragma unroll
                for (int i = 0; i < kE; ++i) w[i] = 1.0f;
                if (a.w1) E::unpack(ld_plain(a.w1 + c), w);
                if (gate) {
                    float g[kE];
                    E::unpack(ld_plain(gate + c), g);
#pragma unroll
                    for (int i = 0; i < kE; ++i) w[i] *= g[i];
                }
#pragma unroll
                for (int i = 0; i < kE; ++i) f[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                rn[v][i] = fmaf(sr1, f[i], q[i]);
                s[0] = fmaf(rn[v][i], rn[v][i], s[0]);
            }
            if (c < nvec) st_stream_v4(a.Rn + base + c, E::pack(rn[v]));
        }
        if (a.w2) {
            row_sum<1>(s, slots[grp], turn, grp, tid, T);
            const float r2 = 1.0f / sqrtf(s[0] * inv_d + a.eps);
            if (a.rstd2 && tid == 0) a.rstd2[row] = r2;
            // Long rows take W2 at once: a load does not move over a store
            // (300 x 16384 bf16 15.2 against 15.8 us, 100 x 8192 fp32 6.1 and
            // 6.3; with two vectors the registers cost a block per SM).
            constexpr bool kAtOnce = kV > 2;
            uint4 w2[kAtOnce ? kV : 1];
#pragma unroll
            for (int v = 0; kAtOnce && v < kV; ++v)
                if (v * T + tid < nvec) w2[v] = ld_plain(a.w2 + v * T + tid);
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                if (c < nvec) {
                    float w[kE];
                    E::unpack(kAtOnce ? w2[kAtOnce ? v : 0] : ld_plain(a.w2 + c), w);
#pragma unroll
                    for (int i = 0; i < kE; ++i) w[i] *= rn[v][i] * r2;
                    st_stream_v4(a.N + base + c, E::pack(w));
                }
            }
        }
    }
}

// ----------------------------------------------------------- row rings
// With many rows, rows arrive by bulk copies.  Each row group has a ring of
// `stages` rows of its operands in shared memory, filled by its first thread:
// the sums of a row end with a barrier of the group, after which the stage of
// the row before it is free.  What is in flight then depends neither on
// registers nor on where the groups stand between their loads, sums and
// stores.

constexpr int kMaxRing = 8;
constexpr int kMaxGroups = 16;   // row groups of one warp; of more, at most 8
constexpr int kRingThreads = 512;
constexpr uint32_t kRingRoom = 220 * 1024;

// A wait of the ring that gave up: no further copies are made, and those under
// way end before the block does.
__device__ __noinline__ void ring_abandon(uint32_t full, int stages, int stage, uint32_t phase) {
    for (int i = 0; i < stages; ++i) {
        int never = 0;
        (void)mbar_wait(full + 8 * stage, phase, &never);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

// The forward over runs of consecutive rows, one run per block; W1 g and W2
// stay in registers.  M = 8192, D = 4096, bf16: 48 us, 85 % of the measured
// copy bandwidth (the two barriers of a row leave the rest).
template <bool kBf16, int kV>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_ring_kernel(const NormArgs a, const int T, const int groups,
                                                                          const int stages, const int64_t rows,
                                                                          const int longer) {
    using E = Vec<kBf16>;
    constexpr int kE = E::kE, kP = kE / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float slots[8][2 * 16];
    __shared__ __align__(8) unsigned long long bars[kMaxGroups * kMaxRing];
    __shared__ int abort_flag;
    const int grp = threadIdx.x / T, tid = threadIdx.x - grp * T;
    const int nvec = a.D / kE;
    const uint32_t row_bytes = 16u * nvec;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // a stage: Y, R, each `pitch` bytes, of which the copies fill the first
    // row_bytes; the rest is zero from here on
    const uint32_t pitch = 16u * kV * T;
    const uint32_t ring = smem_u32(smem) + grp * stages * 2u * pitch;
    const uint32_t full = smem_u32(bars) + 8u * (grp * kMaxRing);
    if (nvec < kV * T)
        for (int i = tid; i < stages * 2 * kV * T; i += T) sts_v4(ring + 16u * i, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(full + 8 * i, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x;   // `rows` rows each, the first `longer` blocks one more
    const int64_t row0 = b * rows + min(b, longer) + grp, row1 = (b + 1) * rows + min(b + 1, longer);
    auto copy_row = [&](int64_t row, int to) {
        const uint32_t fb = full + 8 * to, st = ring + to * 2u * pitch;
        mbar_arrive_expect_tx(fb, 2u * row_bytes);
        bulk_load(st, a.Y + row * nvec, row_bytes, fb);
        bulk_load(st + pitch, a.R + row * nvec, row_bytes, fb);
    };
    if (tid == 0)
        for (int i = 0; i < stages && row0 + i * groups < row1; ++i) copy_row(row0 + i * groups, i);

    int turn = 0, stage = 0;
    uint32_t phase = 0;
    bool failed = false;
    f2 hold_g[kV][kP], hold_w[kV][kP];
    auto fetch_g = [&](int v, const uint4 *gate, f2 (&o)[kP]) {
        const int c = v * T + tid;
#pragma unroll
        for (int i = 0; i < kP; ++i) o[i] = pack2(1.0f, 1.0f);
        if (c >= nvec) return;
        if (a.w1) E::unpack2(ld_plain(a.w1 + c), o);
        if (gate) {
            f2 f[kP];
            E::unpack2(ld_plain(gate + c), f);
#pragma unroll
            for (int i = 0; i < kP; ++i) o[i] = mul2(o[i], f[i]);
        }
    };
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int c = v * T + tid;
        E::unpack2(a.w2 && c < nvec ? ld_plain(a.w2 + c) : make_uint4(0, 0, 0, 0), hold_w[v]);
    }
    int64_t gate_end = row0;        // first row of the next gate row
    const uint4 *gate = nullptr;
    for (int64_t row = row0; row < row1; row += groups) {
        if (row >= gate_end) {
            const int64_t gr = row / a.rows_per_gate;
            gate_end = (gr + 1) * a.rows_per_gate;
            gate = a.gate ? a.gate + gr * nvec : nullptr;
#pragma unroll
            for (int v = 0; v < kV; ++v) fetch_g(v, gate, hold_g[v]);
        }
        // (a wait that gave up is recorded; the rows that follow are worked
        // on all the same, so that the group's barriers match)
        if (!failed && !mbar_wait(full + 8 * stage, phase, &abort_flag)) {
            failed = true;
            if (tid == 0) ring_abandon(full, stages, stage, phase);
        }
        const uint32_t st = ring + stage * 2u * pitch + 16u * tid;
        f2 y[kV][kP];
#pragma unroll
        for (int v = 0; v < kV; ++v) E::unpack2(lds_v4(st + 16u * v * T), y[v]);
        auto refill = [&]() {   // the whole group is done with the row before this one
            const int64_t next = row + static_cast<int64_t>(stages - 1) * groups;
            if (tid == 0 && row > row0 && next < row1 && !failed) copy_row(next, stage > 0 ? stage - 1 : stages - 1);
        };
        float r1 = 1.0f;
        if (a.w1) {
            f2 q = 0ull;
#pragma unroll
            for (int v = 0; v < kV; ++v)
#pragma unroll
                for (int i = 0; i < kP; ++i) q = fma2(y[v][i], y[v][i], q);
            float s[1] = {lo2(q) + hi2(q)};
            row_sum<1>(s, slots[grp & 7], turn, grp, tid, T);
            r1 = 1.0f / sqrtf(s[0] * inv_d + a.eps);
            if (a.rstd1 && tid == 0) a.rstd1[row] = r1;
        } else if (!a.w2) {
            if (T > 32) row_barrier(grp, T);
            else __syncwarp();
        }
        const f2 sr1 = pack2(a.scale * r1, a.scale * r1);
        uint4 *Rn = a.Rn + row * nvec + tid, *N = a.N + row * nvec + tid;
        f2 q = 0ull;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            f2 r[kP];
            E::unpack2(lds_v4(st + pitch + 16u * v * T), r);
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                y[v][i] = fma2(sr1, mul2(y[v][i], hold_g[v][i]), r[i]);
                q = fma2(y[v][i], y[v][i], q);
            }
            if (v * T + tid < nvec) st_stream_v4(Rn + v * T, E::pack_pairs(y[v]));
        }
        if (a.w2) {
            float s[1] = {lo2(q) + hi2(q)};
            row_sum<1>(s, slots[grp & 7], turn, grp, tid, T);
            const float r2 = 1.0f / sqrtf(s[0] * inv_d + a.eps);
            if (a.rstd2 && tid == 0) a.rstd2[row] = r2;
            refill();
            const f2 r22 = pack2(r2, r2);
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                f2 w[kP];
#pragma unroll
                for (int i = 0; i < kP; ++i) w[i] = mul2(hold_w[v][i], mul2(y[v][i], r22));
                if (v * T + tid < nvec) st_stream_v4(N + v * T, E::pack_pairs(w));
            }
        } else {
            refill();
        }
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (failed) atomicOr(&g_block_norm_status, 1u);
}

// ------------------------------------------------------------- backward

struct NormBwdArgs {
    const uint4 *dRn, *dN, *Y, *Rn;  // dRn null: zero; dN null with w2
    const float *rstd1, *rstd2;
    const uint4 *w1, *w2, *gate;
    uint4 *dY, *dR, *dgate;          // dgate: written here when a gate row has one item
    float *acc2, *acc1, *accg;       // workspaces: [blocks][D], [blocks][D], [items][D]
    int64_t rows_per_gate;           // rows of one gate row (all of them without per-row gates)
    int64_t gates;                   // gate rows (1 without)
    int splits;                      // blocks that share a gate row's rows:
    int64_t rows_per_item;           // so many each,
    int longer;                      // and the first ones one more
    int D;
    int T, groups;                   // threads per row, rows at a time
    int stages;                      // rows of a group's ring
    float scale;
};

// Block b takes items b, b + grid, ...; item = (gate row, split): a run of
// consecutive rows that share their gate row, `groups` of them at a time.
// Column sums stay in registers and leave once per block: acc2 = sum dN n;
// acc1 = sum dX y, or with gate rows sum s g dX y and, where a gate row has
// more than one item, accg = the item's sum dX y.
// What is kept between the two passes over a row: with 16 elements a thread or
// fewer, e and the products of the weights (in registers); with more they are
// formed again, because the column sums alone fill half the registers.
// D = 4096, bf16, with the join: 7.6 ns per row (six rows of HBM at 6.5 TB/s)
// and some 12 us at any M: the rings' fill, the column sums' way out and the
// join, which launched by itself takes 5.4 us.  M = 16384 136 us, 91 % of the
// measured copy bandwidth; M = 2048 28.4 us, 54 %.  One CTA-wide loop over rows
// read straight from memory took 234 and 45 us: its loads waited for its
// barriers.
template <bool kBf16, int kV, bool kGates>
__global__ void __launch_bounds__(kRingThreads, 1) block_norm_bwd_kernel(const NormBwdArgs a) {
    using E = Vec<kBf16>;
    constexpr int kE = E::kE;
    constexpr bool kHold = kV * kE <= 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float slots[8][2 * 3 * 16];
    __shared__ __align__(8) unsigned long long bars[kMaxGroups * kMaxRing];
    __shared__ int abort_flag;
    const int T = a.T, groups = a.groups, stages = a.stages;
    const int grp = threadIdx.x / T, tid = threadIdx.x - grp * T;
    const int nvec = a.D / kE;
    const uint32_t row_bytes = 16u * nvec;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // a stage: dRn, dN, Y, Rn, each `pitch` bytes, of which the copies fill
    // the first row_bytes; what they never fill (the rest, and operands that
    // are not there) is zero from here on
    const uint32_t pitch = 16u * kV * T;
    const uint32_t ring = smem_u32(smem) + grp * stages * 4u * pitch;
    if (nvec < kV * T || !a.dRn || !a.w2)
        for (int i = tid; i < stages * 4 * kV * T; i += T) sts_v4(ring + 16u * i, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    const uint32_t full = smem_u32(bars) + 8u * (grp * kMaxRing);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(full + 8 * i, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    griddep_wait();
    const int64_t items = a.gates * a.splits;
    // (items fit 32 bits; the first copy waits for this)
    auto gate_of = [&](int64_t item) -> int64_t {
        return kGates ? static_cast<uint32_t>(item) / static_cast<uint32_t>(a.splits) : 0u;
    };
    auto rows_of = [&](int64_t item, int64_t &row0, int64_t &row1) {
        const int64_t gr = gate_of(item), sp = item - gr * a.splits;
        row0 = gr * a.rows_per_gate + sp * a.rows_per_item + (sp < a.longer ? sp : a.longer);
        row1 = row0 + a.rows_per_item + (sp < a.longer ? 1 : 0);
    };

    auto copy_row = [&](int64_t row, int to) {
        const uint32_t fb = full + 8 * to, st = ring + to * 4u * pitch;
        mbar_arrive_expect_tx(fb, row_bytes * (1u + (a.dRn ? 1u : 0u) + (a.w2 ? 2u : 0u)));
        const int64_t o = row * nvec;
        if (a.dRn) bulk_load(st, a.dRn + o, row_bytes, fb);
        if (a.w2) bulk_load(st + pitch, a.dN + o, row_bytes, fb);
        bulk_load(st + 2 * pitch, a.Y + o, row_bytes, fb);
        if (a.w2) bulk_load(st + 3 * pitch, a.Rn + o, row_bytes, fb);
    };
    // The group's first thread copies a ring ahead of the row it works on.
    // Without gate rows a block has one item, and the row to copy follows from
    // the row at hand; with them the copies go on into the block's next items.
    int64_t next_item = blockIdx.x, next_row = 0, next_end = 0;
    int put = 0;
    auto copy_next = [&]() {
        while (next_row >= next_end && next_item < items) {
            rows_of(next_item, next_row, next_end);
            next_row += grp;
            next_item += gridDim.x;
        }
        if (next_row >= next_end) return;
        copy_row(next_row, put);
        if (++put == stages) put = 0;
        next_row += groups;
    };
    if (tid == 0)
        for (int i = 0; i < stages; ++i) copy_next();
    int stage = 0;
    uint32_t phase = 0;
    bool failed = false, first = true;

    int turn = 0;
    constexpr int kP = kE / 2;
    // Column sums of this thread's rows: dN n, and dX y (with gate rows, those
    // of the item at hand).  With gate rows sum1[D] gathers the block's
    // sum s g dX y in shared memory, and shares[groups][D] is where the
    // groups' dX y of an item meet.
    f2 s2[kV][kP], sb[kV][kP];
    float *sum1 = reinterpret_cast<float *>(smem + stages * groups * 4u * pitch), *shares = sum1 + a.D;
    const float4 ones = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (kGates) {
        for (int col = threadIdx.x; col < a.D; col += T * groups) sum1[col] = 0.0f;
        block_barrier(T * groups);
    }
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < kP; ++i) s2[v][i] = sb[v][i] = 0ull;

    // s g W1 and W2 of vector v, from memory
    auto fetch_g = [&](int v, const uint4 *gate, f2 (&o)[kP]) {
        const int c = v * T + tid;
#pragma unroll
        for (int i = 0; i < kP; ++i) o[i] = pack2(a.scale, a.scale);
        if (c >= nvec) return;
        f2 f[kP];
        if (a.w1) {
            E::unpack2(ld_plain(a.w1 + c), f);
#pragma unroll
            for (int i = 0; i < kP; ++i) o[i] = mul2(o[i], f[i]);
        }
        if (gate) {
            E::unpack2(ld_plain(gate + c), f);
#pragma unroll
            for (int i = 0; i < kP; ++i) o[i] = mul2(o[i], f[i]);
        }
    };
    auto fetch_w = [&](int v) {
        const int c = v * T + tid;
        return a.w2 && c < nvec ? ld_plain(a.w2 + c) : make_uint4(0, 0, 0, 0);
    };
    f2 hold_g[kHold ? kV : 1][kP];
    f2 hold_w[kHold ? kV : 1][kP];

    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        int64_t row0, row1;
        rows_of(item, row0, row1);
        const int64_t gr = gate_of(item);
        const uint4 *gate = a.gate ? a.gate + gr * nvec : nullptr;
        if constexpr (kHold) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                fetch_g(v, gate, hold_g[v]);
                E::unpack2(fetch_w(v), hold_w[v]);
            }
        }
        auto get_g = [&](int v, f2 (&o)[kP]) {
            if constexpr (kHold) {
#pragma unroll
                for (int i = 0; i < kP; ++i) o[i] = hold_g[v][i];
            } else {
                fetch_g(v, gate, o);
            }
        };
        auto get_w = [&](int v, f2 (&o)[kP]) {
            if constexpr (kHold) {
#pragma unroll
                for (int i = 0; i < kP; ++i) o[i] = hold_w[v][i];
            } else {
                E::unpack2(fetch_w(v), o);
            }
        };
        // a row's statistics are fetched a row ahead
        float r1n = 1.0f, r2n = 0.0f;
        auto stats = [&](int64_t row) {
            if (row >= row1) return;
            if (a.w1) r1n = ld_plain(a.rstd1 + row);
            if (a.w2) r2n = ld_plain(a.rstd2 + row);
        };
        stats(row0 + grp);
        for (int64_t row = row0 + grp; row < row1; row += groups) {
            const float r1 = r1n, r2 = r2n;
            stats(row + groups);
            // (a wait that gave up is recorded; the rows that follow are
            // worked on all the same, so that the group's barriers match)
            if (!failed && !mbar_wait(full + 8 * stage, phase, &abort_flag)) {
                failed = true;
                if (tid == 0) ring_abandon(full, stages, stage, phase);
            }
            const uint32_t st = ring + stage * 4u * pitch + 16u * tid;
            auto load = [&](int which, int v, f2 (&f)[kP]) { E::unpack2(lds_v4(st + which * pitch + 16u * v * T), f); };
            // With R, Y unscaled: sums of a R, (s g W1 Y) e and (s g W1 Y) R,
            // e = dR' + r2 a kept for the second pass
            f2 e[kHold ? kV : 1][kP];
            f2 q0 = 0ull, q1 = 0ull, q2 = 0ull;
            const f2 r22 = pack2(r2, r2);
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                f2 n[kP], y[kP], r[kP], w[kP], g[kP];
                f2 (&ev)[kP] = e[kHold ? v : 0];
                load(0, v, ev);
                load(1, v, n);
                load(2, v, y);
                load(3, v, r);
                get_w(v, w);
                get_g(v, g);
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    const f2 nr = mul2(n[i], r[i]);
                    q0 = fma2(w[i], nr, q0);
                    s2[v][i] = fma2(nr, r22, s2[v][i]);
                    ev[i] = fma2(r22, mul2(w[i], n[i]), ev[i]);
                    const f2 t = mul2(g[i], y[i]);
                    q1 = fma2(t, ev[i], q1);
                    q2 = fma2(t, r[i], q2);
                }
            }
            float s[3] = {lo2(q0) + hi2(q0), lo2(q1) + hi2(q1), lo2(q2) + hi2(q2)};
            row_sum<3>(s, slots[grp & 7], turn, grp, tid, T);   // (one warp: no slots)
            __syncwarp();
            // the whole group is done with the row before this one
            if (kGates) {
                if (tid == 0 && !first && stages > 1 && !failed) copy_next();
                first = false;
            } else {
                const int64_t next = row + static_cast<int64_t>(stages - 1) * groups;
                if (tid == 0 && row >= row0 + groups && stages > 1 && next < row1 && !failed)
                    copy_row(next, stage > 0 ? stage - 1 : stages - 1);
            }
            const float k2 = r2 * (r2 * s[0] * inv_d);                  // r2 mean(a n)
            const float c1 = r1 * (s[1] - k2 * r2 * s[2]) * inv_d;      // mean(b y)
            const f2 kr = pack2(-k2 * r2, -k2 * r2), r12 = pack2(r1, r1);
            const f2 ky = pack2(-c1, -c1);
            uint4 *dR = a.dR + row * nvec + tid, *dY = a.dY + row * nvec + tid;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                f2 y[kP], r[kP], g[kP], dy[kP];
                f2 (&ev)[kP] = e[kHold ? v : 0];
                load(2, v, y);
                load(3, v, r);
                get_g(v, g);
                if constexpr (!kHold) {
                    f2 n[kP], w[kP];
                    load(0, v, ev);
                    load(1, v, n);
                    get_w(v, w);
#pragma unroll
                    for (int i = 0; i < kP; ++i) ev[i] = fma2(r22, mul2(w[i], n[i]), ev[i]);
                }
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    ev[i] = fma2(kr, r[i], ev[i]);
                    const f2 yh = mul2(y[i], r12);
                    sb[v][i] = fma2(ev[i], yh, sb[v][i]);
                    dy[i] = mul2(ev[i], g[i]);
                    if (a.w1) dy[i] = mul2(r12, fma2(ky, yh, dy[i]));
                }
                if (v * T + tid < nvec) {
                    st_stream_v4(dR + v * T, E::pack_pairs(ev));
                    st_stream_v4(dY + v * T, E::pack_pairs(dy));
                }
            }
            if (stages == 1) {
                if (T > 32) row_barrier(grp, T);
                else __syncwarp();
                if (kGates) {
                    if (tid == 0 && !failed) copy_next();
                } else if (tid == 0 && row + groups < row1 && !failed) {
                    copy_row(row + groups, 0);
                }
            }
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if constexpr (kGates) {
            // the item's sum dX y: the row groups' shares meet, in order
            auto finish = [&](int col, float4 x) {
                const float4 g = E::load4(a.gate, gr * a.D + col), w = a.w1 ? E::load4(a.w1, col) : ones;
                const float4 sx = make_float4(a.scale * x.x, a.scale * x.y, a.scale * x.z, a.scale * x.w);
                if (a.splits == 1)
                    E::store4(a.dgate, gr * a.D + col, make_float4(w.x * sx.x, w.y * sx.y, w.z * sx.z, w.w * sx.w));
                else
                    *reinterpret_cast<float4 *>(a.accg + item * a.D + col) = x;
                float4 *to = reinterpret_cast<float4 *>(sum1 + col);
                const float4 o = *to;
                *to = make_float4(fmaf(g.x, sx.x, o.x), fmaf(g.y, sx.y, o.y), fmaf(g.z, sx.z, o.z),
                                  fmaf(g.w, sx.w, o.w));
            };
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
#pragma unroll
                for (int i = 0; i < kP; i += 2) {
                    const float4 x = make_float4(lo2(sb[v][i]), hi2(sb[v][i]), lo2(sb[v][i + 1]), hi2(sb[v][i + 1]));
                    sb[v][i] = sb[v][i + 1] = 0ull;
                    if (c >= nvec) continue;
                    if (groups > 1) *reinterpret_cast<float4 *>(shares + grp * a.D + c * kE + 2 * i) = x;
                    else finish(c * kE + 2 * i, x);
                }
            }
            if (groups > 1) {
                block_barrier(T * groups);
                for (int col = 4 * threadIdx.x; col < a.D; col += 4 * T * groups) {
                    float4 x = *reinterpret_cast<const float4 *>(shares + col);
                    for (int k = 1; k < groups; ++k) {
                        const float4 y = *reinterpret_cast<const float4 *>(shares + k * a.D + col);
                        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                    }
                    finish(col, x);
                }
                block_barrier(T * groups);
            }
        }
    }
    griddep_launch_dependents();
    // The row groups' column sums meet in shared memory (the ring is empty:
    // every row has been read), group by group in order.
    float *meet = reinterpret_cast<float *>(smem);
    if (groups > 1 || kGates) block_barrier(T * groups);
    if (groups > 1) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int c = v * T + tid;
            if (grp > 0 && c < nvec) {
#pragma unroll
                for (int i = 0; i < kP; i += 2) {
                    const int o = (grp - 1) * 2 * a.D + c * kE + 2 * i;
                    *reinterpret_cast<float4 *>(meet + o) =
                        make_float4(lo2(s2[v][i]), hi2(s2[v][i]), lo2(s2[v][i + 1]), hi2(s2[v][i + 1]));
                    if (!kGates)
                        *reinterpret_cast<float4 *>(meet + o + a.D) =
                            make_float4(lo2(sb[v][i]), hi2(sb[v][i]), lo2(sb[v][i + 1]), hi2(sb[v][i + 1]));
                }
            }
        }
        block_barrier(T * groups);
    }
    if (failed) atomicOr(&g_block_norm_status, 1u);
    if (grp > 0) return;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int c = v * T + tid;
        if (c < nvec) {
#pragma unroll
            for (int i = 0; i < kP; i += 2) {
                float4 x = make_float4(lo2(s2[v][i]), hi2(s2[v][i]), lo2(s2[v][i + 1]), hi2(s2[v][i + 1]));
                float4 z = make_float4(lo2(sb[v][i]), hi2(sb[v][i]), lo2(sb[v][i + 1]), hi2(sb[v][i + 1]));
                for (int g = 0; g + 1 < groups; ++g) {
                    const float *m = meet + g * 2 * a.D + c * kE + 2 * i;
                    const float4 p = *reinterpret_cast<const float4 *>(m);
                    x = make_float4(x.x + p.x, x.y + p.y, x.z + p.z, x.w + p.w);
                    if (!kGates) {
                        const float4 q = *reinterpret_cast<const float4 *>(m + a.D);
                        z = make_float4(z.x + q.x, z.y + q.y, z.z + q.z, z.w + q.w);
                    }
                }
                if (kGates) z = *reinterpret_cast<const float4 *>(sum1 + c * kE + 2 * i);
                const int64_t o = static_cast<int64_t>(blockIdx.x) * a.D + static_cast<int64_t>(c) * kE + 2 * i;
                if (a.acc2) *reinterpret_cast<float4 *>(a.acc2 + o) = x;
                if (a.acc1) *reinterpret_cast<float4 *>(a.acc1 + o) = z;
            }
        }
    }
}

struct NormReduceArgs {
    const float *acc2, *acc1, *accg;
    const void *w1, *gate;
    void *dw2, *dw1, *dgate;   // null: not wanted here
    int64_t workers;           // blocks of the main kernel
    int splits;                // sums per gate row
    int64_t gates;             // gate rows
    int D;
    int per_row;               // per-row gates: acc1 holds dW1 itself, accg the gate rows' sums
    float scale;
};

constexpr int kReduceRows = 32;

// Joins the workers' column sums, in a fixed order: blockIdx.y = 0 the
// weights (and the single gate row), the others kReduceRows gate rows each.
template <bool kBf16>
__global__ void __launch_bounds__(32 * kReduceRows) block_norm_reduce_kernel(const NormReduceArgs a) {
    __shared__ float part[2][kReduceRows][33];
    const int col = blockIdx.x * 32 + threadIdx.x;
    const int ty = threadIdx.y;
    auto load = [&](const void *p, int64_t i) {
        return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                     : static_cast<const float *>(p)[i];
    };
    auto store = [&](void *p, int64_t i, float x) {
        if (kBf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
        else static_cast<float *>(p)[i] = x;
    };
    float v0 = 0.0f, v1 = 0.0f;
    griddep_launch_dependents();
    griddep_wait();
    // (a batch's loads are in flight together)
    constexpr int kBatch = 5;
    if (blockIdx.y > 0) {   // a gate row per row of threads
        const int64_t gr = static_cast<int64_t>(blockIdx.y - 1) * kReduceRows + ty;
        if (gr >= a.gates || col >= a.D) return;
        const float *from = a.accg + gr * a.splits * a.D + col;
        for (int i0 = 0; i0 < a.splits; i0 += kBatch) {
            float x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) x[j] = i0 + j < a.splits ? from[static_cast<int64_t>(i0 + j) * a.D] : 0.0f;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) v0 += x[j];
        }
        store(a.dgate, gr * a.D + col, a.scale * (a.w1 ? load(a.w1, col) : 1.0f) * v0);
        return;
    }
    if (col < a.D) {
        for (int64_t i0 = ty; i0 < a.workers; i0 += kReduceRows * kBatch) {
            float x[kBatch], z[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t i = i0 + j * kReduceRows;
                x[j] = a.acc2 && i < a.workers ? a.acc2[i * a.D + col] : 0.0f;
                z[j] = a.acc1 && i < a.workers ? a.acc1[i * a.D + col] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                v0 += x[j];
                v1 += z[j];
            }
        }
    }
    part[0][ty][threadIdx.x] = v0;
    part[1][ty][threadIdx.x] = v1;
    __syncthreads();
    if (ty != 0 || col >= a.D) return;
    v0 = v1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kReduceRows; ++i) {
        v0 += part[0][i][threadIdx.x];
        v1 += part[1][i][threadIdx.x];
    }
    const float w = a.w1 ? load(a.w1, col) : 1.0f;
    if (a.dw2) store(a.dw2, col, v0);
    if (a.dw1) {
        const float g = a.per_row ? 1.0f : a.scale * (a.gate ? load(a.gate, col) : 1.0f);
        store(a.dw1, col, g * v1);
    }
    if (a.dgate && !a.per_row) store(a.dgate, col, a.scale * w * v1);
}

// Row layout: kV vectors per thread, T threads (whole warps) per row and as
// many row groups as fill kBlockThreads.
struct RowShape {
    int v, T, groups;
};

RowShape row_shape(int nvec) {
    RowShape s{};
    s.v = nvec <= 256 ? 1 : (nvec <= 1024 ? 2 : 4);
    s.T = (((nvec + s.v - 1) / s.v) + 31) / 32 * 32;
    s.groups = s.T >= kBlockThreads ? 1 : kBlockThreads / s.T;
    if (s.groups > 8) s.groups = 8;
    return s;
}

// Ring kernels: 16 elements per thread (backward: 8 for rows of up to 1024,
// M = 2368, D = 1024 12.1 against 12.8 us; 32 for bf16 rows of more than 8192),
// whole warps per row, row groups up to kRingThreads.
struct RingShape {
    int v, T, groups;
};

RingShape ring_shape(int D, int f32, bool backward) {
    RingShape s{};
    const int nvec = D / (f32 ? 4 : 8), two = f32 ? 4 : 2;   // vectors of 16 elements
    s.v = backward && nvec <= 64 * two ? two / 2 : (nvec <= 512 * two ? two : 4);
    s.T = (((nvec + s.v - 1) / s.v) + 31) / 32 * 32;
    s.groups = kRingThreads / s.T;
    if (s.groups > kMaxGroups) s.groups = kMaxGroups;   // (T = 32; with more threads it is 8 or fewer)
    return s;
}

// Once per kernel and device: opt in to the ring's shared memory.
template <typename Kernel>
cudaError_t opt_in(Kernel kernel, std::atomic<unsigned> &mask, const DeviceInfo &dev) {
    const unsigned bit = 1u << (dev.device & 31);
    if (mask.load() & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingRoom));
    if (e == cudaSuccess) mask.fetch_or(bit);
    return e;
}

struct BwdPlan {
    int v, T, groups, stages;
    uint32_t smem;
    int64_t splits, blocks;
    size_t bytes;
};

// One block per SM: as many row groups as its threads hold (their column sums
// meet in the block, so a block costs 8 D bytes of sums written and read
// again, however many rows it takes at a time), rings over all of its shared
// memory.  At least `groups` rows per block.
BwdPlan bwd_plan(int64_t M, int D, int f32, bool per_row, int64_t gates, bool w1, bool w2, bool gate,
                 int sm_count) {
    BwdPlan p{};
    const RingShape sh = ring_shape(D, f32, true);
    p.v = sh.v;
    p.T = sh.T;
    p.groups = sh.groups;
    constexpr uint32_t kRoom = kRingRoom;
    const uint32_t row = 4u * 16u * p.v * p.T;   // (operands are padded to whole warps)
    const int64_t rows_per_gate = per_row ? M / gates : M;
    auto sums = [&]() { return per_row ? 4u * D * (1u + (p.groups > 1 ? p.groups : 0u)) : 0u; };
    while (p.groups > 1 && (p.groups * row * 2u + sums() > kRoom || p.groups > rows_per_gate)) --p.groups;
    p.stages = static_cast<int>((kRoom - sums()) / (row * p.groups));
    if (p.stages > kMaxRing) p.stages = kMaxRing;
    p.smem = p.stages * row * p.groups + sums();
    const int64_t most = (rows_per_gate + p.groups - 1) / p.groups;
    p.splits = per_row ? sm_count / gates : sm_count;
    if (p.splits > most) p.splits = most;
    if (p.splits < 1) p.splits = 1;
    const int64_t items = (per_row ? gates : 1) * p.splits;
    p.blocks = items < sm_count ? items : sm_count;
    size_t floats = 0;
    if (w2) floats += static_cast<size_t>(p.blocks) * D;
    if (w1 || (gate && !per_row)) floats += static_cast<size_t>(p.blocks) * D;
    if (per_row && p.splits > 1) floats += static_cast<size_t>(items) * D;
    p.bytes = floats * 4;
    return p;
}

template <bool kBf16, int kV>
cudaError_t launch_fwd_ring(const NormArgs &a, const RingShape &s, const DeviceInfo &dev, cudaStream_t stream) {
    static std::atomic<unsigned> mask{0};
    auto kernel = block_norm_ring_kernel<kBf16, kV>;
    const cudaError_t e = opt_in(kernel, mask, dev);
    if (e != cudaSuccess) return e;
    const uint32_t row = 2u * 16u * s.v * s.T;
    int stages = static_cast<int>(kRingRoom / (row * s.groups));
    if (stages > kMaxRing) stages = kMaxRing;
    return launch_dependent(kernel, dev.sm_count, s.T * s.groups, stages * row * s.groups, stream, a, s.T, s.groups,
                            stages, a.M / dev.sm_count, static_cast<int>(a.M % dev.sm_count));
}

template <bool kBf16, int kV>
cudaError_t launch_fwd_v(const NormArgs &a, const RowShape &s, int sm_count, cudaStream_t stream) {
    int64_t blocks = (a.M + s.groups - 1) / s.groups;
    const int64_t most = static_cast<int64_t>(sm_count) * (2048 / (s.T * s.groups));
    if (blocks > most) blocks = most;
    return launch_dependent(block_norm_kernel<kBf16, kV>, static_cast<unsigned>(blocks), dim3(s.T, s.groups), 0, stream,
                            a);
}

template <bool kBf16>
cudaError_t launch_fwd(const NormArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    const RingShape r = ring_shape(a.D, !kBf16, false);
    const int nvec = a.D / Vec<kBf16>::kE;
    // Rings for rows of 1 KB up to what holds its weights in registers, from
    // two rows per row group on (four where two or fewer groups share a block).
    // Ring against plain, B200, us: 8192 x 4096 bf16 48.2 against 52.8, 16384 x
    // 2048 49.0 and 70.1, 16384 x 512 15.7 and 17.9, 777 x 5120 fp32 11.6 and
    // 17.0; at the limits 4736 x 512 5.1 and 5.6, 2368 x 1024 5.7 and 5.8, 1184 x
    // 4096 9.1 and 9.1; outside, 592 x 4096 5.6 and 4.6, 18944 x 256 10.9 and
    // 9.6, 2048 x 16384 75 and 67.
    if (nvec >= 64 && r.v * Vec<kBf16>::kE <= 16 &&
        a.M >= (r.groups >= 4 ? 2 : 4) * static_cast<int64_t>(dev.sm_count) * r.groups)
        return launch_fwd_ring<kBf16, kBf16 ? 2 : 4>(a, r, dev, stream);
    const RowShape s = row_shape(nvec);
    switch (s.v) {
        case 1: return launch_fwd_v<kBf16, 1>(a, s, dev.sm_count, stream);
        case 2: return launch_fwd_v<kBf16, 2>(a, s, dev.sm_count, stream);
        default: return launch_fwd_v<kBf16, 4>(a, s, dev.sm_count, stream);
    }
}

template <bool kBf16, int kV, bool kGates>
cudaError_t launch_bwd_v(const NormBwdArgs &a, const BwdPlan &p, const DeviceInfo &dev, cudaStream_t stream) {
    static std::atomic<unsigned> mask{0};
    auto kernel = block_norm_bwd_kernel<kBf16, kV, kGates>;
    const cudaError_t e = opt_in(kernel, mask, dev);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, static_cast<unsigned>(p.blocks), p.T * p.groups, p.smem, stream, a);
}

template <bool kGates>
cudaError_t launch_bwd(int f32, const NormBwdArgs &a, const BwdPlan &p, const DeviceInfo &dev, cudaStream_t stream) {
    if (f32)
        return p.v == 2 ? launch_bwd_v<false, 2, kGates>(a, p, dev, stream)
                        : launch_bwd_v<false, 4, kGates>(a, p, dev, stream);
    switch (p.v) {
        case 1: return launch_bwd_v<true, 1, kGates>(a, p, dev, stream);
        case 2: return launch_bwd_v<true, 2, kGates>(a, p, dev, stream);
        default: return launch_bwd_v<true, 4, kGates>(a, p, dev, stream);
    }
}

}  // namespace

cudaError_t launch_block_norm(const void *Y, const void *R, const BlockNorm &n, void *Rn, void *N,
                              float *rstd1, float *rstd2, int64_t M, int D, int f32,
                              const DeviceInfo &dev, cudaStream_t stream) {
    NormArgs a{};
    a.Y = static_cast<const uint4 *>(Y);
    a.R = static_cast<const uint4 *>(R);
    a.w1 = static_cast<const uint4 *>(n.w1);
    a.w2 = static_cast<const uint4 *>(n.w2);
    a.gate = static_cast<const uint4 *>(n.gate);
    a.Rn = static_cast<uint4 *>(Rn);
    a.N = static_cast<uint4 *>(N);
    a.rstd1 = rstd1;
    a.rstd2 = rstd2;
    a.M = M;
    a.rows_per_gate = n.gate ? M / n.gate_rows : M;
    a.D = D;
    a.scale = n.scale;
    a.eps = n.eps;
    return f32 ? launch_fwd<false>(a, dev, stream) : launch_fwd<true>(a, dev, stream);
}

size_t block_norm_bwd_workspace(int64_t M, int D, int f32, const BlockNorm &n, int sm_count) {
    const bool per_row = n.gate && n.gate_rows > 1;
    return bwd_plan(M, D, f32, per_row, per_row ? n.gate_rows : 1, n.w1, n.w2, n.gate, sm_count).bytes;
}

cudaError_t launch_block_norm_bwd(const void *dRn, const void *dN, const void *Y, const void *Rn,
                                  const float *rstd1, const float *rstd2, const BlockNorm &n,
                                  void *dY, void *dR, void *dw1, void *dw2, void *dgate,
                                  void *workspace, int64_t M, int D, int f32,
                                  const DeviceInfo &dev, cudaStream_t stream) {
    const bool per_row = n.gate && n.gate_rows > 1;
    const int64_t gates = per_row ? n.gate_rows : 1;
    const BwdPlan p = bwd_plan(M, D, f32, per_row, gates, n.w1, n.w2, n.gate, dev.sm_count);
    float *ws = static_cast<float *>(workspace);
    NormBwdArgs a{};
    a.dRn = static_cast<const uint4 *>(dRn);
    a.dN = static_cast<const uint4 *>(dN);
    a.Y = static_cast<const uint4 *>(Y);
    a.Rn = static_cast<const uint4 *>(Rn);
    a.rstd1 = rstd1;
    a.rstd2 = rstd2;
    a.w1 = static_cast<const uint4 *>(n.w1);
    a.w2 = static_cast<const uint4 *>(n.w2);
    a.gate = static_cast<const uint4 *>(n.gate);
    a.dY = static_cast<uint4 *>(dY);
    a.dR = static_cast<uint4 *>(dR);
    a.dgate = static_cast<uint4 *>(dgate);
    const size_t per = static_cast<size_t>(p.blocks) * D;
    if (n.w2) {
        a.acc2 = ws;
        ws += per;
    }
    if (n.w1 || (n.gate && !per_row)) {
        a.acc1 = ws;
        ws += per;
    }
    if (per_row && p.splits > 1) a.accg = ws;
    a.rows_per_gate = per_row ? M / gates : M;
    a.gates = gates;
    a.splits = static_cast<int>(p.splits);
    a.rows_per_item = a.rows_per_gate / p.splits;
    a.longer = static_cast<int>(a.rows_per_gate % p.splits);
    a.D = D;
    a.T = p.T;
    a.groups = p.groups;
    a.scale = n.scale;
    a.stages = p.stages;
    cudaError_t e = per_row ? launch_bwd<true>(f32, a, p, dev, stream) : launch_bwd<false>(f32, a, p, dev, stream);
    if (e != cudaSuccess || !(a.acc2 || a.acc1 || a.accg)) return e;
    NormReduceArgs r{};
    r.acc2 = a.acc2;
    r.acc1 = a.acc1;
    r.accg = a.accg;
    r.w1 = n.w1;
    r.gate = n.gate;
    r.dw2 = n.w2 ? dw2 : nullptr;
    r.dw1 = n.w1 ? dw1 : nullptr;
    r.dgate = n.gate ? dgate : nullptr;
    r.workers = p.blocks;
    r.splits = static_cast<int>(p.splits);
    r.gates = gates;
    r.D = D;
    r.per_row = per_row ? 1 : 0;
    r.scale = n.scale;
    const dim3 grid((D + 31) / 32, static_cast<unsigned>(1 + (a.accg ? (gates + kReduceRows - 1) / kReduceRows : 0)));
    const dim3 block(32, kReduceRows);
    return f32 ? launch_dependent(block_norm_reduce_kernel<false>, grid, block, 0, stream, r)
               : launch_dependent(block_norm_reduce_kernel<true>, grid, block, 0, stream, r);
}

cudaError_t block_norm_status_fetch_and_clear(unsigned int *host_out, cudaStream_t stream) {
    return fetch_and_clear(g_block_norm_status, host_out, stream);
}

}  // namespace swiglu
