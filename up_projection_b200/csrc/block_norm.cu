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

#include "kernels.cuh"
#include "ptx.cuh"

namespace swiglu {
namespace {

using namespace dev;

constexpr int kRowThreadsMax = 512;
constexpr int kBlockThreads = 256;  // row groups fill a block up to this

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

// Sum of K values over the T = 32 * warps threads of a row group.  `slots`
// is the group's shared memory, two sets of K * 16 floats used in turn, so
// one barrier per reduction is enough: a set is rewritten only after the
// barrier of the next reduction, which every reader of this one has reached.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *slots, int &turn, int group,
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
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
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
            row_sum<1>(s, slots[grp], turn, grp, T);
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
                if (a.w1) {
                    float w[kE];
                    E::unpack(__ldg(a.w1 + c), w);
#pragma unroll
                    for (int i = 0; i < kE; ++i) f[i] *= w[i];
                }
                if (gate) {
                    float g[kE];
                    E::unpack(__ldg(gate + c), g);
#pragma unroll
                    for (int i = 0; i < kE; ++i) f[i] *= g[i];
                }
            }
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                rn[v][i] = fmaf(sr1, f[i], q[i]);
                s[0] = fmaf(rn[v][i], rn[v][i], s[0]);
            }
            if (c < nvec) st_stream_v4(a.Rn + base + c, E::pack(rn[v]));
        }
        if (a.w2) {
            row_sum<1>(s, slots[grp], turn, grp, T);
            const float r2 = 1.0f / sqrtf(s[0] * inv_d + a.eps);
            if (a.rstd2 && tid == 0) a.rstd2[row] = r2;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                if (c < nvec) {
                    float w[kE];
                    E::unpack(__ldg(a.w2 + c), w);
#pragma unroll
                    for (int i = 0; i < kE; ++i) w[i] *= rn[v][i] * r2;
                    st_stream_v4(a.N + base + c, E::pack(w));
                }
            }
        }
    }
}

struct NormBwdArgs {
    const uint4 *dRn, *dN, *Y, *Rn;  // dRn null: zero; dN null with w2
    const float *rstd1, *rstd2;
    const uint4 *w1, *w2, *gate;
    uint4 *dY, *dR, *dgate;          // dgate: written here when a gate row has one worker
    float *acc2, *acc1, *accg;       // workspaces: [workers][D], [workers][D], [items][D]
    int64_t rows_per_gate;           // rows of one gate row (all of them without per-row gates)
    int64_t groups;                  // gate rows (1 without)
    int splits;                      // workers that share a gate row's rows
    int D;
    float scale;
};

// A worker is one row group (blockDim.x threads); worker w of W takes items
// w, w + W, ...; item = (gate row, split): a run of consecutive rows that
// share their gate row.  Its column sums stay in registers and leave once:
// acc2 = sum dN n; acc1 = sum dX y, or with per-row gates sum s g dX y and
// per item accg = sum dX y.
template <bool kBf16, int kV, bool kGroups>
__global__ void __launch_bounds__(kRowThreadsMax) block_norm_bwd_kernel(const NormBwdArgs a) {
    using E = Vec<kBf16>;
    constexpr int kE = E::kE;
    __shared__ float slots[8][2 * 3 * 16];
    const int T = blockDim.x, tid = threadIdx.x, grp = threadIdx.y;
    const int nvec = a.D / kE;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    int turn = 0;
    const int64_t workers = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * blockDim.y + grp;
    const int64_t items = a.groups * a.splits;

    float s2[kV][kE], s1[kV][kE], sg[kV][kE];
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < kE; ++i) s2[v][i] = s1[v][i] = sg[v][i] = 0.0f;

    for (int64_t item = me; item < items; item += workers) {
        const int64_t gr = item / a.splits;
        const int64_t sp = item - gr * a.splits;
        const int64_t row0 = gr * a.rows_per_gate + a.rows_per_gate * sp / a.splits;
        const int64_t row1 = gr * a.rows_per_gate + a.rows_per_gate * (sp + 1) / a.splits;
        const uint4 *gate = a.gate ? a.gate + gr * nvec : nullptr;
        for (int64_t row = row0; row < row1; ++row) {
            const int64_t base = row * nvec;
            const float r1 = a.w1 ? a.rstd1[row] : 1.0f;
            const float r2 = a.w2 ? a.rstd2[row] : 0.0f;
            uint4 xd[kV], xn[kV], xy[kV], xr[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                xd[v] = xn[v] = xy[v] = xr[v] = make_uint4(0, 0, 0, 0);
                if (c < nvec) {
                    if (a.dRn) xd[v] = ld_stream_v4(a.dRn + base + c);
                    xy[v] = ld_stream_v4(a.Y + base + c);
                    if (a.w2) {
                        xn[v] = ld_stream_v4(a.dN + base + c);
                        xr[v] = ld_stream_v4(a.Rn + base + c);
                    }
                }
            }
            // sums: a n, t e, t n
            float s[3] = {0.0f, 0.0f, 0.0f};
            float sgw[kV][kE];  // s g W1
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                float d[kE], n[kE], y[kE], r[kE], w[kE];
                E::unpack(xd[v], d);
                E::unpack(xn[v], n);
                E::unpack(xy[v], y);
                E::unpack(xr[v], r);
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    sgw[v][i] = a.scale;
                    w[i] = 0.0f;
                }
                if (c < nvec) {
                    float f[kE];
                    if (a.w1) {
                        E::unpack(__ldg(a.w1 + c), f);
#pragma unroll
                        for (int i = 0; i < kE; ++i) sgw[v][i] *= f[i];
                    }
                    if (gate) {
                        E::unpack(__ldg(gate + c), f);
#pragma unroll
                        for (int i = 0; i < kE; ++i) sgw[v][i] *= f[i];
                    }
                    if (a.w2) E::unpack(__ldg(a.w2 + c), w);
                }
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const float nh = r[i] * r2;
                    const float av = w[i] * n[i];
                    const float t = sgw[v][i] * (y[i] * r1);
                    s[0] = fmaf(av, nh, s[0]);
                    s[1] = fmaf(t, fmaf(r2, av, d[i]), s[1]);
                    s[2] = fmaf(t, nh, s[2]);
                    s2[v][i] = fmaf(n[i], nh, s2[v][i]);
                }
            }
            row_sum<3>(s, slots[grp], turn, grp, T);
            const float k2 = r2 * (s[0] * inv_d);                  // r2 mean(a n)
            const float c1 = a.w1 ? (s[1] - k2 * s[2]) * inv_d : 0.0f;  // mean(b y)
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                if (c < nvec) {
                    float d[kE], n[kE], y[kE], r[kE], w[kE], dy[kE];
                    E::unpack(xd[v], d);
                    E::unpack(xn[v], n);
                    E::unpack(xy[v], y);
                    E::unpack(xr[v], r);
                    if (a.w2) {
                        E::unpack(__ldg(a.w2 + c), w);
#pragma unroll
                        for (int i = 0; i < kE; ++i)
                            d[i] = fmaf(r2, w[i] * n[i], d[i]) - k2 * (r[i] * r2);
                    }
#pragma unroll
                    for (int i = 0; i < kE; ++i) {
                        const float yh = y[i] * r1;
                        dy[i] = sgw[v][i] * d[i];
                        if (a.w1) dy[i] = r1 * (dy[i] - yh * c1);
                        if (kGroups) sg[v][i] = fmaf(d[i], yh, sg[v][i]);
                        else s1[v][i] = fmaf(d[i], yh, s1[v][i]);
                    }
                    st_stream_v4(a.dR + base + c, E::pack(d));
                    st_stream_v4(a.dY + base + c, E::pack(dy));
                }
            }
        }
        if constexpr (kGroups) {
            // this item's share of the gate row's gradient
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int c = v * T + tid;
                if (c < nvec) {
                    float g[kE], w[kE];
                    E::unpack(__ldg(gate + c), g);
#pragma unroll
                    for (int i = 0; i < kE; ++i) w[i] = 1.0f;
                    if (a.w1) E::unpack(__ldg(a.w1 + c), w);
                    if (a.splits == 1) {
                        float o[kE];
#pragma unroll
                        for (int i = 0; i < kE; ++i) o[i] = a.scale * w[i] * sg[v][i];
                        a.dgate[gr * nvec + c] = E::pack(o);
                    } else {
#pragma unroll
                        for (int i = 0; i < kE; ++i)
                            a.accg[item * a.D + static_cast<int64_t>(c) * kE + i] = sg[v][i];
                    }
#pragma unroll
                    for (int i = 0; i < kE; ++i) {
                        s1[v][i] = fmaf(a.scale * g[i], sg[v][i], s1[v][i]);
                        sg[v][i] = 0.0f;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int c = v * T + tid;
        if (c < nvec) {
#pragma unroll
            for (int i = 0; i < kE; i += 4) {
                const int64_t o = me * a.D + static_cast<int64_t>(c) * kE + i;
                if (a.acc2)
                    *reinterpret_cast<float4 *>(a.acc2 + o) =
                        make_float4(s2[v][i], s2[v][i + 1], s2[v][i + 2], s2[v][i + 3]);
                if (a.acc1)
                    *reinterpret_cast<float4 *>(a.acc1 + o) =
                        make_float4(s1[v][i], s1[v][i + 1], s1[v][i + 2], s1[v][i + 3]);
            }
        }
    }
}

struct NormReduceArgs {
    const float *acc2, *acc1, *accg;
    const void *w1, *gate;
    void *dw2, *dw1, *dgate;   // null: not wanted here
    int64_t workers;
    int splits;
    int D;
    int per_row;               // per-row gates: acc1 holds dW1 itself, accg the gate rows' sums
    float scale;
};

constexpr int kReduceRows = 16;

// Joins the workers' column sums, in a fixed order: blockIdx.y = 0 the
// weights (and the single gate row), 1 + g gate row g.
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
    const bool gates = blockIdx.y > 0;
    const int64_t gr = static_cast<int64_t>(blockIdx.y) - 1;
    float v0 = 0.0f, v1 = 0.0f;
    if (col < a.D) {
        if (gates) {
            for (int64_t i = ty; i < a.splits; i += kReduceRows)
                v0 += a.accg[(gr * a.splits + i) * a.D + col];
        } else {
            for (int64_t i = ty; i < a.workers; i += kReduceRows) {
                if (a.acc2) v0 += a.acc2[i * a.D + col];
                if (a.acc1) v1 += a.acc1[i * a.D + col];
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
    if (gates) {
        store(a.dgate, gr * a.D + col, a.scale * w * v0);
        return;
    }
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

struct BwdPlan {
    RowShape rows;
    int64_t workers, splits, blocks;
    size_t bytes;
};

// Workers: up to two blocks per SM, at least eight rows each (each worker
// costs 8 D bytes of column sums written and read again).
BwdPlan bwd_plan(int64_t M, int D, int dtype_f32, bool per_row, int64_t groups, bool w1, bool w2,
                 bool gate, int sm_count) {
    BwdPlan p{};
    p.rows = row_shape(D / (dtype_f32 ? 4 : 8));
    int64_t want = static_cast<int64_t>(sm_count) * 2 * p.rows.groups;
    const int64_t most = (M + 7) / 8;
    if (want > most) want = most;
    if (want < 1) want = 1;
    p.splits = per_row ? (want / groups > 0 ? want / groups : 1) : want;
    const int64_t rows_per_group = per_row ? M / groups : M;
    if (p.splits > rows_per_group) p.splits = rows_per_group;
    if (p.splits < 1) p.splits = 1;
    const int64_t items = (per_row ? groups : 1) * p.splits;
    if (want > items) want = items;
    p.blocks = (want + p.rows.groups - 1) / p.rows.groups;
    p.workers = p.blocks * p.rows.groups;
    size_t floats = 0;
    if (w2) floats += static_cast<size_t>(p.workers) * D;
    if (w1 || (gate && !per_row)) floats += static_cast<size_t>(p.workers) * D;
    if (per_row && p.splits > 1) floats += static_cast<size_t>(items) * D;
    p.bytes = floats * 4;
    return p;
}

template <bool kBf16>
void launch_fwd(const NormArgs &a, int sm_count, cudaStream_t stream) {
    const RowShape s = row_shape(a.D / Vec<kBf16>::kE);
    const dim3 block(s.T, s.groups);
    int64_t blocks = (a.M + s.groups - 1) / s.groups;
    const int64_t most = static_cast<int64_t>(sm_count) * (2048 / (s.T * s.groups));
    if (blocks > most) blocks = most;
    const unsigned g = static_cast<unsigned>(blocks);
    switch (s.v) {
        case 1: block_norm_kernel<kBf16, 1><<<g, block, 0, stream>>>(a); break;
        case 2: block_norm_kernel<kBf16, 2><<<g, block, 0, stream>>>(a); break;
        default: block_norm_kernel<kBf16, 4><<<g, block, 0, stream>>>(a); break;
    }
}

template <bool kBf16, bool kGroups>
void launch_bwd(const NormBwdArgs &a, const BwdPlan &p, cudaStream_t stream) {
    const dim3 block(p.rows.T, p.rows.groups);
    const unsigned g = static_cast<unsigned>(p.blocks);
    switch (p.rows.v) {
        case 1: block_norm_bwd_kernel<kBf16, 1, kGroups><<<g, block, 0, stream>>>(a); break;
        case 2: block_norm_bwd_kernel<kBf16, 2, kGroups><<<g, block, 0, stream>>>(a); break;
        default: block_norm_bwd_kernel<kBf16, 4, kGroups><<<g, block, 0, stream>>>(a); break;
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
    if (f32) launch_fwd<false>(a, dev.sm_count, stream);
    else launch_fwd<true>(a, dev.sm_count, stream);
    return cudaGetLastError();
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
    const int64_t groups = per_row ? n.gate_rows : 1;
    const BwdPlan p = bwd_plan(M, D, f32, per_row, groups, n.w1, n.w2, n.gate, dev.sm_count);
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
    const size_t per = static_cast<size_t>(p.workers) * D;
    if (n.w2) {
        a.acc2 = ws;
        ws += per;
    }
    if (n.w1 || (n.gate && !per_row)) {
        a.acc1 = ws;
        ws += per;
    }
    if (per_row && p.splits > 1) a.accg = ws;
    a.rows_per_gate = per_row ? M / groups : M;
    a.groups = groups;
    a.splits = static_cast<int>(p.splits);
    a.D = D;
    a.scale = n.scale;
    if (f32) {
        if (per_row) launch_bwd<false, true>(a, p, stream);
        else launch_bwd<false, false>(a, p, stream);
    } else {
        if (per_row) launch_bwd<true, true>(a, p, stream);
        else launch_bwd<true, false>(a, p, stream);
    }
    cudaError_t e = cudaGetLastError();
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
    r.workers = p.workers;
    r.splits = a.splits;
    r.D = D;
    r.per_row = per_row ? 1 : 0;
    r.scale = n.scale;
    const dim3 grid((D + 31) / 32, static_cast<unsigned>(1 + (a.accg ? groups : 0)));
    const dim3 block(32, kReduceRows);
    if (f32) block_norm_reduce_kernel<false><<<grid, block, 0, stream>>>(r);
    else block_norm_reduce_kernel<true><<<grid, block, 0, stream>>>(r);
    return cudaGetLastError();
}

}  // namespace swiglu
