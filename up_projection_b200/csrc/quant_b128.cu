// quant_b128.cu -- e4m3 quantisation with one scale per block of 128: the
// operands of the block-scaled products (gemm_b128.cu).
//
//   amax = max |x| over the block (1 x 128 along the row, or 128 x 128)
//   e    = the smallest integer with amax <= 448 * 2^e, in [-126, 127]
//   s    = 2^e (1 for a block of zeros),  q = e4m3_rne(x / s).
//
// Power-of-two scales as in the fp8 forward's (1,32) blocks: x / s is exact,
// so each code is the correctly rounded one whatever the block.  A block
// holding Inf or NaN gets a NaN scale and NaN codes (0x7F).
//
// B200, 8192 x 14336 bf16: rows 60 us, 90 % of the measured copy bandwidth, the
// transpose's rows 60 us (91 %; each column's scale formed by one thread: by all
// sixteen that use it 72 us), 128 x 128 tiles of 14336 x 4096 30 us (88 %).
//
// HBM-bound: each element is read once (16-byte loads held in registers
// between the maximum and the conversion) and its code written once.  The
// transposed forms (blocks along the rows, for products that reduce over
// them) turn the codes in shared memory, 8 x 8 per thread.
#include <cuda_bf16.h>

#include "kernels.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace swiglu {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;   // a half warp holds one row of 128
constexpr int kRowsPerBlock = kHalfWarps;   // row kernel: rows per CTA
constexpr int kRowBlocks = 4;               // row kernel: 128-wide blocks per CTA

// 8 consecutive elements, as they were loaded.
template <bool kBf16>
struct Oct {
    uint4 v[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *base, int64_t elem) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) +
                                                        elem * (kBf16 ? 2 : 4));
        if constexpr (kBf16) {
            v[0] = ld_stream_v4(p);
        } else {   // (the second 16 bytes of each sector come out of L1)
            v[0] = ld_plain(p);
            v[1] = ld_plain(p + 1);
        }
    }
    __device__ __forceinline__ void zero() {
        v[0] = make_uint4(0, 0, 0, 0);
        if constexpr (!kBf16) v[1] = v[0];
    }
    // Bits of element i as fp32 (i a compile-time constant).
    __device__ __forceinline__ uint32_t bits(int i) const {
        const uint4 &w = v[kBf16 ? 0 : i / 4];
        const int k = kBf16 ? i / 2 : i % 4;
        const uint32_t x = k == 0 ? w.x : (k == 1 ? w.y : (k == 2 ? w.z : w.w));
        return kBf16 ? ((i & 1) ? (x & 0xFFFF0000u) : (x << 16)) : x;
    }
};

// Scale of a block whose largest |x| has these fp32 bits, and 1 / scale.
// Magnitude bits order as the values do, with Inf and NaN on top.
struct BlockScale {
    float s, inv;
    bool finite;
    __device__ __forceinline__ explicit BlockScale(uint32_t amax) {
        finite = amax < 0x7f800000u;
        // amax = 1.f * 2^(ef-127) <= 1.75 * 2^(e+8)
        int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(e, -126);  // (the largest finite amax has e = 120)
        s = __uint_as_float(finite ? static_cast<uint32_t>(e + 127) << 23 : 0x7fc00000u);
        inv = __uint_as_float(static_cast<uint32_t>(127 - min(e, 126)) << 23);
        if (amax == 0) s = inv = 1.0f;
    }
    // Another thread's 1 / scale, NaN where the block is not finite.
    __device__ __forceinline__ explicit BlockScale(float inverse) : s(0.0f), inv(inverse), finite(true) {}
};

// Codes of two elements, a in the low byte.
__device__ __forceinline__ uint32_t code2(uint32_t a, uint32_t b, const BlockScale &s) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r)
        : "f"(__uint_as_float(b) * s.inv), "f"(__uint_as_float(a) * s.inv));
    return s.finite ? r : 0x7f7fu;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t oct_amax(const Oct<kBf16> &x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, x.bits(i) & 0x7fffffffu);
    return m;
}

// 1 x 128 blocks: a half warp per (row, block), kRowBlocks blocks of a row
// each, all loads before the first use.  S is [ceil(C/128)][lds], rows
// innermost: the 16 rows of a CTA write 64 consecutive bytes per block.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const void *X, uint8_t *Q, float *S,
                                                              int64_t R, int C, int64_t lds) {
    const int lane = threadIdx.x & 15;
    const int cb = (C + 127) / 128;
    const unsigned across = (cb + kRowBlocks - 1) / kRowBlocks;
    const int64_t row = static_cast<int64_t>(blockIdx.x / across) * kRowsPerBlock + (threadIdx.x >> 4);
    const int b0 = static_cast<int>(blockIdx.x % across) * kRowBlocks;
    griddep_launch_dependents();
    griddep_wait();
    // bf16: a lane's 8 elements are consecutive; fp32: its two halves are 64
    // apart, so that the lanes of a load lie side by side (8192 x 4096 26.4 us;
    // 8 consecutive ones 29.0)
    constexpr int kHalf = kBf16 ? 8 : 4;
    Oct<kBf16> x[kRowBlocks];
#pragma unroll
    for (int j = 0; j < kRowBlocks; ++j) {
        const int col = (b0 + j) * 128 + kHalf * lane;
        x[j].zero();
        if constexpr (kBf16) {
            if (row < R && col < C) x[j].load(X, row * C + col);
        } else {
            const float *p = static_cast<const float *>(X) + row * C + col;
            if (row < R && col < C) x[j].v[0] = ld_stream_v4(p);
            if (row < R && col + 64 < C) x[j].v[1] = ld_stream_v4(p + 64);
        }
    }
#pragma unroll
    for (int j = 0; j < kRowBlocks; ++j) {
        uint32_t m = oct_amax(x[j]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const BlockScale s(m);
        const int col = (b0 + j) * 128 + kHalf * lane;
        if (row < R && col < C) {
            uint2 q;
            q.x = code2(x[j].bits(0), x[j].bits(1), s) | (code2(x[j].bits(2), x[j].bits(3), s) << 16);
            q.y = code2(x[j].bits(4), x[j].bits(5), s) | (code2(x[j].bits(6), x[j].bits(7), s) << 16);
            if constexpr (kBf16) {
                *reinterpret_cast<uint2 *>(Q + row * C + col) = q;
            } else {
                *reinterpret_cast<uint32_t *>(Q + row * C + col) = q.x;
                if (col + 64 < C) *reinterpret_cast<uint32_t *>(Q + row * C + col + 64) = q.y;
            }
        }
        if (row < R && lane == 0 && b0 + j < cb) S[static_cast<int64_t>(b0 + j) * lds + row] = s.s;
    }
}

// A 128 x 128 tile of X per CTA: half warp h holds rows 8 h .. 8 h + 7, its
// lane l columns 8 l .. 8 l + 7.  kTile: one scale for the tile; otherwise
// one per column (1 x 128 blocks of the transpose).  kTrans: codes to
// [C][Rp], Rp = R rounded up to 16 with zero codes, else to [R][C].
// S: tile [ceil(R/128)][ceil(C/128)] (transposed: [ceil(C/128)][ceil(R/128)]),
// columns [ceil(R/128)][C].
template <bool kBf16, bool kTile, bool kTrans>
__global__ void __launch_bounds__(kThreads) quant_tile_kernel(const void *X, uint8_t *Q, float *S,
                                                              int64_t R, int C, int64_t Rp) {
    __shared__ uint32_t colmax[kTile ? 1 : kThreads / 32][128];
    __shared__ float inverse[kTile ? 1 : 128];
    __shared__ uint2 turned[kTrans ? 128 * 16 : 1];
    const int h = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const unsigned across = (C + 127) / 128;
    const int64_t tr = blockIdx.x / across;              // tile row and column
    const int tc = static_cast<int>(blockIdx.x % across);
    const int64_t r0 = tr * 128 + 8 * h;
    const int c0 = tc * 128 + 8 * lane;
    griddep_launch_dependents();
    griddep_wait();
    Oct<kBf16> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + i < R && c0 < C) x[i].load(X, (r0 + i) * C + c0);
        else x[i].zero();
    }
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[j] = max(m[j], x[i].bits(j) & 0x7fffffffu);
    }
    if constexpr (kTile) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, m[j]);
        a = __reduce_max_sync(0xffffffffu, a);
        if ((threadIdx.x & 31) == 0) colmax[0][threadIdx.x >> 5] = a;
        __syncthreads();
        a = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) a = max(a, colmax[0][w]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = a;
        if (threadIdx.x == 0) {
            S[kTrans ? tc * ((R + 127) / 128) + tr : tr * across + tc] = BlockScale(a).s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        uint32_t *mine = &colmax[threadIdx.x >> 5][8 * lane];
        if ((threadIdx.x & 16) == 0) {
            *reinterpret_cast<uint4 *>(mine) = make_uint4(m[0], m[1], m[2], m[3]);
            *reinterpret_cast<uint4 *>(mine + 4) = make_uint4(m[4], m[5], m[6], m[7]);
        }
        __syncthreads();
        // one thread per column: its scale, and 1 / scale for all (NaN for a
        // block that is not finite, which makes its codes 0x7F)
        if (threadIdx.x < 128) {
            uint32_t a = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) a = max(a, colmax[w][threadIdx.x]);
            const BlockScale sc(a);
            const int c = tc * 128 + threadIdx.x;
            if (c < C) S[tr * C + c] = sc.s;
            inverse[threadIdx.x] = sc.finite ? sc.inv : __uint_as_float(0x7fc00000u);
        }
        __syncthreads();
    }
    if constexpr (!kTrans) {
        const BlockScale s(m[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i < R && c0 < C) {
                uint2 q;
                q.x = code2(x[i].bits(0), x[i].bits(1), s) | (code2(x[i].bits(2), x[i].bits(3), s) << 16);
                q.y = code2(x[i].bits(4), x[i].bits(5), s) | (code2(x[i].bits(6), x[i].bits(7), s) << 16);
                *reinterpret_cast<uint2 *>(Q + (r0 + i) * C + c0) = q;
            }
        }
    } else {
        // column 8 l + j of the tile: 16 chunks of 8 rows, chunk h at
        // h ^ l (the 16 lanes of a half warp write 16 different banks pairs,
        // and so do the 16 that read one column back)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const BlockScale s = kTile ? BlockScale(m[j]) : BlockScale(inverse[kTile ? 0 : 8 * lane + j]);
            uint2 q;
            q.x = code2(x[0].bits(j), x[1].bits(j), s) | (code2(x[2].bits(j), x[3].bits(j), s) << 16);
            q.y = code2(x[4].bits(j), x[5].bits(j), s) | (code2(x[6].bits(j), x[7].bits(j), s) << 16);
            turned[(8 * lane + j) * 16 + (h ^ lane)] = q;
        }
        if (r0 + 8 > R) {   // rows behind the last: code 0, in a NaN block too
            const int n = r0 < R ? static_cast<int>(R - r0) : 0;
            const uint32_t lo = n < 4 ? (1u << (8 * n)) - 1u : ~0u, hi = n < 4 ? 0u : (1u << (8 * (n - 4))) - 1u;
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                uint2 &q = turned[(8 * lane + j) * 16 + (h ^ lane)];
                q.x &= lo;
                q.y &= hi;
            }
        }
        __syncthreads();
        const int64_t r = tr * 128 + 8 * lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = h * 8 + i;
            const int c = tc * 128 + col;
            if (c < C && r < Rp)
                *reinterpret_cast<uint2 *>(Q + static_cast<int64_t>(c) * Rp + r) =
                    turned[col * 16 + (lane ^ h)];
        }
    }
}

template <bool kBf16>
cudaError_t launch(const void *X, uint8_t *Q, float *S, int64_t R, int C, bool tile, bool trans,
            cudaStream_t stream) {
    const int cb = (C + 127) / 128;
    if (!tile && !trans) {
        const unsigned grid = static_cast<unsigned>((cb + kRowBlocks - 1) / kRowBlocks *
                                                    ((R + kRowsPerBlock - 1) / kRowsPerBlock));
        return launch_dependent(quant_rows_kernel<kBf16>, grid, kThreads, 0, stream, X, Q, S, R, C, (R + 3) / 4 * 4);
    }
    const unsigned grid = static_cast<unsigned>(cb * ((R + 127) / 128));
    const int64_t Rp = (R + 15) / 16 * 16;
    if (!trans) return launch_dependent(quant_tile_kernel<kBf16, true, false>, grid, kThreads, 0, stream, X, Q, S, R, C, Rp);
    if (tile) return launch_dependent(quant_tile_kernel<kBf16, true, true>, grid, kThreads, 0, stream, X, Q, S, R, C, Rp);
    return launch_dependent(quant_tile_kernel<kBf16, false, true>, grid, kThreads, 0, stream, X, Q, S, R, C, Rp);
}

}  // namespace

cudaError_t launch_quant_b128(const void *X, void *Q, float *S, int64_t R, int C, int f32,
                              bool tile, bool trans, cudaStream_t stream) {
    return f32 ? launch<false>(X, static_cast<uint8_t *>(Q), S, R, C, tile, trans, stream)
               : launch<true>(X, static_cast<uint8_t *>(Q), S, R, C, tile, trans, stream);
}

}  // namespace swiglu
