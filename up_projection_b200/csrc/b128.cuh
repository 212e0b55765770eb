// b128.cuh -- pieces shared by the two kernels of the block-scaled e4m3
// products (gemm_b128.cu: large M; gemm_b128_stream.cu: few rows).
#pragma once

#include <cuda_bf16.h>

#include "activation.cuh"
#include "gemm_common.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace swiglu {
namespace b128 {

using namespace dev;
using gemm::mbar_wait_drain;

constexpr int kBM = 128;                     // rows of A per CTA
constexpr int kBlockK = 128;                 // bytes = e4m3 values per block and stage row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 4);  // (register shares go by groups of 4 warps)
// 384 threads start with 168 registers each; the accumulating warps take
// what the third group of warps gives back: 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kRegsLaunch = 168, kRegsEpi = 224, kRegsRest = 56;
static_assert(256 * kRegsEpi + 128 * kRegsRest <= kThreads * kRegsLaunch, "register split");
constexpr int kTmemCols = 512;
constexpr uint32_t kMaxSmem = 227 * 1024;

enum : int { kTileScales = 0, kRowScales = 1, kGated = 2 };

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

// The MMAs and commits below are called by a whole converged warp and issued by
// the thread that elect.sync names (the same one each time): with the loop's
// values uniform over the warp the compiler keeps descriptors in uniform
// registers.  (B200, one CTA, chains of four MMAs with M = 128: 39 cycles each
// at N = 16, 128 at N = 256; issued under `lane == 0` 51 at best and, with a
// few address computations between them, up to 160 -- more than the MMA.)
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
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

// One block's 32 accumulator columns of a warp, times their one scale, into the
// running sums.
__device__ __forceinline__ void add_block(unsigned long long (&acc)[16], const uint32_t (&v)[32], float s) {
    const unsigned long long s2 = pair2(s, s);
#pragma unroll
    for (int i = 0; i < 16; ++i) fma2(acc[i], v[2 * i], v[2 * i + 1], s2);
}

// The same with row scales: one per column, in shared memory at sb.
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

// Opt in to the shared memory and check that the launch starts with the
// registers its split hands out.
template <typename Kernel>
inline cudaError_t prepare_kernel(Kernel kernel, uint32_t smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    return fa.numRegs < kRegsLaunch ? cudaErrorInvalidConfiguration : cudaSuccess;
}

}  // namespace b128
}  // namespace swiglu
