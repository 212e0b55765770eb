// api_block.cu -- C entry points of the operators around the projection:
// block norms, e4m3 quantisation in blocks of 128, block-scaled products.
// Validation is pure host logic and runs before any CUDA call, as in api.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_util.cuh"
#include "kernels.cuh"
#include "swiglu.h"

namespace swiglu {
namespace {

constexpr int64_t kMaxGrid = (1LL << 31) - 1;
constexpr int64_t kNormRowBytes = 32768;  // a norm's row stays in registers

struct Span {
    const void *p;
    int64_t bytes;
};

// Pointers present and 16-byte aligned; no output over an input or another
// output, except (in place) output i over input in_place[i] exactly.
int check_spans(const Span *in, int n_in, const Span *out, int n_out, const int *in_place) {
    for (int i = 0; i < n_in; ++i)
        if (in[i].bytes > 0 && !in[i].p) return SWIGLU_ERR_NULL_POINTER;
    for (int i = 0; i < n_out; ++i)
        if (out[i].bytes > 0 && !out[i].p) return SWIGLU_ERR_NULL_POINTER;
    for (int i = 0; i < n_in; ++i)
        if (in[i].bytes > 0 && !aligned16(in[i].p)) return SWIGLU_ERR_MISALIGNED_PTR;
    for (int i = 0; i < n_out; ++i)
        if (out[i].bytes > 0 && !aligned16(out[i].p)) return SWIGLU_ERR_MISALIGNED_PTR;
    for (int i = 0; i < n_out; ++i) {
        if (out[i].bytes == 0) continue;
        for (int j = 0; j < n_in; ++j) {
            if (in[j].bytes == 0 || (in_place && in_place[i] == j && out[i].p == in[j].p)) continue;
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return SWIGLU_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (out[j].bytes > 0 && overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                return SWIGLU_ERR_OVERLAP;
    }
    return SWIGLU_OK;
}

int check_norm_shape(int64_t M, int64_t D, int dtype, const swiglu_block_norm_params *p) {
    if (!p) return SWIGLU_ERR_NULL_POINTER;
    if (dtype != SWIGLU_BF16 && dtype != SWIGLU_FP32) return SWIGLU_ERR_BAD_DTYPE;
    if (M < 0 || D < 0 || M > kMaxDim || D > kNormRowBytes / elem_size(dtype)) return SWIGLU_ERR_BAD_DIM;
    if (D * elem_size(dtype) % 16 != 0) return SWIGLU_ERR_MISALIGNED_DIM;
    if (!isfinite(p->residual_scale) || !isfinite(p->eps) || p->eps < 0.0f)
        return SWIGLU_ERR_BAD_EPILOGUE;
    if (p->gate && (p->gate_rows < 1 || p->gate_rows > kMaxDim || (M > 0 && M % p->gate_rows != 0)))
        return SWIGLU_ERR_BAD_DIM;
    return SWIGLU_OK;
}

BlockNorm norm_of(const swiglu_block_norm_params *p) {
    BlockNorm n;
    n.w1 = p->post_weight;
    n.w2 = p->pre_weight;
    n.gate = p->gate;
    n.gate_rows = p->gate ? p->gate_rows : 1;
    n.scale = p->residual_scale;
    n.eps = p->eps;
    return n;
}

int64_t blocks128(int64_t n) { return (n + 127) / 128; }
int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

// Bytes of the scales of `rows` x `cols` in 1 x 128 (rows innermost, padded
// to 4) or 128 x 128 blocks.
int64_t scale_bytes(int64_t rows, int64_t cols, int block) {
    return 4 * blocks128(cols) * (block == SWIGLU_BLOCK_TILE ? blocks128(rows) : up4(rows));
}

int check_product_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return SWIGLU_ERR_BAD_DIM;
    if (N % 8 != 0 || K % 16 != 0) return SWIGLU_ERR_MISALIGNED_DIM;
    // (tiles are 128 rows by at least one unit of 8 columns)
    if (blocks128(M) * (N / 8) > kMaxGrid) return SWIGLU_ERR_BAD_DIM;
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

SWIGLU_API int swiglu_block_norm(const void *Y, const void *R, const swiglu_block_norm_params *p,
                                 void *Rn, void *N, float *rstd_post, float *rstd_pre, int64_t M,
                                 int64_t D, int dtype, cudaStream_t stream) {
    int st = check_norm_shape(M, D, dtype, p);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || D == 0) return SWIGLU_OK;
    const int es = elem_size(dtype);
    const int64_t mat = M * D * es, vec = D * es;
    const Span in[] = {{R, mat},
                       {Y, mat},
                       {p->post_weight, p->post_weight ? vec : 0},
                       {p->pre_weight, p->pre_weight ? vec : 0},
                       {p->gate, p->gate ? vec * p->gate_rows : 0}};
    const Span out[] = {{Rn, mat}, {N, p->pre_weight ? mat : 0},
                        {rstd_post, p->post_weight && rstd_post ? 4 * M : 0},
                        {rstd_pre, p->pre_weight && rstd_pre ? 4 * M : 0}};
    const int in_place[] = {0, 1, -1, -1};
    st = check_spans(in, 5, out, 4, in_place);
    if (st != SWIGLU_OK) return st;
    DeviceInfo dev;
    st = current_device(dev);
    if (st != SWIGLU_OK) return st;
    return from_cuda(launch_block_norm(Y, R, norm_of(p), Rn, N, p->post_weight ? rstd_post : nullptr,
                                       p->pre_weight ? rstd_pre : nullptr, M, static_cast<int>(D),
                                       dtype == SWIGLU_FP32, dev, stream));
}

SWIGLU_API int64_t swiglu_block_norm_bwd_workspace(const swiglu_block_norm_params *p, int64_t M,
                                                   int64_t D, int dtype) {
    if (check_norm_shape(M, D, dtype, p) != SWIGLU_OK) return -1;
    if (M == 0 || D == 0) return 0;
    DeviceInfo dev;
    if (current_device(dev) != SWIGLU_OK) return -1;
    return static_cast<int64_t>(
        block_norm_bwd_workspace(M, static_cast<int>(D), dtype == SWIGLU_FP32, norm_of(p), dev.sm_count));
}

SWIGLU_API int swiglu_block_norm_bwd(const void *dRn, const void *dN, const void *Y, const void *Rn,
                                     const float *rstd_post, const float *rstd_pre,
                                     const swiglu_block_norm_params *p, void *dY, void *dR,
                                     void *d_post, void *d_pre, void *d_gate, void *workspace,
                                     int64_t workspace_bytes, int64_t M, int64_t D, int dtype,
                                     cudaStream_t stream) {
    int st = check_norm_shape(M, D, dtype, p);
    if (st != SWIGLU_OK) return st;
    if (D == 0) return SWIGLU_OK;
    const int es = elem_size(dtype);
    const int64_t mat = M * D * es, vec = D * es;
    const int64_t post = p->post_weight ? 1 : 0, pre = p->pre_weight ? 1 : 0;
    const int64_t gates = p->gate ? p->gate_rows : 0;
    const Span in[] = {{dRn, dRn ? mat : 0}, {dN, pre * mat},        {Y, mat},
                       {Rn, pre * mat},      {rstd_post, post * 4 * M}, {rstd_pre, pre * 4 * M},
                       {p->post_weight, post * vec}, {p->pre_weight, pre * vec}, {p->gate, gates * vec}};
    const Span out[] = {{dY, mat}, {dR, mat}, {d_post, post * vec}, {d_pre, pre * vec}, {d_gate, gates * vec}};
    if (!dRn && !pre && M > 0) return SWIGLU_ERR_NULL_POINTER;
    st = check_spans(in, 9, out, 5, nullptr);
    if (st != SWIGLU_OK) return st;
    DeviceInfo dev;
    st = current_device(dev);
    if (st != SWIGLU_OK) return st;
    if (M == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        for (int i = 2; i < 5; ++i)
            if (out[i].bytes > 0 && e == cudaSuccess)
                e = cudaMemsetAsync(const_cast<void *>(out[i].p), 0, static_cast<size_t>(out[i].bytes), stream);
        return from_cuda(e);
    }
    const BlockNorm n = norm_of(p);
    const int64_t need = static_cast<int64_t>(
        block_norm_bwd_workspace(M, static_cast<int>(D), dtype == SWIGLU_FP32, n, dev.sm_count));
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return SWIGLU_ERR_WORKSPACE;
        const Span ws[] = {{workspace, need}};
        Span rest[14];
        for (int i = 0; i < 9; ++i) rest[i] = in[i];
        for (int i = 0; i < 5; ++i) rest[9 + i] = out[i];
        st = check_spans(rest, 14, ws, 1, nullptr);
        if (st != SWIGLU_OK) return st;
    }
    return from_cuda(launch_block_norm_bwd(dRn, dN, Y, Rn, rstd_post, rstd_pre, n, dY, dR, d_post,
                                           d_pre, d_gate, workspace, M, static_cast<int>(D),
                                           dtype == SWIGLU_FP32, dev, stream));
}

SWIGLU_API int swiglu_quant_b128(const void *X, void *Q, float *S, int64_t R, int64_t C, int dtype,
                                 int block, int transpose, cudaStream_t stream) {
    if (dtype != SWIGLU_BF16 && dtype != SWIGLU_FP32) return SWIGLU_ERR_BAD_DTYPE;
    if (block != SWIGLU_BLOCK_ROW && block != SWIGLU_BLOCK_TILE) return SWIGLU_ERR_BAD_BLOCK;
    if (R < 0 || C < 0 || R > kMaxDim || C > kMaxDim) return SWIGLU_ERR_BAD_DIM;
    if (C % 16 != 0) return SWIGLU_ERR_MISALIGNED_DIM;
    if (R == 0 || C == 0) return SWIGLU_OK;
    // (the row kernel's blocks hold 16 rows by 512 columns, the others 128 x 128)
    if (((R + 15) / 16) * ((C + 511) / 512) > kMaxGrid || blocks128(R) * blocks128(C) > kMaxGrid)
        return SWIGLU_ERR_BAD_DIM;
    const int64_t qbytes = transpose ? C * ((R + 15) / 16 * 16) : R * C;
    const int64_t sbytes = transpose ? scale_bytes(C, R, block) : scale_bytes(R, C, block);
    const Span in[] = {{X, R * C * elem_size(dtype)}};
    const Span out[] = {{Q, qbytes}, {S, sbytes}};
    int st = check_spans(in, 1, out, 2, nullptr);
    if (st != SWIGLU_OK) return st;
    DeviceInfo dev;
    st = current_device(dev);
    if (st != SWIGLU_OK) return st;
    return from_cuda(launch_quant_b128(X, Q, S, R, static_cast<int>(C), dtype == SWIGLU_FP32,
                                       block == SWIGLU_BLOCK_TILE, transpose != 0, stream));
}

SWIGLU_API int swiglu_gemm_b128(const void *A, const float *As, const void *B, const float *Bs,
                                void *Y, int64_t M, int64_t N, int64_t K, int b_block,
                                int out_dtype, cudaStream_t stream) {
    if (out_dtype != SWIGLU_BF16 && out_dtype != SWIGLU_FP32) return SWIGLU_ERR_BAD_DTYPE;
    if (b_block != SWIGLU_BLOCK_ROW && b_block != SWIGLU_BLOCK_TILE) return SWIGLU_ERR_BAD_BLOCK;
    int st = check_product_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return SWIGLU_OK;
    const Span in[] = {{A, M * K}, {As, scale_bytes(M, K, SWIGLU_BLOCK_ROW)},
                       {B, N * K}, {Bs, scale_bytes(N, K, b_block)}};
    const Span out[] = {{Y, M * N * elem_size(out_dtype)}};
    st = check_spans(in, 4, out, 1, nullptr);
    if (st != SWIGLU_OK) return st;
    DeviceInfo dev;
    st = current_device(dev);
    if (st != SWIGLU_OK) return st;
    if (K == 0) return from_cuda(cudaMemsetAsync(Y, 0, static_cast<size_t>(out[0].bytes), stream));
    return from_cuda(launch_gemm_b128(A, As, B, Bs, Y, static_cast<int>(M), static_cast<int>(N),
                                      static_cast<int>(K), b_block == SWIGLU_BLOCK_ROW,
                                      out_dtype == SWIGLU_FP32, dev, stream));
}

SWIGLU_API int swiglu_fwd_b128(const void *X, const float *Xs, const void *Wg, const float *Wgs,
                               const void *Wu, const float *Wus, void *H, int64_t M, int64_t K,
                               int64_t N, const swiglu_epilogue *epi, cudaStream_t stream) {
    int st = check_product_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    Epilogue ep;
    if (epi) {
        if (epi->activation != SWIGLU_ACT_SILU && epi->activation != SWIGLU_ACT_GELU_TANH)
            return SWIGLU_ERR_BAD_EPILOGUE;
        if (!isfinite(epi->gate_multiplier)) return SWIGLU_ERR_BAD_EPILOGUE;
        if ((epi->G == nullptr) != (epi->U == nullptr)) return SWIGLU_ERR_BAD_EPILOGUE;
        ep.activation = epi->activation;
        ep.gate_multiplier = epi->gate_multiplier;
        ep.G = epi->G;
        ep.U = epi->U;
    }
    if (M == 0 || N == 0) return SWIGLU_OK;
    const int64_t ws = scale_bytes(N, K, SWIGLU_BLOCK_TILE), ob = 2 * M * N;
    const Span in[] = {{X, M * K},  {Xs, scale_bytes(M, K, SWIGLU_BLOCK_ROW)},
                       {Wg, N * K}, {Wgs, ws},
                       {Wu, N * K}, {Wus, ws}};
    const Span out[] = {{H, ob}, {ep.G, ep.G ? ob : 0}, {ep.U, ep.U ? ob : 0}};
    st = check_spans(in, 6, out, 3, nullptr);
    if (st != SWIGLU_OK) return st;
    DeviceInfo dev;
    st = current_device(dev);
    if (st != SWIGLU_OK) return st;
    if (K == 0) {  // G = U = 0 and act(0) = 0
        cudaError_t e = cudaSuccess;
        for (const Span &o : out)
            if (o.bytes > 0 && e == cudaSuccess)
                e = cudaMemsetAsync(const_cast<void *>(o.p), 0, static_cast<size_t>(o.bytes), stream);
        return from_cuda(e);
    }
    return from_cuda(launch_fwd_b128(X, Xs, Wg, Wgs, Wu, Wus, H, static_cast<int>(M),
                                     static_cast<int>(N), static_cast<int>(K), ep, dev, stream));
}

}  // extern "C"
