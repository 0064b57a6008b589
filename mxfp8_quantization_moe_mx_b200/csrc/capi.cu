// capi.cu -- the extern "C" entry points of libmxq (declared in include/mxq.h).
//
// Each call checks its arguments on the host, launches nothing on an argument error,
// and otherwise enqueues its kernel(s) on the caller's stream and returns without
// synchronizing.  No call allocates memory.

#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "mxq.h"
#include "mxq_launch.h"

namespace {

thread_local char g_last_cuda_error[256] = "";

// The runtime keeps a refused call's error for this thread until it is read, and the launches
// that end in cudaGetLastError() would report it for a later, correct call: read it here.
int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MXQ_OK;
    (void)cudaGetLastError();
    std::strncpy(g_last_cuda_error, cudaGetErrorString(e), sizeof(g_last_cuda_error) - 1);
    g_last_cuda_error[sizeof(g_last_cuda_error) - 1] = '\0';
    return MXQ_ERR_CUDA;
}

// The status of a diagnostic read that failed.
int failed_read() {
    cuda_status(cudaPeekAtLastError());
    return MXQ_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// a * b * c without int64 overflow (all non-negative)
bool mul_ok(int64_t a, int64_t b, int64_t c, int64_t* out) {
    const int64_t lim = INT64_MAX / 4;  // keep byte offsets of 2-byte elements in range
    if (a != 0 && b > lim / a) return false;
    const int64_t ab = a * b;
    if (ab != 0 && c > lim / ab) return false;
    *out = ab * c;
    return true;
}

bool route_args_ok(int type, int score, float scale) {
    return (type == MXQ_TYPE_BF16 || type == MXQ_TYPE_F32) &&
           (score == MXQ_SCORE_SOFTMAX || score == MXQ_SCORE_SIGMOID) && std::isfinite(scale);
}

bool route_shape_ok(int64_t T, int64_t E, int32_t k) {
    int64_t n = 0;
    return T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= 32 && k <= E && mul_ok(T, E, 4, &n);
}

bool norm_shape_ok(int64_t M, int64_t D) {
    int64_t n = 0;
    return M >= 0 && D >= 0 && D % 32 == 0 && D <= 16384 && mul_ok(M, D, 1, &n);
}

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

namespace mxq {

int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 0 || dev >= 64) return 148;
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cached[dev] = n;
    }
    return cached[dev];
}

}  // namespace mxq

extern "C" {

int mx_quantize(const void* x_bf16, int64_t batch, int64_t rows, int64_t cols, int axes,
                uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, void* stream) {
    if (axes < 1 || axes > 3) return MXQ_ERR_ARG;
    if (batch < 0 || rows < 0 || cols < 0) return MXQ_ERR_SHAPE;
    const bool do_row = (axes & MXQ_AXIS_ROW) != 0, do_col = (axes & MXQ_AXIS_COL) != 0;
    if (cols % 32 != 0 || (do_col && rows % 32 != 0)) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(batch, rows, cols, &n)) return MXQ_ERR_SHAPE;
    if (n == 0) return MXQ_OK;  // empty tensors may carry NULL data pointers
    if (!x_bf16) return MXQ_ERR_NULL;
    if (do_row && (!q_row || !s_row)) return MXQ_ERR_NULL;
    if (do_col && (!q_col || !s_col)) return MXQ_ERR_NULL;
    if (!aligned(x_bf16, 16)) return MXQ_ERR_ALIGN;
    if (do_row && !aligned(q_row, 16)) return MXQ_ERR_ALIGN;
    if (do_col && !aligned(q_col, 16)) return MXQ_ERR_ALIGN;
    const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
    cudaError_t e;
    if (do_row && !do_col)
        e = mxq::launch_quant_rows(x, q_row, s_row, n / 32, as_stream(stream));
    else
        e = mxq::launch_quant_tile(x, batch, rows, cols, do_row, do_col, q_row, s_row, q_col, s_col,
                                   as_stream(stream));
    return cuda_status(e);
}

int mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t batch, int64_t rows, int64_t cols,
                  int axis, void* y_bf16, void* stream) {
    if (axis != MXQ_AXIS_ROW && axis != MXQ_AXIS_COL) return MXQ_ERR_ARG;
    if (batch < 0 || rows < 0 || cols < 0) return MXQ_ERR_SHAPE;
    if (cols % 32 != 0 || (axis == MXQ_AXIS_COL && rows % 32 != 0)) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(batch, rows, cols, &n)) return MXQ_ERR_SHAPE;
    if (n == 0) return MXQ_OK;  // empty tensors may carry NULL data pointers
    if (!q || !s || !y_bf16) return MXQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(y_bf16, 16)) return MXQ_ERR_ALIGN;
    uint16_t* y = static_cast<uint16_t*>(y_bf16);
    cudaError_t e = axis == MXQ_AXIS_ROW
                        ? mxq::launch_dequant_rows(q, s, y, n, as_stream(stream))
                        : mxq::launch_dequant_tile(q, s, batch, rows, cols, y, as_stream(stream));
    return cuda_status(e);
}

int fp8_per_group_rowwise_quant(const void* x_bf16, int64_t M, int64_t K, const int32_t* offs,
                                int32_t G, int out_layout, uint8_t* q, float* scales,
                                void* stream) {
    if (out_layout != MXQ_LAYOUT_ROW_MAJOR && out_layout != MXQ_LAYOUT_COL_MAJOR) return MXQ_ERR_ARG;
    if (M < 0 || K < 0 || G < 0) return MXQ_ERR_SHAPE;
    if (K % 8 != 0 || G > 65535) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(M, K, 1, &n)) return MXQ_ERR_SHAPE;
    if (K == 0 || G == 0) return MXQ_OK;
    if (!offs || !scales) return MXQ_ERR_NULL;
    if (M > 0 && (!x_bf16 || !q)) return MXQ_ERR_NULL;
    if (!aligned(offs, 4) || !aligned(scales, 4)) return MXQ_ERR_ALIGN;
    if (M > 0 && (!aligned(x_bf16, 16) || !aligned(q, 16))) return MXQ_ERR_ALIGN;
    cudaError_t e = mxq::launch_per_group(static_cast<const uint16_t*>(x_bf16), M, K, offs, G,
                                          out_layout == MXQ_LAYOUT_COL_MAJOR, q, scales,
                                          as_stream(stream));
    return cuda_status(e);
}

int fp8_per_group_rowwise_quant_batched(const void* x_bf16, int64_t E, int64_t M, int64_t K, int out_layout,
                                        uint8_t* q, float* scales, void* stream) {
    if (out_layout != MXQ_LAYOUT_ROW_MAJOR && out_layout != MXQ_LAYOUT_COL_MAJOR) return MXQ_ERR_ARG;
    if (E < 0 || M < 0 || K < 0) return MXQ_ERR_SHAPE;
    if (K % 8 != 0 || E > 65535) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(E, M, K, &n) || E * M > 0x7FFFFFFFLL) return MXQ_ERR_SHAPE;
    if (K == 0 || E == 0) return MXQ_OK;
    if (!scales) return MXQ_ERR_NULL;
    if (M > 0 && (!x_bf16 || !q)) return MXQ_ERR_NULL;
    if (!aligned(scales, 4)) return MXQ_ERR_ALIGN;
    if (M > 0 && (!aligned(x_bf16, 16) || !aligned(q, 16))) return MXQ_ERR_ALIGN;
    if (M == 0) {  // every matrix empty: only the scales, 448 / fp32(1e-12)
        cudaError_t e = mxq::launch_per_group(nullptr, 0, K, nullptr, (int32_t)E, false, nullptr, scales,
                                              as_stream(stream), 1);
        return cuda_status(e);
    }
    cudaError_t e = mxq::launch_per_group(static_cast<const uint16_t*>(x_bf16), E * M, K, nullptr, (int32_t)E,
                                          out_layout == MXQ_LAYOUT_COL_MAJOR, q, scales, as_stream(stream),
                                          (int)M);
    return cuda_status(e);
}

int fp8_per_group_rowwise_plan(int64_t M, int64_t K, int32_t G, int out_layout, int n_sm, int* kernel,
                               int* slab_cols, int* cluster, int* tile_rows, int* threads) {
    if (!kernel || !slab_cols || !cluster || !tile_rows || !threads) return MXQ_ERR_NULL;
    if (out_layout != MXQ_LAYOUT_ROW_MAJOR && out_layout != MXQ_LAYOUT_COL_MAJOR) return MXQ_ERR_ARG;
    if (M < 0 || K < 0 || G < 0 || n_sm < 0) return MXQ_ERR_SHAPE;
    if (K % 8 != 0 || G > 65535) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(M, K, 1, &n)) return MXQ_ERR_SHAPE;
    if (n_sm == 0) {
        n_sm = mxq::sm_count();
        if (n_sm <= 0) return MXQ_ERR_CUDA;
    }
    const mxq::PerGroupPlan p = mxq::plan_per_group(M, K, G, out_layout == MXQ_LAYOUT_COL_MAJOR, n_sm);
    *kernel = p.kind;
    *slab_cols = p.w;
    *cluster = p.cl;
    *tile_rows = p.r_cap;
    *threads = p.threads;
    return MXQ_OK;
}

int mxq_transpose_u8(const uint8_t* src, int64_t batch, int64_t rows, int64_t cols, uint8_t* dst, void* stream) {
    if (batch < 0 || rows < 0 || cols < 0) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(batch, rows, cols, &n)) return MXQ_ERR_SHAPE;
    if (n == 0) return MXQ_OK;
    if (!src || !dst) return MXQ_ERR_NULL;
    return cuda_status(mxq::launch_transpose_u8(src, batch, rows, cols, dst, as_stream(stream)));
}

int64_t mx_scales_blocked_bytes(int64_t batch, int64_t rows, int64_t n_k, int32_t G) {
    if (batch < 0 || rows < 0 || n_k < 0 || G < 0 || (G > 0 && batch != 1)) return -1;
    int64_t n = 0;
    if (!mul_ok(batch, rows + 128 * (int64_t)G + 128, n_k + 4, &n)) return -1;
    return mxq::scales_blocked_bytes(batch, rows, n_k, G);
}

int mx_scales_to_blocked(const uint8_t* s, int64_t batch, int64_t rows, int64_t n_k, const int32_t* offs,
                         int32_t G, uint8_t* out, void* stream) {
    if (batch < 0 || rows < 0 || n_k < 0 || G < 0) return MXQ_ERR_SHAPE;
    if (G > 0 && batch != 1) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(batch, rows + 128 * (int64_t)G + 128, n_k + 4, &n)) return MXQ_ERR_SHAPE;
    if (n_k == 0 || batch == 0 || (G == 0 && rows == 0)) return MXQ_OK;
    if (G > 0 && !offs) return MXQ_ERR_NULL;
    if (!out || (rows > 0 && !s)) return MXQ_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(out) & 15) != 0) return MXQ_ERR_ALIGN;
    if (G > 0 && (reinterpret_cast<uintptr_t>(offs) & 3) != 0) return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_scales_to_blocked(s, batch, rows, n_k, offs, G, out, as_stream(stream)));
}

int mx_grouped_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                    const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* out_bf16, void* stream) {
    if (M < 0 || N < 0 || K < 0 || G < 0) return MXQ_ERR_SHAPE;
    if (K % 128 != 0 || N % 256 != 0 || G > 65535) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(M + 128 * (int64_t)G, N + K, 1, &n) || !mul_ok(G, N, K, &n)) return MXQ_ERR_SHAPE;
    if (M == 0 || N == 0 || K == 0 || G == 0) return MXQ_OK;
    if (!qa || !sfa || !qb || !sfb || !offs || !out_bf16) return MXQ_ERR_NULL;
    if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) || !aligned(out_bf16, 16) ||
        !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_mx_grouped_gemm(qa, sfa, qb, sfb, offs, G, M, N, K,
                                                   static_cast<uint16_t*>(out_bf16), as_stream(stream)));
}

int moe_route(const void* logits, int type, int64_t T, int64_t E, const float* bias, int score, int32_t n_groups,
              int32_t top_groups, int32_t group_top, int32_t k, int renorm, float scale, float* weights,
              int32_t* ids, void* stream) {
    if (!route_args_ok(type, score, scale)) return MXQ_ERR_ARG;
    if (n_groups < 1 || n_groups > 32 || top_groups < 1 || top_groups > n_groups || group_top < 1 || group_top > 2)
        return MXQ_ERR_ARG;
    if (!route_shape_ok(T, E, k) || E % n_groups != 0) return MXQ_ERR_SHAPE;
    if (T == 0) return MXQ_OK;
    if (!logits || !weights || !ids) return MXQ_ERR_NULL;
    const uintptr_t size = type == MXQ_TYPE_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(ids, 4)) return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_moe_route(logits, type == MXQ_TYPE_BF16, T, (int)E, bias, score, n_groups,
                                             top_groups, group_top, k, renorm != 0, scale, weights, ids,
                                             as_stream(stream)));
}

int moe_route_backward(const void* logits, int type, int64_t T, int64_t E, const int32_t* ids, int32_t k,
                       const float* grad_weights, int score, int renorm, float scale, void* grad_logits,
                       void* stream) {
    if (!route_args_ok(type, score, scale)) return MXQ_ERR_ARG;
    if (!route_shape_ok(T, E, k)) return MXQ_ERR_SHAPE;
    if (T == 0) return MXQ_OK;
    if (!logits || !ids || !grad_weights || !grad_logits) return MXQ_ERR_NULL;
    const uintptr_t size = type == MXQ_TYPE_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(ids, 4) || !aligned(grad_weights, 4) || !aligned(grad_logits, size))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_moe_route_backward(logits, type == MXQ_TYPE_BF16, T, (int)E, ids, k, grad_weights,
                                                      score, renorm != 0, scale, grad_logits, as_stream(stream)));
}

int64_t moe_plan_workspace_bytes(int64_t n, int64_t E) {
    if (n < 0 || n > 0x7FFFFFFFLL || E < 1 || E > 1024) return -1;
    return mxq::plan_workspace_bytes(n, (int)E);
}

int moe_plan(const int32_t* ids, int64_t n, int64_t E, int32_t* offs, int32_t* rows, int32_t* src, void* workspace,
             void* stream) {
    const int64_t need = moe_plan_workspace_bytes(n, E);
    if (need < 0) return MXQ_ERR_SHAPE;
    if (!offs || (n > 0 && (!ids || !rows || !src)) || (need > 0 && !workspace)) return MXQ_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(offs, 4) || !aligned(rows, 4) || !aligned(src, 4) || !aligned(workspace, 4))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_moe_plan(ids, n, (int)E, offs, rows, src, static_cast<int32_t*>(workspace),
                                            as_stream(stream)));
}

int rmsnorm_mx_quantize(const void* x_bf16, const void* residual_bf16, const void* weight, int weight_type,
                        int64_t M, int64_t D, float eps, void* res_out_bf16, void* y_bf16, uint8_t* q, uint8_t* s,
                        float* rstd, void* stream) {
    if ((weight_type != MXQ_TYPE_BF16 && weight_type != MXQ_TYPE_F32) || !(eps > 0.0f) || std::isinf(eps))
        return MXQ_ERR_ARG;
    if (!norm_shape_ok(M, D)) return MXQ_ERR_SHAPE;
    if (M == 0 || D == 0) return MXQ_OK;
    if (!x_bf16 || !weight || !q || !s) return MXQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(weight, 16) || !aligned(res_out_bf16, 16) ||
        !aligned(y_bf16, 16) || !aligned(q, 16) || !aligned(rstd, 4))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_rmsnorm_mx(
        static_cast<const uint16_t*>(x_bf16), static_cast<const uint16_t*>(residual_bf16), weight,
        weight_type == MXQ_TYPE_BF16, M, (int)D, eps, static_cast<uint16_t*>(res_out_bf16),
        static_cast<uint16_t*>(y_bf16), q, s, rstd, as_stream(stream)));
}

int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t D) {
    return norm_shape_ok(M, D) ? mxq::rmsnorm_workspace_bytes(M, D) : -1;
}

int rmsnorm_backward(const void* grad_y_bf16, const void* h_bf16, const void* weight, int weight_type,
                     const float* rstd, const void* grad_res_bf16, int64_t M, int64_t D, void* grad_x_bf16,
                     float* grad_weight, void* workspace, void* stream) {
    if (weight_type != MXQ_TYPE_BF16 && weight_type != MXQ_TYPE_F32) return MXQ_ERR_ARG;
    if (!norm_shape_ok(M, D)) return MXQ_ERR_SHAPE;
    if (D == 0) return MXQ_OK;
    if (!grad_weight) return MXQ_ERR_NULL;
    if (M > 0 && (!grad_y_bf16 || !h_bf16 || !weight || !rstd || !grad_x_bf16 || !workspace)) return MXQ_ERR_NULL;
    if (!aligned(grad_y_bf16, 16) || !aligned(h_bf16, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
        !aligned(grad_res_bf16, 16) || !aligned(grad_x_bf16, 16) || !aligned(grad_weight, 16) ||
        !aligned(workspace, 16))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_rmsnorm_backward(
        static_cast<const uint16_t*>(grad_y_bf16), static_cast<const uint16_t*>(h_bf16), weight,
        weight_type == MXQ_TYPE_BF16, rstd, static_cast<const uint16_t*>(grad_res_bf16), M, (int)D,
        static_cast<uint16_t*>(grad_x_bf16), grad_weight, static_cast<float*>(workspace), as_stream(stream)));
}

int mxfp4_quantize(const void* x_bf16, int64_t batch, int64_t rows, int64_t cols, uint8_t* q, uint8_t* s,
                   uint8_t* sf_blocked, const int32_t* offs, int32_t G, void* stream) {
    if (batch < 0 || rows < 0 || cols < 0 || G < 0 || cols % 32 != 0 || (G > 0 && batch != 1)) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(batch, rows, cols, &n) || rows > INT64_MAX / 4 ||
        !mul_ok(batch, rows + 128 * (int64_t)G + 128, cols / 32 + 4, &n))
        return MXQ_ERR_SHAPE;
    if (batch == 0 || rows == 0 || cols == 0) return MXQ_OK;
    if (!x_bf16 || !q || (!s && !sf_blocked) || (G > 0 && (!offs || !sf_blocked))) return MXQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(sf_blocked, 16) || !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_f4_quant(static_cast<const uint16_t*>(x_bf16), batch, rows, cols, q, s, sf_blocked,
                                            offs, G, as_stream(stream)));
}

int mxfp4_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols, void* y_bf16, void* stream) {
    if (rows < 0 || cols < 0 || cols % 32 != 0) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(rows, cols, 1, &n)) return MXQ_ERR_SHAPE;
    if (n == 0) return MXQ_OK;
    if (!q || !s || !y_bf16) return MXQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(y_bf16, 16)) return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_f4_dequant(q, s, static_cast<uint16_t*>(y_bf16), n, as_stream(stream)));
}

int mxfp4_grouped_gemm(const uint8_t* qa, const uint8_t* sfa, const uint8_t* qb, const uint8_t* sfb,
                       const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* out_bf16, void* stream) {
    if (M < 0 || N < 0 || K < 0 || G < 0) return MXQ_ERR_SHAPE;
    if (K % 128 != 0 || N % 256 != 0 || G > 65535 || M > 0x7FFFFFFFLL) return MXQ_ERR_SHAPE;
    int64_t n = 0;
    if (!mul_ok(M + 128 * (int64_t)G, N, 1, &n) || !mul_ok(M + 128 * (int64_t)G, K, 1, &n) || !mul_ok(G, N, K, &n))
        return MXQ_ERR_SHAPE;
    if (M == 0 || N == 0 || K == 0 || G == 0) return MXQ_OK;
    if (!qa || !sfa || !qb || !sfb || !offs || !out_bf16) return MXQ_ERR_NULL;
    if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) || !aligned(out_bf16, 16) ||
        !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_mxfp4_grouped_gemm(qa, sfa, qb, sfb, offs, G, M, N, K,
                                                      static_cast<uint16_t*>(out_bf16), as_stream(stream)));
}

int mx_e4m3_encode_f32(const float* x, int64_t n, uint8_t* q, void* stream) {
    if (n < 0) return MXQ_ERR_SHAPE;
    if (n == 0) return MXQ_OK;
    if (!x || !q) return MXQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16)) return MXQ_ERR_ALIGN;
    return cuda_status(mxq::launch_encode_f32(x, q, n, as_stream(stream)));
}

const char* mxq_status_string(int status) {
    switch (status) {
        case MXQ_OK: return "MXQ_OK";
        case MXQ_ERR_NULL: return "MXQ_ERR_NULL: a required pointer is NULL";
        case MXQ_ERR_SHAPE: return "MXQ_ERR_SHAPE: invalid sizes for this layout";
        case MXQ_ERR_ALIGN: return "MXQ_ERR_ALIGN: pointer alignment rule violated";
        case MXQ_ERR_ARG: return "MXQ_ERR_ARG: enum argument out of range";
        case MXQ_ERR_CUDA: return "MXQ_ERR_CUDA: the CUDA runtime rejected a launch";
        case MXQ_ERR_NOT_IMPLEMENTED: return "MXQ_ERR_NOT_IMPLEMENTED";
        default: return "unknown mxq status";
    }
}

const char* mxq_last_cuda_error(void) { return g_last_cuda_error; }

int mxq_wait_timeouts(unsigned int* count) {
    if (!count) return MXQ_ERR_NULL;
    const unsigned int n = mxq::read_wait_timeouts(), m = mxq::read_gemm_timeouts(),
                       f = mxq::read_f4_gemm_timeouts(), r = mxq::read_norm_timeouts();
    if (n == 0xFFFFFFFFu || m == 0xFFFFFFFFu || f == 0xFFFFFFFFu || r == 0xFFFFFFFFu)
        return failed_read();
    *count = n + m + f + r;
    return MXQ_OK;
}

int mxq_wait_abandoned(unsigned int* count) {
    if (!count) return MXQ_ERR_NULL;
    const unsigned int n = mxq::read_wait_abandoned();
    if (n == 0xFFFFFFFFu) return failed_read();
    *count = n;
    return MXQ_OK;
}

int mxq_set_wait_limit_ns(uint64_t ns) {
    mxq::set_wait_limit_ns(ns);
    return MXQ_OK;
}

}  // extern "C"
