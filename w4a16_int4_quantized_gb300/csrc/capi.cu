// capi.cu -- the extern "C" boundary of libw4gb300 (declared in include/w4.h).
//
// Host-side validation happens here, before anything is launched or read,
// in the order the header documents; then each call is routed to one CUDA
// path: the quantizers, the decode GEMV (M <= 16), the tcgen05 prefill GEMM
// (M > 16, shapes it can tile) or the generic kernel (anything else).  There
// is no CPU fallback: every result comes from a kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "w4.h"
#include "common.cuh"
#include "internal.h"

namespace {

__device__ uint32_t g_status_word;

thread_local int32_t t_last_cuda_error = 0;

w4_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return W4_OK;
    t_last_cuda_error = (int32_t)e;
    return W4_ECUDA;
}

// Device address of the status word on the current device (resolved once per device).
cudaError_t status_ptr(uint32_t **out) {
    constexpr int kMaxDev = 64;
    static std::atomic<uint32_t *> cache[kMaxDev];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    uint32_t *p = cache[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lk(mu);
        p = cache[dev].load(std::memory_order_relaxed);
        if (!p) {
            void *addr = nullptr;
            e = cudaGetSymbolAddress(&addr, g_status_word);
            if (e != cudaSuccess) return e;
            p = static_cast<uint32_t *>(addr);
            cache[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return cudaSuccess;
}

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

constexpr int64_t kMaxKQ4 = 1000000;        // |sum xq*u| < 2^31 needs K <= 1,127,288
constexpr int64_t kMaxKQ8 = 131072;         // |sum xq*w| < 2^31 for any int8 weights needs K <= 133,144
constexpr int64_t kMaxKDot = 1127288;
constexpr int64_t kMaxDim = (int64_t)1 << 31;

w4_status run_linear(w4::LinearArgs &a, cudaStream_t st) {
    uint32_t *status = nullptr;
    cudaError_t e = status_ptr(&status);
    if (e != cudaSuccess) return cuda_status(e);
    a.status = status;
    if (a.M <= 16 && w4::gemv_supported(a)) return cuda_status(w4::launch_gemv(a, st));
    if (a.M > 16 && w4::gemm_supported(a)) return cuda_status(w4::launch_gemm(a, st));
    // M > 16 shapes the tensor-core GEMM does not take (interleaved layout,
    // odd K, W8A8 with K > 1024): slices of 16 activation rows through the
    // decode kernel, which handles them exactly.
    w4::LinearArgs s16 = a;
    s16.M = 16;
    if (a.M > 16 && w4::gemv_supported(s16)) {
        const size_t xrow = (size_t)a.K * (a.kind == w4::KIND_W4A16 ? 2 : a.kind == w4::KIND_W8A16 ? 4 : 1);
        for (int64_t m0 = 0; m0 < a.M; m0 += 16) {
            w4::LinearArgs sl = a;
            sl.M = std::min<int64_t>(16, a.M - m0);
            sl.x = static_cast<const uint8_t *>(a.x) + (size_t)m0 * xrow;
            sl.sx = a.sx ? a.sx + m0 : nullptr;
            sl.y = a.y + (size_t)m0 * a.N;
            sl.flags = 0;
            const cudaError_t e = w4::launch_gemv(sl, st);
            if (e != cudaSuccess) return cuda_status(e);
        }
        return W4_OK;
    }
    return cuda_status(w4::launch_generic(a, st));
}

w4_status check_workspace(int32_t op, int64_t M, int64_t N, int64_t K, int64_t G, void *ws, size_t ws_bytes) {
    const size_t need = w4_workspace_bytes(op, M, N, K, G);
    if (need > ws_bytes) return W4_EINVAL;
    if (need > 0 && ws == nullptr) return W4_EINVAL;
    return W4_OK;
}

bool type_ok(int32_t t) { return t == W4_F32 || t == W4_BF16 || t == W4_F16; }
int64_t type_bytes(int32_t t) { return t == W4_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The linears on MXFP4 weights: x bf16, or (xq, sx) in MXFP4.
w4_status run_mxfp4(const uint16_t *x, const uint8_t *xq, const uint8_t *sx, const uint8_t *w, const uint8_t *sw,
                    void *y, int32_t y_type, int64_t M, int64_t N, int64_t K, uint32_t flags, bool a4, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(y_type) || (flags & ~(uint32_t)W4_FLAG_PDL)) return W4_EINVAL;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || !aligned(y, type_bytes(y_type))) return W4_EINVAL;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N * type_bytes(y_type)), as_stream(stream)));
    if (!w || !sw || (a4 ? !xq || !sx : !x)) return W4_EINVAL;
    if (!aligned(w, 16) || !aligned(a4 ? (const void *)xq : (const void *)x, 16)) return W4_EINVAL;
    // Few rows of x: the kernel that decodes, unless W is so high that the 4-bit product with
    // its tile of 128 rows is done first.  K moves the crossing little.  In us, decoded / 4-bit
    // product, W from memory, at K = 256, 2048 and 8192:
    //   M = 16, N =  4864  3.1 / 3.4    5.5 / 6.2   13.1 / 14.6
    //           N =  9728  3.8 / 3.7    7.8 / 7.6   21.5 / 20.1
    //           N = 13312  4.6 / 3.8   10.4 / 7.8   31.6 / 22.5
    //   M =  8, N = 13312  3.6 / 3.8    7.9 / 7.7   22.9 / 23.3
    //           N = 26624  6.0 / 5.0   13.7 / 10.5  42.0 / 28.7
    // (the widest miss: M = 16, N = 7168, 12.0 / 10.5 at K = 4096, 5.0 / 5.2 at 1024).
    if (!a4 || M <= (N > 2 * 9728 ? 0 : N > 9728 ? 8 : 16))
        return cuda_status(w4::launch_mxfp4_decode(x, xq, sx, w, sw, y, y_type, M, N, K, flags, as_stream(stream)));
    uint32_t *status = nullptr;
    const cudaError_t e = status_ptr(&status);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(w4::launch_mxfp4_gemm(xq, sx, w, sw, y, y_type, M, N, K, status, as_stream(stream)));
}

// A cache that the kernels can address (its pointers are looked at by the callers).
w4_status check_cache(const w4_paged_cache *c, bool f32_too) {
    if (!c || !type_ok(c->type) || (c->type == W4_F32 && !f32_too)) return W4_EINVAL;
    if (c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1) return W4_EINVAL;
    if (c->pages >= kMaxDim || c->head_dim % 8 || c->head_dim > 256) return W4_ESHAPE;
    const int64_t el = type_bytes(c->type);
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
        if (s < 0 || s * el % 16) return W4_EINVAL;
    return W4_OK;
}

// An 8-bit cache that the kernels can address (its pointers are looked at by the callers).
w4_status check_kv8(const w4_kv8_cache *c) {
    if (!c || c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1 || c->reserved != 0) return W4_EINVAL;
    if (c->pages >= kMaxDim || c->head_dim % 16 || c->head_dim > 256) return W4_ESHAPE;
    if (c->page_size < W4_KV8_BLOCK || (c->page_size & (c->page_size - 1)) || c->heads >= (1 << 20)) return W4_ESHAPE;
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
        if (s < 0 || s % 16) return W4_EINVAL;
    return W4_OK;
}

bool kv8_pointers(const w4_kv8_cache *c) {
    return c->k && c->v && c->k_scale && c->v_scale && aligned(c->k, 16) && aligned(c->v, 16);
}

}  // namespace

namespace w4 {
w4_status record_cuda_error(cudaError_t e) { return cuda_status(e); }
}  // namespace w4

extern "C" {

w4_status w4_quantize_row_q8(const float *x, int64_t M, int64_t K, int8_t *q, float *sx, int32_t *rowsum,
                             void *stream) {
    if (M < 0 || K < 0) return W4_EINVAL;
    if (M >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (M == 0) return W4_OK;
    if (!sx || (K > 0 && (!x || !q))) return W4_EINVAL;
    return cuda_status(w4::launch_quantize_rows(x, M, K, 127, q, sx, rowsum, as_stream(stream)));
}

w4_status w4_quantize_matrix_q4(const float *W, int64_t N, int64_t K, uint8_t *packed, float *sw, void *stream) {
    if (N < 0 || K < 0) return W4_EINVAL;
    if (N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (N == 0) return W4_OK;
    if (!sw || (K > 0 && (!W || !packed))) return W4_EINVAL;
    return cuda_status(w4::launch_quantize_matrix_q4(W, N, K, packed, sw, as_stream(stream)));
}

w4_status w4_quantize_matrix_q8(const float *W, int64_t N, int64_t K, int8_t *q, float *sw, void *stream) {
    if (N < 0 || K < 0) return W4_EINVAL;
    if (N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (N == 0) return W4_OK;
    if (!sw || (K > 0 && (!W || !q))) return W4_EINVAL;
    return cuda_status(w4::launch_quantize_rows(W, N, K, 127, q, sw, nullptr, as_stream(stream)));
}

w4_status w4_dot_i32_q4(const int8_t *xq, const uint8_t *wrow, int64_t K, int32_t *out, void *stream) {
    if (K < 0) return W4_EINVAL;
    if (K > kMaxKDot) return W4_ESHAPE;
    if (!out || (K > 0 && (!xq || !wrow))) return W4_EINVAL;
    if (K == 0) return cuda_status(cudaMemsetAsync(out, 0, sizeof(int32_t), as_stream(stream)));
    return cuda_status(w4::launch_dot_i32_q4(xq, wrow, K, out, as_stream(stream)));
}

w4_status w4_linear_q4(const int8_t *xq, const float *sx, const uint8_t *w, const float *sw, float *y, int64_t M,
                       int64_t N, int64_t K, int32_t layout, void *workspace, size_t ws_bytes, uint32_t flags,
                       void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (layout != W4_LAYOUT_ROWMAJOR && layout != W4_LAYOUT_N64) return W4_EINVAL;
    if (K > kMaxKQ4 || M >= kMaxDim || N >= kMaxDim) return W4_ESHAPE;
    if (layout == W4_LAYOUT_N64 && N % 64) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || !sx || !sw || (K > 0 && (!xq || !w))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_Q4, M, N, K, 0, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), as_stream(stream)));
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W4A8;
    a.x = xq; a.w = w; a.scale = sw; a.sx = sx; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = 0; a.layout = layout; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    return run_linear(a, as_stream(stream));
}

w4_status w4_linear_q4_f32(const float *x, const uint8_t *w, const float *sw, float *y, int8_t *xq, float *sx,
                           int64_t M, int64_t N, int64_t K, int32_t layout, void *workspace, size_t ws_bytes,
                           uint32_t flags, void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (layout != W4_LAYOUT_ROWMAJOR && layout != W4_LAYOUT_N64) return W4_EINVAL;
    if (K > kMaxKQ4 || M >= kMaxDim || N >= kMaxDim) return W4_ESHAPE;
    if (layout == W4_LAYOUT_N64 && N % 64) return W4_ESHAPE;
    if (M == 0) return W4_OK;
    if (!sx || (K > 0 && (!x || !xq))) return W4_EINVAL;
    if (N > 0 && (!y || !sw || (K > 0 && !w))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_Q4, M, N, K, 0, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    cudaStream_t st = as_stream(stream);
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W4A8;
    a.x = xq; a.w = w; a.scale = sw; a.sx = sx; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = 0; a.layout = layout; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    if (N > 0 && K > 0 && M <= 8 && layout == W4_LAYOUT_ROWMAJOR && w4::gemv_supported(a)) {
        uint32_t *status = nullptr;
        const cudaError_t e = status_ptr(&status);
        if (e != cudaSuccess) return cuda_status(e);
        a.status = status;
        a.xf = x; a.xq_out = xq; a.sx_out = sx;
        return cuda_status(w4::launch_gemv(a, st));  // fused, or the quantizer then the linear
    }
    // Prefill on the tensor cores: one pass writes the codes, the scales and
    // the f16 image of the codes the GEMM reads (no separate prepass).
    if (N > 0 && K > 0 && M > 16 && K % 8 == 0 && w4::gemm_supported(a) &&
        reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(xq) % 4 == 0 &&
        reinterpret_cast<uintptr_t>(workspace) % 16 == 0) {
        const cudaError_t e = w4::launch_quantize_rows_f16(x, M, K, xq, sx, static_cast<uint16_t *>(workspace), st);
        if (e != cudaSuccess) return cuda_status(e);
        a.x16_ready = true;
        return run_linear(a, st);
    }
    const cudaError_t e = w4::launch_quantize_rows(x, M, K, 127, xq, sx, nullptr, st);
    if (e != cudaSuccess) return cuda_status(e);
    if (N == 0) return W4_OK;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), st));
    return run_linear(a, st);
}

w4_status w4_linear_q8(const int8_t *xq, const float *sx, const int8_t *w, const float *sw, float *y, int64_t M,
                       int64_t N, int64_t K, void *workspace, size_t ws_bytes, uint32_t flags, void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (K > kMaxKQ8 || M >= kMaxDim || N >= kMaxDim) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || !sx || !sw || (K > 0 && (!xq || !w))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_Q8, M, N, K, 0, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), as_stream(stream)));
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W8A8;
    a.x = xq; a.w = reinterpret_cast<const uint8_t *>(w); a.scale = sw; a.sx = sx; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = 0; a.layout = W4_LAYOUT_ROWMAJOR; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    return run_linear(a, as_stream(stream));
}

w4_status w4_linear_w4a16_group(const uint16_t *x_bf16, const uint8_t *w, const uint16_t *scales_f16, float *y,
                                int64_t M, int64_t N, int64_t K, int64_t G, int32_t layout, void *workspace,
                                size_t ws_bytes, uint32_t flags, void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (layout != W4_LAYOUT_ROWMAJOR && layout != W4_LAYOUT_N64 && layout != W4_LAYOUT_B32) return W4_EINVAL;
    const int64_t Kp = K + (K & 1);
    if (G <= 0 || (G & 1) || (Kp % G) != 0) return W4_ESHAPE;
    if (layout == W4_LAYOUT_B32 && G != 32) return W4_ESHAPE;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (layout == W4_LAYOUT_N64 && N % 64) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || (K > 0 && (!x_bf16 || !w || (layout != W4_LAYOUT_B32 && !scales_f16)))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_W4A16, M, N, K, G, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), as_stream(stream)));
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W4A16;
    a.x = x_bf16; a.w = w; a.scale = scales_f16; a.sx = nullptr; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = G; a.layout = layout; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    return run_linear(a, as_stream(stream));
}

w4_status w4_linear_w8a16(const float *x, const int8_t *w, const float *sw, float *y, int64_t M, int64_t N,
                          int64_t K, void *workspace, size_t ws_bytes, uint32_t flags, void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || !sw || (K > 0 && (!x || !w))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_W8A16, M, N, K, 0, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), as_stream(stream)));
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W8A16;
    a.x = x; a.w = reinterpret_cast<const uint8_t *>(w); a.scale = sw; a.sx = nullptr; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = 0; a.layout = W4_LAYOUT_ROWMAJOR; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    return run_linear(a, as_stream(stream));
}

w4_status w4_linear_q4_group(const int8_t *xq, const float *sx, const uint8_t *w, const uint16_t *scales_f16,
                             const uint8_t *zeros, float *y, int64_t M, int64_t N, int64_t K, int64_t G,
                             int32_t layout, void *workspace, size_t ws_bytes, uint32_t flags, void *stream) {
    if (M < 0 || N < 0 || K < 0) return W4_EINVAL;
    if (layout != W4_LAYOUT_ROWMAJOR && layout != W4_LAYOUT_N64) return W4_EINVAL;
    const int64_t Kp = K + (K & 1);
    if (G <= 0 || (G & 1) || (Kp % G) != 0) return W4_ESHAPE;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (layout == W4_LAYOUT_N64 && N % 64) return W4_ESHAPE;
    if (M == 0 || N == 0) return W4_OK;
    if (!y || !sx || (K > 0 && (!xq || !w || !scales_f16 || !zeros))) return W4_EINVAL;
    const w4_status ws = check_workspace(W4_OP_LINEAR_Q4_GROUP, M, N, K, G, workspace, ws_bytes);
    if (ws != W4_OK) return ws;
    if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, (size_t)(M * N) * sizeof(float), as_stream(stream)));
    w4::LinearArgs a = {};
    a.kind = w4::KIND_W4A8G;
    a.x = xq; a.w = w; a.scale = scales_f16; a.zeros = zeros; a.sx = sx; a.y = y;
    a.M = M; a.N = N; a.K = K; a.G = G; a.layout = layout; a.flags = flags;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    return run_linear(a, as_stream(stream));
}

w4_status w4_add_rmsnorm_q8(const void *x, int32_t x_type, int64_t ld, const void *residual, void *residual_out,
                            int32_t r_type, const float *w, float eps, int64_t T, int64_t H, int8_t *q, float *sx,
                            void *y, int32_t y_type, void *stream) {
    if (T < 0 || H < 0 || !type_ok(x_type) || !type_ok(r_type) || !type_ok(y_type)) return W4_EINVAL;
    if (T >= kMaxDim || H >= kMaxDim || ld >= kMaxDim) return W4_ESHAPE;
    if (T == 0 || H == 0) return W4_OK;
    if (ld < H || !x || !w || !q || !sx || !residual != !residual_out) return W4_EINVAL;
    if (!aligned(x, type_bytes(x_type)) || !aligned(residual, type_bytes(r_type)) ||
        !aligned(residual_out, type_bytes(r_type)) || !aligned(y, type_bytes(y_type)) || !aligned(w, 4) || !aligned(sx, 4))
        return W4_EINVAL;
    return cuda_status(w4::launch_add_rmsnorm_q8(x, x_type, ld, residual, residual_out, r_type, w, eps, T, H, q, sx, y,
                                                 y_type, as_stream(stream)));
}

w4_status w4_qk_norm_rope_kv8(const void *qkv, int32_t x_type, int64_t ld, int64_t T, int32_t q_heads, const float *wq,
                              const float *wk, float eps, const int32_t *positions, const float *cos_sin,
                              int64_t max_pos, int32_t rot, int32_t interleaved, const int32_t *block_table,
                              int64_t width, const int32_t *ctx_len, const int32_t *cu_new, int64_t B,
                              const w4_kv8_cache *cache, void *q_out, int32_t q_type, void *stream) {
    if (T < 0 || B < 0 || width < 0 || q_heads < 1 || rot < 0 || max_pos < 0 || !type_ok(x_type) ||
        (q_type != W4_BF16 && q_type != W4_F16))
        return W4_EINVAL;
    const w4_status c = check_kv8(cache);
    if (c != W4_OK) return c;
    if (T >= kMaxDim || B >= kMaxDim / 4 || width >= kMaxDim || rot % 16 || rot > cache->head_dim) return W4_ESHAPE;
    const int64_t row = (q_heads + 2 * (int64_t)cache->heads) * cache->head_dim;
    if (row >= kMaxDim) return W4_ESHAPE;
    if (T > 0 && B > 0 && w4::kv8_store_ctas(T, B, q_heads, cache->heads, cache->head_dim) >= (1 << 30)) return W4_ESHAPE;
    if (ld < row || ld * type_bytes(x_type) % 16) return W4_EINVAL;
    if (T == 0 || B == 0) return W4_OK;
    if (!qkv || !positions || !q_out || !ctx_len || !cu_new || (width > 0 && !block_table) || (rot > 0 && !cos_sin))
        return W4_EINVAL;
    if (cache->pages > 0 && !kv8_pointers(cache)) return W4_EINVAL;
    for (const void *p : {qkv, (const void *)wq, (const void *)wk, (const void *)cos_sin, (const void *)q_out})
        if (!aligned(p, 16)) return W4_EINVAL;
    return cuda_status(w4::launch_qk_norm_rope_kv8(qkv, x_type, ld, T, q_heads, wq, wk, eps, positions, cos_sin, max_pos,
                                                   rot, interleaved, block_table, width, ctx_len, cu_new, B, *cache, q_out,
                                                   q_type, as_stream(stream)));
}

w4_status w4_dequantize_kv8(const w4_kv8_cache *cache, void *k_out, void *v_out, int32_t type, void *stream) {
    const w4_status c = check_kv8(cache);
    if (c != W4_OK) return c;
    if (!type_ok(type)) return W4_EINVAL;
    if (cache->pages == 0) return W4_OK;
    if (!w4::kv8_read_fits(*cache)) return W4_ESHAPE;
    if (!kv8_pointers(cache) || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return W4_EINVAL;
    return cuda_status(w4::launch_dequantize_kv8(*cache, k_out, v_out, type, as_stream(stream)));
}

// The shapes that attention_kv8 takes, beyond its cache.
static w4_status check_attn8(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len,
                             int64_t max_new, int64_t window, int64_t sinks) {
    if (B < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || max_len < 0 || max_new < 0 || window < 0 || sinks < 0)
        return W4_EINVAL;
    if (head_dim % 16 || head_dim > 256 || q_heads % kv_heads) return W4_ESHAPE;
    for (int64_t n : {max_len, max_new, window, sinks})
        if (n >= kMaxDim - 256) return W4_ESHAPE;
    if (B >= kMaxDim / 4 || (int64_t)q_heads * head_dim >= kMaxDim || max_new * (q_heads / kv_heads) >= kMaxDim - 256)
        return W4_ESHAPE;
    // rows of all requests' tiles: the kernels count tiles and their heads in 32 bits
    int64_t rows = max_new * (q_heads / kv_heads);
    rows = rows <= 32 ? 32 : (rows + 255) / 256 * 256;
    if (B * kv_heads > (kMaxDim - 1) / rows) return W4_ESHAPE;
    return W4_OK;
}

size_t w4_attention_kv8_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len,
                                        int64_t max_new, int64_t window, int64_t sinks) {
    if (check_attn8(B, q_heads, kv_heads, head_dim, max_len, max_new, window, sinks) != W4_OK) return SIZE_MAX;
    if (B == 0 || max_len == 0 || max_new == 0) return 0;
    return w4::attention_kv8_workspace(B, q_heads, kv_heads, head_dim, max_len, max_new, window, sinks);
}

w4_status w4_attention_kv8(const void *q, int32_t q_type, int64_t ld, const w4_kv8_cache *cache,
                           const int32_t *block_table, int64_t width, const int32_t *ctx_len, const int32_t *cu_new,
                           int64_t B, int64_t T, int32_t q_heads, float scale, int64_t max_len, int64_t max_new,
                           int64_t window, int64_t sinks, void *out, void *workspace, size_t ws_bytes, void *stream) {
    w4_status s = check_kv8(cache);
    if (s != W4_OK) return s;
    if (T < 0 || width < 0 || (q_type != W4_BF16 && q_type != W4_F16)) return W4_EINVAL;
    s = check_attn8(B, q_heads, cache->heads, cache->head_dim, max_len, max_new, window, sinks);
    if (s != W4_OK) return s;
    if (T >= kMaxDim || width >= kMaxDim) return W4_ESHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale * w4::kLog2e)) return W4_EINVAL;
    if (ld < (int64_t)q_heads * cache->head_dim || ld % 8) return W4_EINVAL;
    if (B == 0 || T == 0 || max_len == 0 || max_new == 0) return W4_OK;
    if (cache->pages < 1 || width < 1 || !kv8_pointers(cache) || !q || !block_table || !ctx_len || !cu_new || !out)
        return W4_EINVAL;
    for (const void *p : {q, (const void *)out, (const void *)workspace})
        if (!aligned(p, 16)) return W4_EINVAL;
    const size_t need = w4::attention_kv8_workspace(B, q_heads, cache->heads, cache->head_dim, max_len, max_new, window, sinks);
    if (ws_bytes < need || (need > 0 && !workspace)) return W4_EINVAL;
    uint32_t *status = nullptr;
    const cudaError_t e = status_ptr(&status);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(w4::launch_attention_kv8(q, q_type, ld, *cache, block_table, width, ctx_len, cu_new, B, T, q_heads,
                                                scale, max_len, max_new, window, sinks, out, workspace, status,
                                                as_stream(stream)));
}

w4_status w4_token_logprobs(const void *logits, int32_t type, int64_t ld, int64_t T, int64_t V, const int32_t *ids,
                            int32_t top, float *logp, float *entropy, int32_t *top_ids, float *top_logp, void *stream) {
    if (T < 0 || V < 0 || top < 0 || !type_ok(type)) return W4_EINVAL;
    if (T >= kMaxDim || V >= kMaxDim - 16 || top > W4_MAX_TOP) return W4_ESHAPE;
    if (T == 0) return W4_OK;
    if (ld < V || V == 0 || !logits || !ids || !logp || !entropy || (top > 0 && (!top_ids || !top_logp))) return W4_EINVAL;
    if (!aligned(logits, type_bytes(type))) return W4_EINVAL;
    for (const void *p : {(const void *)ids, (const void *)logp, (const void *)entropy, (const void *)top_ids,
                          (const void *)top_logp})
        if (!aligned(p, 4)) return W4_EINVAL;
    return cuda_status(w4::launch_token_logprobs(logits, type, ld, T, V, ids, top, logp, entropy, top_ids, top_logp,
                                                 as_stream(stream)));
}

w4_status w4_pack_interleaved_n64(const uint8_t *w_rowmajor, uint8_t *w_il, int64_t N, int64_t K, void *stream) {
    if (N < 0 || K < 0) return W4_EINVAL;
    if (N % 64) return W4_ESHAPE;
    if (N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (N == 0 || K == 0) return W4_OK;
    if (!w_rowmajor || !w_il) return W4_EINVAL;
    return cuda_status(w4::launch_pack_n64(w_rowmajor, w_il, N, K, as_stream(stream)));
}

static w4_status chain_q4_impl(const float *x0, int32_t K0, const w4_chain_linear *lin, int32_t n_lin, int32_t passes,
                               int32_t pass_output, void *workspace, size_t ws_bytes, void *stream, uint64_t wait_ns,
                               int32_t hold_stage) {
    if (n_lin < 1 || n_lin > W4_CHAIN_MAX_LINEARS || passes < 0 || K0 <= 0 || !lin) return W4_EINVAL;
    if (pass_output < 0 || pass_output >= n_lin) return W4_EINVAL;
    for (int32_t i = 0; i < n_lin; ++i) {
        const w4_chain_linear &L = lin[i];
        if (L.N <= 0 || L.K <= 0 || L.input < -1 || L.input >= i || L.reserved != 0) return W4_EINVAL;
    }
    if (K0 % 32 || K0 > W4_CHAIN_MAX_K) return W4_ESHAPE;
    for (int32_t i = 0; i < n_lin; ++i) {
        const w4_chain_linear &L = lin[i];
        if (L.K % 32 || L.K > W4_CHAIN_MAX_K) return W4_ESHAPE;
        if (L.K != (L.input < 0 ? K0 : lin[L.input].N)) return W4_ESHAPE;
    }
    if (passes > 1 && lin[pass_output].N != K0) return W4_ESHAPE;
    if (!w4::chain_stages_ok(lin, n_lin, passes, pass_output)) return W4_ESHAPE;
    if (passes == 0) return W4_OK;
    auto misaligned = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) != 0; };
    if (!x0 || misaligned(x0)) return W4_EINVAL;
    for (int32_t i = 0; i < n_lin; ++i) {
        const w4_chain_linear &L = lin[i];
        if (!L.w || !L.sw || !L.y || misaligned(L.w) || misaligned(L.y)) return W4_EINVAL;
    }
    if (!workspace || misaligned(workspace) || ws_bytes < w4::chain_workspace_bytes(lin, n_lin, K0))
        return W4_EINVAL;
    uint32_t *status = nullptr;
    cudaError_t e = status_ptr(&status);
    if (e != cudaSuccess) return cuda_status(e);
    const int rc = w4::chain_plan_launch(x0, K0, lin, n_lin, passes, pass_output, workspace, status,
                                         as_stream(stream), &e, wait_ns, hold_stage);
    if (rc == W4_ECUDA) return cuda_status(e);
    return (w4_status)rc;
}

w4_status w4_chain_q4(const float *x0, int32_t K0, const w4_chain_linear *lin, int32_t n_lin, int32_t passes,
                      int32_t pass_output, void *workspace, size_t ws_bytes, void *stream) {
    return chain_q4_impl(x0, K0, lin, n_lin, passes, pass_output, workspace, ws_bytes, stream, w4::kWaitLimitNs, -1);
}

w4_status w4_chain_q4_test_timeout(const float *x0, int32_t K0, const w4_chain_linear *lin, int32_t n_lin,
                                   int32_t passes, int32_t pass_output, void *workspace, size_t ws_bytes,
                                   uint64_t wait_limit_ns, int32_t hold_stage, void *stream) {
    if (wait_limit_ns == 0 || wait_limit_ns > w4::kWaitLimitNs || hold_stage < -1) return W4_EINVAL;
    return chain_q4_impl(x0, K0, lin, n_lin, passes, pass_output, workspace, ws_bytes, stream, wait_limit_ns,
                         hold_stage);
}

w4_status w4_pack_block32(const uint8_t *w_rowmajor, const uint16_t *scales_f16, uint8_t *blocks, int64_t N,
                          int64_t K, void *stream) {
    if (N < 0 || K < 0) return W4_EINVAL;
    if ((K + (K & 1)) % 32) return W4_ESHAPE;
    if (N >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (N == 0 || K == 0) return W4_OK;
    if (!w_rowmajor || !scales_f16 || !blocks) return W4_EINVAL;
    return cuda_status(w4::launch_pack_block32(w_rowmajor, scales_f16, blocks, N, K, as_stream(stream)));
}

w4_status w4_quantize_mxfp4(const void *x, int32_t x_type, int64_t R, int64_t K, uint8_t *codes, uint8_t *scales,
                            void *stream) {
    if (R < 0 || K < 0 || !type_ok(x_type)) return W4_EINVAL;
    if (R >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (R == 0 || K == 0) return W4_OK;
    if (!x || !codes || !scales || !aligned(codes, 16) || !aligned(x, type_bytes(x_type))) return W4_EINVAL;
    return cuda_status(w4::launch_quantize_mxfp4(x, x_type, R, K, codes, scales, as_stream(stream)));
}

w4_status w4_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K, void *y,
                              int32_t y_type, void *stream) {
    if (R < 0 || K < 0 || !type_ok(y_type)) return W4_EINVAL;
    if (R >= kMaxDim || K >= kMaxDim) return W4_ESHAPE;
    if (R == 0 || K == 0) return W4_OK;
    if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(y, type_bytes(y_type))) return W4_EINVAL;
    return cuda_status(w4::launch_dequantize_mxfp4(codes, scales, R, K, y, y_type, as_stream(stream)));
}

w4_status w4_linear_mxfp4(const uint16_t *x_bf16, const uint8_t *w, const uint8_t *sw, void *y, int32_t y_type,
                          int64_t M, int64_t N, int64_t K, uint32_t flags, void *stream) {
    return run_mxfp4(x_bf16, nullptr, nullptr, w, sw, y, y_type, M, N, K, flags, false, stream);
}

w4_status w4_linear_mxfp4_a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, void *y,
                             int32_t y_type, int64_t M, int64_t N, int64_t K, uint32_t flags, void *stream) {
    return run_mxfp4(nullptr, xq, sx, w, sw, y, y_type, M, N, K, flags, true, stream);
}

w4_status w4_draft_plan(const int32_t *ctx_len, const int32_t *new_len, const int32_t *parents,
                        const int32_t *free_pages, int64_t n_free, int32_t *block_table, int64_t B, int64_t width,
                        int32_t page_size, int64_t max_tokens, int32_t *cu_new, int64_t *slots, int32_t *positions,
                        uint32_t *mask, int32_t *taken, void *stream) {
    if (B < 0 || width < 0 || n_free < 0 || max_tokens < 0 || page_size < 1) return W4_EINVAL;
    if (B >= kMaxDim / W4_MAX_DRAFT || width >= kMaxDim || max_tokens >= kMaxDim) return W4_ESHAPE;
    if (!cu_new || !taken || (max_tokens > 0 && (!slots || !positions || !mask)) || !aligned(mask, 16)) return W4_EINVAL;
    if (B > 0 && (!ctx_len || !new_len || (width > 0 && !block_table) || (n_free > 0 && !free_pages))) return W4_EINVAL;
    cudaStream_t st = as_stream(stream);
    if (B == 0) {
        cudaError_t e = cudaMemsetAsync(cu_new, 0, sizeof(int32_t), st);
        if (e == cudaSuccess) e = cudaMemsetAsync(taken, 0, sizeof(int32_t), st);
        if (e == cudaSuccess && max_tokens > 0) e = cudaMemsetAsync(slots, 0xFF, (size_t)max_tokens * 8, st);
        if (e == cudaSuccess && max_tokens > 0) e = cudaMemsetAsync(positions, 0, (size_t)max_tokens * 4, st);
        if (e == cudaSuccess && max_tokens > 0) e = cudaMemsetAsync(mask, 0, (size_t)max_tokens * 16, st);
        return cuda_status(e);
    }
    return cuda_status(w4::launch_draft_plan(ctx_len, new_len, parents, free_pages, n_free, block_table, B, width,
                                             page_size, max_tokens, cu_new, slots, positions, mask, taken, st));
}

w4_status w4_qk_norm_rope(const void *qkv, int32_t x_type, int64_t ld, int64_t T, int32_t q_heads, const float *wq,
                          const float *wk, float eps, const int32_t *positions, const float *cos_sin, int64_t max_pos,
                          int32_t rot, int32_t interleaved, const int64_t *slots, const w4_paged_cache *cache,
                          void *q_out, void *stream) {
    if (T < 0 || q_heads < 1 || rot < 0 || max_pos < 0 || !type_ok(x_type)) return W4_EINVAL;
    const w4_status c = check_cache(cache, true);
    if (c != W4_OK) return c;
    if (T >= kMaxDim || rot % 16 || rot > cache->head_dim) return W4_ESHAPE;
    if ((q_heads + 2 * (int64_t)cache->heads) * cache->head_dim >= kMaxDim) return W4_ESHAPE;
    if (ld < (q_heads + 2 * (int64_t)cache->heads) * cache->head_dim || ld * type_bytes(x_type) % 16) return W4_EINVAL;
    if (T == 0) return W4_OK;
    if (!qkv || !positions || !slots || !q_out || (rot > 0 && !cos_sin)) return W4_EINVAL;
    if (cache->pages > 0 && (!cache->k || !cache->v)) return W4_EINVAL;
    for (const void *p : {qkv, (const void *)wq, (const void *)wk, (const void *)cos_sin, (const void *)q_out,
                          (const void *)cache->k, (const void *)cache->v})
        if (!aligned(p, 16)) return W4_EINVAL;
    return cuda_status(w4::launch_qk_norm_rope(qkv, x_type, ld, T, q_heads, wq, wk, eps, positions, cos_sin, max_pos,
                                               rot, interleaved, slots, *cache, q_out, as_stream(stream)));
}

// The shapes that tree_attention takes, beyond its cache.
static w4_status check_tree(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len,
                            int32_t max_new) {
    if (B < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || max_len < 0 || max_new < 0) return W4_EINVAL;
    if (head_dim % 8 || head_dim > 256 || q_heads % kv_heads || q_heads / kv_heads > 128) return W4_ESHAPE;
    if (B >= kMaxDim / W4_MAX_DRAFT || max_len >= kMaxDim - 256) return W4_ESHAPE;
    return W4_OK;
}

size_t w4_tree_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t max_len, int32_t max_new) {
    if (check_tree(B, q_heads, kv_heads, head_dim, max_len, max_new) != W4_OK) return SIZE_MAX;
    if (B == 0 || max_len == 0 || max_new == 0) return 0;
    return w4::tree_attention_workspace(B, q_heads, kv_heads, head_dim, max_len, std::min(max_new, W4_MAX_DRAFT));
}

w4_status w4_tree_attention(const void *q, int64_t ld, const w4_paged_cache *cache, const int32_t *block_table,
                            int64_t width, const int32_t *ctx_len, const int32_t *cu_new, const uint32_t *mask,
                            int64_t B, int64_t T, int32_t q_heads, float scale, int64_t max_len, int32_t max_new,
                            void *out, void *workspace, size_t ws_bytes, void *stream) {
    w4_status s = check_cache(cache, false);
    if (s != W4_OK) return s;
    if (T < 0 || width < 0) return W4_EINVAL;
    s = check_tree(B, q_heads, cache->heads, cache->head_dim, max_len, max_new);
    if (s != W4_OK) return s;
    if (T >= kMaxDim || width >= kMaxDim || cache->page_size < 8 || (cache->page_size & (cache->page_size - 1)))
        return W4_ESHAPE;
    if (!(scale > 0.0f) || !std::isfinite(scale * w4::kLog2e)) return W4_EINVAL;
    if (ld < (int64_t)q_heads * cache->head_dim || ld % 8) return W4_EINVAL;
    if (B == 0 || T == 0 || max_len == 0 || max_new == 0) return W4_OK;
    if (cache->pages < 1 || width < 1 || !cache->k || !cache->v || !q || !block_table || !ctx_len || !cu_new || !mask ||
        !out)
        return W4_EINVAL;
    for (const void *p : {q, (const void *)cache->k, (const void *)cache->v, (const void *)mask, (const void *)out,
                          (const void *)workspace})
        if (!aligned(p, 16)) return W4_EINVAL;
    max_new = std::min(max_new, W4_MAX_DRAFT);
    const size_t need = w4::tree_attention_workspace(B, q_heads, cache->heads, cache->head_dim, max_len, max_new);
    if (ws_bytes < need || (need > 0 && !workspace)) return W4_EINVAL;
    uint32_t *status = nullptr;
    const cudaError_t e = status_ptr(&status);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(w4::launch_tree_attention(q, ld, *cache, block_table, width, ctx_len, cu_new, mask, B, T, q_heads,
                                                 scale, max_len, max_new, out, workspace, status, as_stream(stream)));
}

size_t w4_chain_workspace_bytes(const w4_chain_linear *lin, int32_t n_lin, int32_t K0) {
    if (!lin || n_lin < 1 || n_lin > W4_CHAIN_MAX_LINEARS || K0 < 0) return 0;
    return w4::chain_workspace_bytes(lin, n_lin, K0);
}

size_t w4_workspace_bytes(int32_t op, int64_t M, int64_t N, int64_t K, int64_t G) {
    if (M <= 16 || N <= 0 || K <= 0) return 0;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return SIZE_MAX;  // beyond every call's limits
    switch (op) {
        case W4_OP_LINEAR_Q4: return w4::gemm_workspace_bytes(w4::KIND_W4A8, M, N, K, G);
        case W4_OP_LINEAR_Q8: return w4::gemm_workspace_bytes(w4::KIND_W8A8, M, N, K, G);
        case W4_OP_LINEAR_W4A16: return w4::gemm_workspace_bytes(w4::KIND_W4A16, M, N, K, G);
        case W4_OP_LINEAR_Q4_GROUP: return w4::gemm_workspace_bytes(w4::KIND_W4A8G, M, N, K, G);
        case W4_OP_LINEAR_W8A16: return w4::gemm_workspace_bytes(w4::KIND_W8A16, M, N, K, G);
        default: return 0;
    }
}

w4_status w4_device_status(uint32_t *out, int32_t clear) {
    if (!out) return W4_EINVAL;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_status_word, sizeof(uint32_t));
    if (e != cudaSuccess) return cuda_status(e);
    if (clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_status_word, &zero, sizeof(uint32_t));
        if (e != cudaSuccess) return cuda_status(e);
    }
    return W4_OK;
}

int32_t w4_last_cuda_error(void) { return t_last_cuda_error; }

const char *w4_status_string(w4_status s) {
    switch (s) {
        case W4_OK: return "W4_OK";
        case W4_EINVAL: return "W4_EINVAL: invalid argument";
        case W4_ESHAPE: return "W4_ESHAPE: shape not supported by the layout";
        case W4_ECUDA: return "W4_ECUDA: CUDA call failed";
        default: return "unknown w4_status";
    }
}

int32_t w4_version(void) { return 100; }

}  // extern "C"
