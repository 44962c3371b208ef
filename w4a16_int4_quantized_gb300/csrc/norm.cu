// norm.cu -- the residual's addition and the RMS norm, with the Q8 rows that the W4A8 linears read.
//
// A CTA to a row: h = x + residual stays in registers (8 values a thread and chunk, four
// chunks; what a longer row has beyond them is read again from the new residual), its sum of
// squares and then the largest |y| are joined over the CTA, and the codes follow.  Every
// value is read and written once: 7 bytes a value with bf16 rows and no y.
// 4,096 rows of 8,192, bf16: 47.4 us, 5.0 TB/s (85 with a division a code and stores between the loads);
// one row of 2,048 2.9 us, a launch; 8,192 rows of 2,048 25.7 us and 1,024 of 16,384 30.5 (17.6 by their bytes: no
// loads while a CTA computes).  Rows that 16-byte accesses cannot take (odd widths) go value by value: 2,048 rows
// of 5,121 39 us, of 5,120 20.  Values next to a tie cost an exact division: with norm weights of 1 and bf16 rows a
// third of the warps have one (6 in 100 with weights about 1), and 4,096 rows of 8,192 take 65 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kHeld = 4;  // chunks of 8 values that a thread holds
constexpr int kMostThreads = 512;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23

struct NormParams {
    const void *x, *res;
    const float *w;
    void *res_out, *y;
    int8_t *q;
    float *sx;
    int64_t ld, H;
    int y_type;
    float eps, inv_h;
};

// The 8 values of a chunk as they lie in memory: one run (VEC), or blockDim.x apart (rows that
// 16-byte accesses cannot take).
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
};
template <typename T, bool VEC>
W4_DEV Raw8<T> get8(const T *row, int64_t at, int64_t H) {
    Raw8<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = *(reinterpret_cast<const uint4 *>(row + at) + i);
    } else {
        uint32_t w[2 * sizeof(T)];
#pragma unroll
        for (int e = 0; e < (int)(2 * sizeof(T)); ++e) w[e] = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t i = at + (int64_t)e * blockDim.x;
            if (i < H) {
                if constexpr (sizeof(T) == 4) w[e] = *reinterpret_cast<const uint32_t *>(row + i);
                else w[e / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(row + i) << (16 * (e & 1));
            }
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    return r;
}
template <typename T>
W4_DEV void unpack8(const Raw8<T> &r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.u[i].x);
            v[4 * i + 1] = __uint_as_float(r.u[i].y);
            v[4 * i + 2] = __uint_as_float(r.u[i].z);
            v[4 * i + 3] = __uint_as_float(r.u[i].w);
        }
    } else {
        Raw4<T> lo, hi;
        lo.r[0] = r.u[0].x; lo.r[1] = r.u[0].y; hi.r[0] = r.u[0].z; hi.r[1] = r.u[0].w;
        unpack4<T>(lo, v);
        unpack4<T>(hi, v + 4);
    }
}

template <typename T, bool VEC>
W4_DEV void put8(T *row, int64_t at, int64_t H, const float (&v)[8]) {
    if constexpr (VEC) {
        if constexpr (sizeof(T) == 4) {
            store4<T>(row + at, v);
            store4<T>(row + at + 4, v + 4);
        } else {
            *reinterpret_cast<uint4 *>(row + at) = make_uint4(pack_pair<T>(v[0], v[1]), pack_pair<T>(v[2], v[3]),
                                                              pack_pair<T>(v[4], v[5]), pack_pair<T>(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t i = at + (int64_t)e * blockDim.x;
            if (i < H) row[i] = from_f32<T>(v[e]);
        }
    }
}

// Where the thread's chunk c begins.
template <bool VEC>
W4_DEV int64_t place(int64_t c, int tid) { return VEC ? 8 * (c * blockDim.x + tid) : 8 * c * blockDim.x + tid; }

// Bits of |v|: as whole numbers they order like the values, and NaN is above infinity.
W4_DEV uint32_t top8(const float (&v)[8], uint32_t top) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return top;
}

template <typename TX, typename TR, bool VEC>
__global__ void __launch_bounds__(kMostThreads, sizeof(TX) + sizeof(TR) > 4 ? 1 : 2) add_rmsnorm_kernel(const NormParams p) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_top[32];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x, H = p.H;
    const TX *x = static_cast<const TX *>(p.x) + row * p.ld;
    const TR *res = p.res ? static_cast<const TR *>(p.res) + row * H : nullptr;
    TR *kept = static_cast<TR *>(p.res_out) + row * H;
    const int64_t chunks = ceil_div(H, 8 * (int64_t)blockDim.x);

    // the sum, as it is kept
    auto sum_of = [&](const Raw8<TX> &xr, const Raw8<TR> &rr, float (&h)[8]) {
        unpack8<TX>(xr, h);
        if (!res) return;
        float r[8];
        unpack8<TR>(rr, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = load_f32(from_f32<TR>(h[e] + r[e]));
    };
    // h again, of a chunk that is not held: this thread wrote it
    auto again = [&](int64_t at, float (&h)[8]) {
        if (res) unpack8<TR>(get8<TR, VEC>(kept, at, H), h);
        else unpack8<TX>(get8<TX, VEC>(x, at, H), h);
    };
    auto square = [](const float (&h)[8], float s) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            a = fmaf(h[e], h[e], a);
            b = fmaf(h[e + 1], h[e + 1], b);
        }
        return s + (a + b);
    };

    float h[kHeld][8], ss = 0.0f;
    Raw8<TX> xr[kHeld] = {};
    Raw8<TR> rr[kHeld] = {};
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int64_t at = place<VEC>(c, tid);
        if (at < H) {
            xr[c] = get8<TX, VEC>(x, at, H);
            if (res) rr[c] = get8<TR, VEC>(res, at, H);
        }
    }
    // (stores after all loads: the new residual may lie where the old one is)
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int64_t at = place<VEC>(c, tid);
        sum_of(xr[c], rr[c], h[c]);
        if (res && at < H) put8<TR, VEC>(kept, at, H, h[c]);
        ss = square(h[c], ss);
    }
    for (int64_t c = kHeld; c < chunks; ++c) {
        const int64_t at = place<VEC>(c, tid);
        float v[8];
        if (at < H) {
            Raw8<TR> r = {};
            if (res) r = get8<TR, VEC>(res, at, H);
            sum_of(get8<TX, VEC>(x, at, H), r, v);
            if (res) put8<TR, VEC>(kept, at, H, v);
            ss = square(v, ss);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    ss = lane < warps ? s_sum[lane] : 0.0f;  // every warp joins the partial sums, in the same order
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rstd = rsqrtf(ss * p.inv_h + p.eps);

    // y = (h rstd) w
    auto scale = [&](int64_t at, float (&v)[8]) {
        float w[8];
        unpack8<float>(get8<float, VEC>(p.w, at, H), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[e];
    };
    uint32_t top = 0u;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int64_t at = place<VEC>(c, tid);
        if (at < H) {
            scale(at, h[c]);
            top = top8(h[c], top);
        }
    }
    for (int64_t c = kHeld; c < chunks; ++c) {
        const int64_t at = place<VEC>(c, tid);
        float v[8];
        if (at < H) {
            again(at, v);
            scale(at, v);
            top = top8(v, top);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
    // a sum of squares beyond f32 gives y = 0 and must not pass for a row of zeros
    const bool fine = isfinite(ss) && top < 0x7F800000u;
    const float sx = fine ? __fdiv_rn(__uint_as_float(top), 127.0f) : __uint_as_float(0x7FC00000u);
    if (tid == 0) p.sx[row] = sx;
    const float r = !fine || sx == 0.0f ? 0.0f : __frcp_rn(sx);
    const bool fast = isfinite(r);

    int8_t *q = p.q + row * H;
    auto finish = [&](int64_t at, const float (&v)[8]) {
        // z = v r + 1.5 * 2^23 has rint(v r) in its low bits; v r lies within 2^-15 of fl(v / sx), so
        // that is its rint too unless v r is within 2^-13 of a half-integer
        uint32_t c[8];
        bool near = !fast;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = fmaf(v[e], r, kMagic);
            near |= fabsf(fmaf(v[e], r, -(z - kMagic))) > 0.5f - 0x1p-13f;
            c[e] = __float_as_uint(z);
        }
        if (near) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                float x = v[0];  // (no address of a register)
#pragma unroll
                for (int i = 1; i < 8; ++i) x = e == i ? v[i] : x;
                const uint32_t code = (uint32_t)q8_code(x, sx, r, fast);
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = e == i ? code : c[i];
            }
        }
        if (!fine) {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = 0u;
        }
        if constexpr (VEC) {
            *reinterpret_cast<uint2 *>(q + at) = make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t i = at + (int64_t)e * blockDim.x;
                if (i < H) q[i] = (int8_t)c[e];
            }
        }
        if (p.y) {
            if (p.y_type == W4_F32) put8<float, VEC>(static_cast<float *>(p.y) + row * H, at, H, v);
            else if (p.y_type == W4_BF16) put8<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16 *>(p.y) + row * H, at, H, v);
            else put8<__half, VEC>(static_cast<__half *>(p.y) + row * H, at, H, v);
        }
    };
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int64_t at = place<VEC>(c, tid);
        if (at < H) finish(at, h[c]);
    }
    for (int64_t c = kHeld; c < chunks; ++c) {
        const int64_t at = place<VEC>(c, tid);
        float v[8];
        if (at < H) {
            again(at, v);
            scale(at, v);
            finish(at, v);
        }
    }
}

template <typename TX, typename TR>
cudaError_t norm_launch(const NormParams &p, bool vec, int64_t T, int threads, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)T, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<TX, TR, true>, p)
               : cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<TX, TR, false>, p);
}

template <typename TX>
cudaError_t norm_launch_r(const NormParams &p, int r_type, bool vec, int64_t T, int threads, cudaStream_t st) {
    switch (r_type) {
        case W4_F32: return norm_launch<TX, float>(p, vec, T, threads, st);
        case W4_BF16: return norm_launch<TX, __nv_bfloat16>(p, vec, T, threads, st);
        default: return norm_launch<TX, __half>(p, vec, T, threads, st);
    }
}

}  // namespace

cudaError_t launch_add_rmsnorm_q8(const void *x, int32_t x_type, int64_t ld, const void *residual, void *residual_out,
                                  int32_t r_type, const float *w, float eps, int64_t T, int64_t H, int8_t *q, float *sx,
                                  void *y, int32_t y_type, cudaStream_t st) {
    NormParams p = {};
    p.x = x; p.res = residual; p.w = w; p.res_out = residual_out; p.y = y; p.q = q; p.sx = sx;
    p.ld = ld; p.H = H; p.y_type = y_type; p.eps = eps; p.inv_h = (float)(1.0 / (double)H);
    auto on = [](const void *a, uintptr_t n) { return reinterpret_cast<uintptr_t>(a) % n == 0; };
    const int64_t el = x_type == W4_F32 ? 4 : 2;
    const bool vec = H % 8 == 0 && on(x, 16) && ld * el % 16 == 0 && on(residual, 16) && on(residual_out, 16) && on(w, 16) &&
                     on(q, 8) && on(y, 16);
    // few rows: a chunk a thread, up to the most threads; with rows for every SM all that a thread holds
    const int64_t need = ceil_div(H, 8), held = T >= 152 ? 4 : 1;
    const int threads = (int)std::min<int64_t>(kMostThreads, round_up(std::max<int64_t>(ceil_div(need, held), 1), 32));
    switch (x_type) {
        case W4_F32: return norm_launch_r<float>(p, r_type, vec, T, threads, st);
        case W4_BF16: return norm_launch_r<__nv_bfloat16>(p, r_type, vec, T, threads, st);
        default: return norm_launch_r<__half>(p, r_type, vec, T, threads, st);
    }
}

}  // namespace w4
