// logprob.cu -- log probabilities of given tokens, the entropy and the top alternatives of rows of logits.
//
// One pass over a row, by 1 to 8 CTAs of a cluster.  With m a running maximum of each lane
// and d = x - m: s = sum exp(d), t = sum d exp(d), from which log p(i) = d_i - log s and the
// entropy is log s - t / s.  Each warp keeps its 32 largest logits in order, one a lane, as
// whole numbers (value, then lowest index), and looks closer at a vector only when one of
// its values reaches the least of the first `top`.  Lists and sums are joined over the
// warps, then over the cluster in shared memory, in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kLpWarps = 16;
constexpr int kLpUnroll = 4;  // vectors of 16 bytes a lane in flight
constexpr int kMaxSplit = 8;
constexpr float kFloor = -1e5f;  // a lower d counts as this: its power is 0, and 0 d must be 0

struct LogpParams {
    const void *x;
    const int32_t *ids;
    float *logp, *entropy, *top_logp;
    int32_t *top_ids;
    int64_t ld;
    int V, top, split;
};

template <typename T>
W4_DEV float lp_value(uint32_t w, int half) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((uint16_t)(half ? w >> 16 : w)));
    else return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
}

W4_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger; NaN if one is.
W4_DEV float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A logit and its index as one number that orders by value, then by lowest index.  0: nothing (NaN).
W4_DEV uint64_t lp_key(float x, int idx) {
    if (!(x == x)) return 0ull;
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 is 0
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (uint64_t)o << 32 | (uint32_t)~idx;
}
W4_DEV float lp_key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// Sorts a bitonic sequence of 32 keys, the largest to lane 0.
W4_DEV uint64_t bitonic_down(uint64_t k, int lane) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
        k = ((lane & o) == 0) == (k > other) ? k : other;
    }
    return k;
}

// The 32 largest of two descending lists, descending.
W4_DEV uint64_t join_lists(uint64_t a, uint64_t b_reversed, int lane) {
    return bitonic_down(a > b_reversed ? a : b_reversed, lane);
}

// The warp's list with the vectors' values that belong into it (v: a vector a lane, of
// which the values [lo, hi) are the row's, the first one's index is idx).  Out of line:
// rare after a row's first vectors.
template <typename T>
__device__ __noinline__ uint64_t take(uint64_t list, uint4 v, int idx, int lo, int hi, int top) {
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
        const int word = sizeof(T) == 4 ? e : e >> 1;
        const uint32_t w = word == 0 ? v.x : word == 1 ? v.y : word == 2 ? v.z : v.w;
        uint64_t key = e >= lo && e < hi ? lp_key(lp_value<T>(w, e & 1), idx + e) : 0ull;
        const uint64_t least = __shfl_sync(0xffffffffu, list, top - 1);
        uint32_t in = __ballot_sync(0xffffffffu, key > least);
        if (__popc(in) > 6) {  // sort the keys, join (250 instructions; one insertion takes about 20)
#pragma unroll
            for (int size = 2; size < 32; size *= 2)
#pragma unroll
                for (int o = size / 2; o; o >>= 1) {
                    const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
                    const bool larger_here = ((lane & o) == 0) != ((lane & size) != 0);
                    key = larger_here == (key > other) ? key : other;
                }
            key = bitonic_down(key, lane);
            list = join_lists(list, __shfl_sync(0xffffffffu, key, 31 - lane), lane);
        } else {
            while (in) {
                const uint64_t k = __shfl_sync(0xffffffffu, key, __ffs(in) - 1);
                in &= in - 1;
                const int at = __popc(__ballot_sync(0xffffffffu, list > k));
                const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
                if (lane == at) list = k;
                else if (lane > at) list = up;
            }
        }
    }
    return list;
}

struct Sums {
    float m, s, t;  // largest logit, sum exp(x - m), sum (x - m) exp(x - m)
};
// What d is taken from: the largest logit, 0 while there is none above -infinity.
W4_DEV float zero_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Moves the sums to another largest logit, not below theirs.
W4_DEV void shift(Sums &a, float m) {
    const float d = max_nan(a.m - zero_of(m), kFloor), f = ex2(d * kLog2e);
    a.t = f * fmaf(a.s, d, a.t);
    a.s *= f;
    a.m = m;
}
W4_DEV void join(Sums &a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    shift(a, m);
    shift(b, m);
    a.s += b.s;
    a.t += b.t;
}

template <typename T>
__global__ void __launch_bounds__(32 * kLpWarps, 2) token_logprobs_kernel(const LogpParams p) {
    constexpr int E = 16 / sizeof(T);
    __shared__ uint64_t s_list[kLpWarps][32];
    __shared__ Sums s_sums[kLpWarps];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / p.split;
    const int rank = (int)(blockIdx.x - row * p.split);
    const T *x = static_cast<const T *>(p.x) + row * p.ld;

    // the row in vectors of 16 aligned bytes: the first one begins `off` values before it
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const uint4 *vec = reinterpret_cast<const uint4 *>(x - off);
    const int64_t n = ceil_div((int64_t)off + p.V, E);
    const int64_t begin = n * rank / p.split, end = n * (rank + 1) / p.split;

    Sums a = {-INFINITY, 0.0f, 0.0f};
    uint64_t list = 0ull;
    float least = p.top > 0 ? -INFINITY : INFINITY;  // of the list's first `top`
    constexpr int kStep = 32 * kLpUnroll;
    for (int64_t j0 = begin + warp * kStep; j0 < end; j0 += kLpWarps * kStep) {
        uint4 v[kLpUnroll];
        int lo[kLpUnroll], hi[kLpUnroll];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const int64_t j = j0 + 32 * u + lane;
            lo[u] = 0;
            hi[u] = 0;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (j < end) {
                const int64_t first = j * E - off;  // index of the vector's first value
                lo[u] = first < 0 ? (int)-first : 0;
                hi[u] = first + E > p.V ? (int)(p.V - first) : E;
                if (hi[u] - lo[u] == E) {
                    v[u] = __ldcs(vec + j);
                } else {  // an end of the row: only its own values are read
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (e >= lo[u] && e < hi[u]) {
                            if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(x[first + e]);
                            else w[e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(x + first + e) << (16 * (e & 1));
                        }
                    v[u] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = lp_value<T>(w[sizeof(T) == 4 ? e : e >> 1], e & 1);
            if (hi[u] - lo[u] < E) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (e < lo[u] || e >= hi[u]) f[e] = -INFINITY;
            }
            float vm = f[0];
#pragma unroll
            for (int e = 1; e < E; ++e) vm = fmaxf(vm, f[e]);
            if (vm > a.m) shift(a, vm);
            const float zero = zero_of(a.m);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = max_nan(f[e] - zero, kFloor), q = ex2(d * kLog2e);
                a.s += q;
                a.t = fmaf(q, d, a.t);
            }
            if (__any_sync(0xffffffffu, hi[u] > lo[u] && vm >= least)) {
                list = take<T>(list, v[u], (int)((j0 + 32 * u + lane) * E - off), lo[u], hi[u], p.top);
                const uint64_t k = __shfl_sync(0xffffffffu, list, p.top - 1);
                least = k ? lp_key_value(k) : -INFINITY;
            }
        }
    }

    // the warp's sums, then the CTA's, then the cluster's
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Sums b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
        join(a, b);
    }
    if (lane == 0) s_sums[warp] = a;
    s_list[warp][lane] = list;
    __syncthreads();
#pragma unroll
    for (int o = kLpWarps / 2; o; o >>= 1) {
        if (warp < o) {
            list = join_lists(list, s_list[warp + o][31 - lane], lane);
            s_list[warp][lane] = list;
        }
        __syncthreads();
    }
    if (warp == 0) {
        a = s_sums[0];
#pragma unroll 1
        for (int w = 1; w < kLpWarps; ++w) join(a, s_sums[w]);
        if (lane == 0) s_sums[0] = a;
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync();
        if (rank == 0 && warp == 0) {
#pragma unroll 1
            for (int r = 1; r < p.split; ++r) {
                const uint32_t at = dsmem_map(&s_sums[0], (uint32_t)r), l = dsmem_map(&s_list[0][31 - lane], (uint32_t)r);
                Sums b;
                b.m = __uint_as_float(dsmem_ld_u32(at));
                b.s = __uint_as_float(dsmem_ld_u32(at + 4));
                b.t = __uint_as_float(dsmem_ld_u32(at + 8));
                join(a, b);
                list = join_lists(list, (uint64_t)dsmem_ld_u32(l + 4) << 32 | dsmem_ld_u32(l), lane);
            }
        }
        __syncwarp();
        cluster_sync();  // the others' shared memory is there until it has been read
    }
    if (rank != 0 || warp != 0) return;
    const float none = __uint_as_float(0x7FC00000u);
    if (!(a.m > -INFINITY)) a.s = none;  // nothing above -infinity
    const float ls = logf(a.s);
    auto logp_of = [&](float v) { return v - a.m - ls; };
    if (lane == 0) {
        const int id = __ldg(p.ids + row);
        p.logp[row] = id >= 0 && id < p.V ? logp_of(lp_value<T>(sizeof(T) == 4 ? __float_as_uint((float)x[id])
                                                                               : *reinterpret_cast<const uint16_t *>(x + id), 0))
                                          : none;
        p.entropy[row] = ls - a.t / a.s;
    }
    if (lane < p.top) {
        p.top_ids[row * p.top + lane] = list ? (int32_t)~(uint32_t)list : -1;
        p.top_logp[row * p.top + lane] = list ? logp_of(lp_key_value(list)) : none;
    }
}

template <typename T>
cudaError_t logp_launch(const LogpParams &p, int64_t T_rows, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(T_rows * p.split), 1, 1);
    cfg.blockDim = dim3(32 * kLpWarps, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, p);
}

}  // namespace

cudaError_t launch_token_logprobs(const void *logits, int32_t type, int64_t ld, int64_t T, int64_t V, const int32_t *ids,
                                  int32_t top, float *logp, float *entropy, int32_t *top_ids, float *top_logp,
                                  cudaStream_t st) {
    LogpParams p = {};
    p.x = logits; p.ids = ids; p.logp = logp; p.entropy = entropy; p.top_ids = top_ids; p.top_logp = top_logp;
    p.ld = ld; p.V = (int)V; p.top = top;
    // CTAs of a row: until every SM has two, as long as each has a step for every warp
    const int64_t per = (type == W4_F32 ? 4 : 8) * 32 * kLpWarps;
    p.split = 1;
    while (p.split < kMaxSplit && T * p.split < 152 && V > per * p.split) p.split *= 2;
    switch (type) {
        case W4_F32: return logp_launch<float>(p, T, st);
        case W4_BF16: return logp_launch<__nv_bfloat16>(p, T, st);
        default: return logp_launch<__half>(p, T, st);
    }
}

}  // namespace w4
