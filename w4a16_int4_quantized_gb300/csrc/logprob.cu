// logprob.cu -- log probabilities of given tokens, the entropy and the top alternatives of rows of logits.
//
// One pass over a row, by 1 to 8 CTAs of a cluster.  In units of log2, y = x log2(e) - m2 with
// m2 about a running maximum of each lane: s = sum 2^y, t = sum y 2^y, from which
// log p(i) = ln2 (y_i - log2 s) and the entropy is ln2 (log2 s - t / s); m2 cancels, so its
// rounding does not matter.
// The top values are found from each lane's largest value in each quarter of its vectors: the
// top-th of the lanes' largest over the CTA is no larger than the top-th value of what the CTA read,
// and not many values reach it.  The quarters whose largest value does (about `top` of 1,024) are
// read again, and what reaches the bound goes through shared memory into the warp's list of its 32
// largest, as whole numbers (value, then lowest index), 32 sorted and joined at a time.
// Lists and sums are joined over the warps, then over the cluster in shared memory, in a
// fixed order.
// 2048 rows of 131,072 bf16: 101 us, 5.3 TB/s (84 without top values); 1024 of f32: 93 us.  By insertion
// of every value above a warp's own 20th the former took 542 us, with a bound that followed
// along 144.  Bound by memory, then by issue (about 7 instructions a value); one row of 32,000: 8 us of
// latency (launch, loads, the bound, the joins).
// A bound that most values reach costs a second look at all of them and a sort for each 32: rows with fewer values
// above -infinity than `top`, or of one value.  2048 rows of 131,072 then take 2,140 us, one row of 32,000 16 to
// 41 (with 99 in 100 masked, and 20 asked for, as plain rows: 104 and 8).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kLpWarps = 8;
constexpr int kDepth = 4;  // pairs of 16-byte vectors in a lane's ring (a power of two)
constexpr int kQuarters = 4;  // of a lane's vectors
constexpr int kAgain = 4;     // vectors of a lane in flight when some are read again
constexpr int kMaxSplit = 8;
constexpr int kFill = 152;  // CTAs from which on rows are not split: 608 measured slower at 64 to 512 rows (33 and 37 us at 512 of 131,072)
constexpr float kLn2 = 0.693147181f;
constexpr float kGrowth = 8.0f;  // by which a logit may exceed m before the sums are moved (each lane would else move at most vectors)
constexpr float kFloor = -1e5f;  // exponents below count as this: their power is 0, and 0 times them must be 0
constexpr float kLeast = -0x1.5Ap127f;  // -2.3e38: logits below count as this in the sums, so that a y is finite
constexpr uint32_t kLeastBf16 = 0xFF2DFF2Du;  // the same in bf16, twice

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

template <typename T>
W4_DEV float value_at(const T *x, int i) {
    if constexpr (sizeof(T) == 4) return x[i];
    else return lp_value<T>(*reinterpret_cast<const uint16_t *>(x + i), 0);
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

// The warp's 32 largest with another key of each lane.
W4_DEV uint64_t take(uint64_t list, uint64_t key, int lane) {
#pragma unroll
    for (int size = 2; size < 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            const bool larger_here = ((lane & o) == 0) != ((lane & size) != 0);
            key = larger_here == (key > other) ? key : other;
        }
    key = bitonic_down(key, lane);
    return join_lists(list, __shfl_sync(0xffffffffu, key, 31 - lane), lane);
}

// m: what the sums are relative to; y = x c - m2; s = sum 2^y, t = sum y 2^y.
// Logits of 2^30 and more differ by 64 or not at all, so for such an m any c that keeps y finite
// gives the same sums (weights 1 and 0), and m2 = m c is exact; log2(e) would leave y = m c - m2 too large there.
struct Sums {
    float m, s, t;
};
W4_DEV float factor_of(float m) {
    const float a = fabsf(m);
    return a <= 0x1p30f || a == INFINITY ? kLog2e : a <= 0x1p100f ? 1.0f : 0x1p-60f;
}
// (nothing above -infinity yet: 0)
W4_DEV float zero_of(float m) { return m == -INFINITY ? 0.0f : m * factor_of(m); }

// Moves the sums to another m, not below theirs.
W4_DEV void shift(Sums &a, float m) {
    const bool plain = fabsf(a.m) <= 0x1p30f && fabsf(m) <= 0x1p30f;
    float d = plain ? zero_of(a.m) - zero_of(m) : a.m == m ? 0.0f : a.m - m;
    d = max_nan(d, kFloor);
    const float f = ex2(d);
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
W4_DEV Sums sums_of(float m, uint64_t s2, uint64_t t2) {
    float s0, s1, t0, t1;
    f32x2_split(s2, s0, s1);
    f32x2_split(t2, t0, t1);
    return {m, s0 + s1, t0 + t1};
}

// A value's place in the order, as a whole number; 0 below all (NaN).
W4_DEV uint32_t lp_order(float x) { return (uint32_t)(lp_key(x, 0) >> 32); }

// The sums of a lane, two of each.
struct Running {
    float m, c, minus;  // what they are relative to, and y = x c + minus
    uint64_t s2, t2;
};
W4_DEV void move_to(Running &r, float m) {
    m = fmaxf(m, kLeast);
    Sums a = sums_of(r.m, r.s2, r.t2);
    shift(a, m);
    r.m = m;
    r.c = factor_of(m);
    r.minus = -zero_of(m);
    r.s2 = f32x2(a.s, 0.0f);
    r.t2 = f32x2(a.t, 0.0f);
}
// x0, x1: logits not below kLeast, so that y is finite
W4_DEV void count_in(Running &r, float x0, float x1) {
    const uint64_t y = f32x2_fma(f32x2(x0, x1), f32x2(r.c, r.c), f32x2(r.minus, r.minus));
    float y0, y1;
    f32x2_split(y, y0, y1);
    const uint64_t q = f32x2(ex2(y0), ex2(y1));
    r.s2 = f32x2_add(r.s2, q);
    r.t2 = f32x2_fma(q, y, r.t2);
}

// The values of a vector, and the largest of them.
template <typename T>
W4_DEV void values_of(const uint4 &v, float (&f)[16 / sizeof(T)]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(T)); ++e) f[e] = lp_value<T>(w[sizeof(T) == 4 ? e : e >> 1], e & 1);
}
template <typename T>
W4_DEV float largest_of(const uint4 &v) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        // in pairs, as they lie
        using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const P *h = reinterpret_cast<const P *>(&v);
        const P m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
        return fmaxf(lp_value<T>(w, 0), lp_value<T>(w, 1));
    }
}
template <typename T>
W4_DEV void count_vector(Running &r, const uint4 &v) {
    constexpr int E = 16 / sizeof(T);
    float f[E];
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        uint4 u;
        asm("max.NaN.bf16x2 %0, %4, %8;\n\tmax.NaN.bf16x2 %1, %5, %8;\n\tmax.NaN.bf16x2 %2, %6, %8;\n\tmax.NaN.bf16x2 %3, %7, %8;"
            : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
            : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(kLeastBf16));
        values_of<T>(u, f);
    } else {
        values_of<T>(v, f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = max_nan(f[e], kLeast);
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) count_in(r, f[e], f[e + 1]);
}

// The warp's 32 largest keys, one a lane, and how many more wait in shared memory (below 32).
struct Top {
    uint64_t list;
    int waiting;
};
// With the values of the lanes' vectors that reach the bound (idx: index of the first).  Out of
// line: rare.
template <typename T>
__device__ __noinline__ Top collect(Top t, uint4 v, int idx, bool on, float least, uint64_t *wait) {
    const int lane = threadIdx.x & 31;
    float f[16 / sizeof(T)];
    values_of<T>(v, f);
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(T)); ++e) {
        const bool in = on && f[e] >= least;
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (!who) continue;
        if (in) wait[t.waiting + __popc(who & ((1u << lane) - 1u))] = lp_key(f[e], idx + e);
        __syncwarp();
        t.waiting += __popc(who);
        if (t.waiting >= 32) {
            const uint64_t next = wait[32 + lane];
            t.list = take(t.list, wait[lane], lane);
            __syncwarp();
            wait[lane] = next;
            __syncwarp();
            t.waiting -= 32;
        }
    }
    return t;
}

// The largest finite bound below which nothing is among the top: see above.  By the whole CTA.
W4_DEV float bound_of(float m, bool any, int top, uint32_t (*sorted)[32], int warp, int lane) {
    uint32_t k = any ? lp_order(m) : 0u;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o; o >>= 1) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, k, o);
            const bool larger_here = ((lane & o) == 0) != ((lane & size) != 0 && size < 32);
            k = larger_here == (k > other) ? k : other;
        }
    __syncthreads();  // (the bound before has been read)
    sorted[warp][lane] = k;
#pragma unroll 1
    for (int half = kLpWarps / 2; half; half >>= 1) {
        __syncthreads();
        if (warp < half) {
            k = max(k, sorted[warp + half][31 - lane]);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, k, o);
                k = ((lane & o) == 0) == (k > other) ? k : other;
            }
            sorted[warp][lane] = k;
        }
    }
    __syncthreads();
    k = sorted[0][top - 1];
    return k == 0u ? -INFINITY : __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <typename T>
__global__ void __launch_bounds__(32 * kLpWarps, 4) token_logprobs_kernel(const LogpParams p) {
    constexpr int E = 16 / sizeof(T);
    __shared__ __align__(16) uint4 s_ring[kLpWarps][kDepth][2][32];
    __shared__ uint64_t s_list[kLpWarps][32];
    __shared__ uint64_t s_wait[kLpWarps][64];
    __shared__ uint32_t s_sorted[kLpWarps][32];
    __shared__ float s_most[kQuarters][32 * kLpWarps];  // (each thread reads its own)
    __shared__ int s_found[kLpWarps];
    __shared__ Sums s_sums[kLpWarps];
    __shared__ uint64_t s_ranks[kMaxSplit][32];  // the CTAs' lists and sums, in the first one's memory
    __shared__ Sums s_rank_sums[kMaxSplit];
    if (p.split > 1) cluster_arrive();  // the others' shared memory is there once all have come
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / p.split;
    const int rank = (int)(blockIdx.x - row * p.split);
    const T *x = static_cast<const T *>(p.x) + row * p.ld;

    // (asked for early: the last thing that is needed)
    const int id = rank == 0 ? __ldg(p.ids + row) : -1;
    const bool known = id >= 0 && id < p.V;
    const float x_id = known ? value_at(x, id) : 0.0f;

    // The row in vectors of 16 aligned bytes, `head` values before the first; those and what
    // is behind the last one go one by one.
    const int head = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
    const int n = (p.V - head) / E, tail = head + n * E;
    const uint4 *vec = reinterpret_cast<const uint4 *>(x + head);
    const int begin = (int)((int64_t)n * rank / p.split), end = (int)((int64_t)n * (rank + 1) / p.split);
    constexpr int kStep = 64 * kLpWarps;  // two vectors a lane
    const int steps = (end - begin + kStep - 1) / kStep;

    float most = -INFINITY;  // of the lane's quarter
    Running run = {-INFINITY, kLog2e, 0.0f, 0ull, 0ull};
    // Every lane copies what it will read itself, kDepth - 1 steps ahead.
    const int j0 = begin + 64 * warp + lane;
    const uint32_t ring = smem_u32(&s_ring[warp][0][0][lane]);
    auto copy = [&](int r) {
        const int j = j0 + r * kStep;
        const uint32_t to = ring + (uint32_t)((r % kDepth) * 1024);
        if (j < end) cp_async16(to, vec + j);
        if (j + 32 < end) cp_async16(to + 512, vec + j + 32);
        cp_commit();
    };
#pragma unroll
    for (int r = 0; r < kDepth - 1; ++r) copy(r);
    const int quarter = (steps + kQuarters - 1) / kQuarters;  // steps of one
    int left = quarter, c_at = 0;
#pragma unroll
    for (int c = 0; c < kQuarters; ++c) s_most[c][threadIdx.x] = -INFINITY;
    const uint4 *ahead = vec + j0 + (kDepth - 1) * kStep;
    int at = 0;  // of the ring
#pragma unroll 1
    for (int r = 0; r < steps; ++r) {
        const int j = j0 + r * kStep;
        const int base = j - lane;
        {
            const uint32_t to = ring + (uint32_t)(((at + kDepth - 1) & (kDepth - 1)) * 1024);
            if (base + (kDepth - 1) * kStep + 64 <= end) {
                cp_async16(to, ahead);
                cp_async16(to + 512, ahead + 32);
            } else {
                if (j + (kDepth - 1) * kStep < end) cp_async16(to, ahead);
                if (j + (kDepth - 1) * kStep + 32 < end) cp_async16(to + 512, ahead + 32);
            }
            cp_commit();
            ahead += kStep;
        }
        cp_wait<kDepth - 1>();
        const uint32_t from = ring + (uint32_t)(at * 1024);
        at = (at + 1) & (kDepth - 1);
        uint4 v[2];
        float vm[2];
        bool on[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            v[u] = lds_u128(from + 512 * u);
            on[u] = j + 32 * u < end;
            vm[u] = on[u] ? largest_of<T>(v[u]) : -INFINITY;
        }
        const float vmax = fmaxf(vm[0], vm[1]);
        most = fmaxf(most, vmax);
        if (--left == 0 || r == steps - 1) {
            s_most[c_at++][threadIdx.x] = most;
            most = -INFINITY;
            left = quarter;
        }
        if (vmax > run.m + kGrowth) move_to(run, vmax);
        if (base + 64 <= end) {
            count_vector<T>(run, v[0]);
            count_vector<T>(run, v[1]);
        } else {
            if (on[0]) count_vector<T>(run, v[0]);
            if (on[1]) count_vector<T>(run, v[1]);
        }
    }
    uint64_t list = 0ull;
    if (p.top > 0) {
        float most = -INFINITY;
#pragma unroll
        for (int c = 0; c < kQuarters; ++c) most = fmaxf(most, s_most[c][threadIdx.x]);
        const float least = bound_of(most, j0 < end, p.top, s_sorted, warp, lane);
        Top top = {0ull, 0};
        uint64_t *wait = s_wait[warp];
        // the quarters that reach the bound, in order of warp, quarter and lane
        uint32_t who[kQuarters];
        int mine = 0;
#pragma unroll
        for (int c = 0; c < kQuarters; ++c) {
            who[c] = __ballot_sync(0xffffffffu, j0 < end && s_most[c][threadIdx.x] >= least);
            mine += __popc(who[c]);
        }
        if (lane == 0) s_found[warp] = mine;
        __syncthreads();
        int before = 0, found = 0;
#pragma unroll
        for (int w = 0; w < kLpWarps; ++w) {
            if (w < warp) before += s_found[w];
            found += s_found[w];
        }
        uint16_t *again = reinterpret_cast<uint16_t *>(&s_ring[0][0][0][0]);  // (nobody reads the ring any more)
#pragma unroll
        for (int c = 0; c < kQuarters; ++c) {
            if (who[c] >> lane & 1u) again[before + __popc(who[c] & ((1u << lane) - 1u))] = (uint16_t)(c << 8 | (int)threadIdx.x);
            before += __popc(who[c]);
        }
        __syncthreads();
        // their vectors, 32 to a warp in turn: vector i of a quarter is vector i & 1 of its step i >> 1
        const int each = 2 * quarter, all = found * each;
#pragma unroll 1
        for (int t0 = 32 * warp; t0 < all; t0 += 32 * kLpWarps * kAgain) {
            uint4 v[kAgain];
            int j[kAgain];
#pragma unroll
            for (int u = 0; u < kAgain; ++u) {
                const int t = t0 + 32 * kLpWarps * u + lane, f = t / each, i = t - f * each;
                j[u] = end;
                v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (t < all) {
                    const int which = again[f], thread = which & 255;
                    j[u] = begin + 64 * (thread >> 5) + (thread & 31) + ((which >> 8) * quarter + (i >> 1)) * kStep + 32 * (i & 1);
                    if (j[u] < end) v[u] = __ldg(vec + j[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kAgain; ++u) {
                const bool in = j[u] < end && largest_of<T>(v[u]) >= least;
                if (__any_sync(0xffffffffu, in)) top = collect<T>(top, v[u], head + j[u] * E, in, least, wait);
            }
        }
        list = take(top.list, lane < top.waiting ? wait[lane] : 0ull, lane);
    }
    if (rank == 0 && warp == 0) {
        // the values before and behind the vectors, one to a lane
        const int i = lane < head ? lane : tail + lane - head;
        const bool on = i < p.V;
        const float f = on ? value_at(x, i) : -INFINITY;
        if (f > run.m + kGrowth) move_to(run, f);
        if (on) {
            const float y = fmaf(max_nan(f, kLeast), run.c, run.minus), q = ex2(y);
            run.s2 = f32x2_add(run.s2, f32x2(q, 0.0f));
            run.t2 = f32x2_add(run.t2, f32x2(q * y, 0.0f));
        }
        __syncwarp();
        list = take(list, on ? lp_key(f, i) : 0ull, lane);
    }

    // the warp's sums, then the CTA's, then the cluster's
    Sums a = sums_of(run.m, run.s2, run.t2);
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
        cluster_wait();
        if (warp == 0) {
            const uint32_t at = dsmem_map(&s_ranks[rank][lane], 0), sums = dsmem_map(&s_rank_sums[rank], 0);
            dsmem_st_u32(at, (uint32_t)list);
            dsmem_st_u32(at + 4, (uint32_t)(list >> 32));
            if (lane == 0) {
                dsmem_st_u32(sums, __float_as_uint(a.m));
                dsmem_st_u32(sums + 4, __float_as_uint(a.s));
                dsmem_st_u32(sums + 8, __float_as_uint(a.t));
            }
        }
        __syncwarp();
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
        if (warp == 0) {
#pragma unroll 1
            for (int r = 1; r < p.split; ++r) {
                join(a, s_rank_sums[r]);
                list = join_lists(list, s_ranks[r][31 - lane], lane);
            }
        }
    }
    if (rank != 0 || warp != 0) return;
    const float none = __uint_as_float(0x7FC00000u);
    if (!(a.m > -INFINITY)) a.s = none;  // nothing above -infinity
    const float ls = log2f(a.s), c = factor_of(a.m), minus = -zero_of(a.m);
    auto logp_of = [&](float v) {
        if (c == kLog2e && !(fabsf(v) > 0x1p30f)) return kLn2 * (fmaf(v, kLog2e, minus) - ls);
        // far below m, or all of the row far from 0: a logit's own size is all that counts
        return (a.m == kLeast && v > -INFINITY ? fmaxf(v, kLeast) : v) - a.m - kLn2 * ls;
    };
    if (lane == 0) {
        p.logp[row] = known ? logp_of(x_id) : none;
        p.entropy[row] = kLn2 * (ls - a.t / a.s);
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
    // CTAs of a row: until every SM has one, as long as each has a step for every warp
    const int64_t per = (type == W4_F32 ? 4 : 8) * 64 * kLpWarps;
    p.split = 1;
    while (p.split < kMaxSplit && T * p.split < kFill && V > per * p.split) p.split *= 2;
    switch (type) {
        case W4_F32: return logp_launch<float>(p, T, st);
        case W4_BF16: return logp_launch<__nv_bfloat16>(p, T, st);
        default: return logp_launch<__half>(p, T, st);
    }
}

}  // namespace w4
