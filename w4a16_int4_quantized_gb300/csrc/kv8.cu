// kv8.cu -- a paged cache held in 8 bits: the store of a step's keys and values (with the head
// norms and the rotation on the way), and reading it back.
//
// Codes are int8, one power-of-two scale for 16 tokens of a head.  A power of two costs up to
// one bit of the 8 against the exact max / 127, and buys that a code's value is exact
// in bf16 and f32, that a scale that grows with a later token halves the kept codes (an
// error of one step at most over all growths, 1/2 + 1/4 + ...), and that the
// attention applies it to scores and weights without a rounding.
// 4,095 tokens of 32 query and 8 key heads of 128 from bf16: 26.2 us, 3.6 TB/s, bound by issue (norm and
// rotation) before memory; 128 requests of one token 7.4 us, rounds of latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "rows.cuh"
#include "w4.h"

namespace w4 {
namespace {

struct StoreParams {
    const void *qkv;
    const float *wq, *wk, *cos_sin;
    const int32_t *positions, *table, *ctx_len, *cu_new;
    void *q_out;
    int8_t *kc, *vc;
    uint8_t *ks, *vs;
    int64_t ld, T, B, max_pos, width, pages;
    int64_t page_stride, token_stride, head_stride;
    int64_t kv_ctas;  // CTAs of keys and values: (place of a block, head)
    int D, rot, inter, Hq, Hkv;
    int page_shift;
    int lanes, lanes2;  // lanes of a head (8 values each), and that rounded up to a power of two
    int groups;         // warps that share a token's query heads
    float eps, inv_d;
};

constexpr int kStoreWarps = 4;
constexpr int kQPasses = 4;  // head groups of a warp

// What a lane has of a head, as two runs of 4 values: those of the rotated part rot/2
// apart, so that a pair lies in one lane, the others half of the rest apart.
struct Runs {
    int i0, i1;
    bool rotated;
};
W4_DEV Runs runs_of(const StoreParams &p, int l) {
    Runs r;
    const int rl = p.rot / 8;
    r.rotated = l < rl;
    r.i0 = r.rotated ? 4 * l : p.rot + 4 * (l - rl);
    r.i1 = r.i0 + (r.rotated ? p.rot / 2 : (p.D - p.rot) / 2);
    return r;
}

// Angles of a token: half split, those of the pairs (i0 + e, i1 + e); interleaved, of the pairs in both runs.
W4_DEV void angles_of(const StoreParams &p, const Runs &r, int64_t pos, float (&cs)[4], float (&sn)[4]) {
    if (!r.rotated) return;
    const float *c = p.cos_sin + pos * p.rot, *s = c + p.rot / 2;
    if (p.inter) {
        const float2 a = __ldg(reinterpret_cast<const float2 *>(c + r.i0 / 2)), b = __ldg(reinterpret_cast<const float2 *>(c + r.i1 / 2));
        const float2 d = __ldg(reinterpret_cast<const float2 *>(s + r.i0 / 2)), e = __ldg(reinterpret_cast<const float2 *>(s + r.i1 / 2));
        cs[0] = a.x; cs[1] = a.y; cs[2] = b.x; cs[3] = b.y;
        sn[0] = d.x; sn[1] = d.y; sn[2] = e.x; sn[3] = e.y;
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(c + r.i0)), d = __ldg(reinterpret_cast<const float4 *>(s + r.i0));
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
        sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w;
    }
}

// The norm (w: null for none) and the rotation of a head; a converged warp.  In packed pairs; the root
// is brought to the nearest step or next to it by a step of Newton's, since an error there moves every
// code of the head that lies next to a tie.
W4_DEV void norm_turn(const StoreParams &p, const Runs &r, const float *w, bool live, const float (&cs)[4], const float (&sn)[4],
                      float (&v)[8]) {
    if (w) {
        uint64_t sq = 0ull;  // two sums
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint64_t x = f32x2(v[e], v[e + 1]);
            sq = f32x2_fma(x, x, sq);
        }
        float ss, s1;
        f32x2_split(sq, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = 16; o; o >>= 1) {  // no branch: a shuffle beyond the head is dropped
            const float x = __shfl_xor_sync(0xffffffffu, ss, o);
            if (o < p.lanes2) ss += x;
        }
        if (live) {
            const float m = ss * p.inv_d + p.eps, g = rsqrtf(m), n = fmaf(0.5f * g, fmaf(-m * g, g, 1.0f), g);
            const float f = isfinite(n) ? n : g;  // (0 and infinity)
            const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + r.i0)), w1 = __ldg(reinterpret_cast<const float4 *>(w + r.i1));
            const uint64_t ff = f32x2(f, f);
            const uint64_t ws[4] = {f32x2(w0.x, w0.y), f32x2(w0.z, w0.w), f32x2(w1.x, w1.y), f32x2(w1.z, w1.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f32x2_split(f32x2_mul(f32x2_mul(f32x2(v[2 * e], v[2 * e + 1]), ff), ws[e]), v[2 * e], v[2 * e + 1]);
        }
    }
    if (!r.rotated) return;
    if (p.inter) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = v[2 * e], b = v[2 * e + 1];
            v[2 * e] = a * cs[e] - b * sn[e];
            v[2 * e + 1] = b * cs[e] + a * sn[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const uint64_t a = f32x2(v[e], v[e + 1]), b = f32x2(v[e + 4], v[e + 5]);
            const uint64_t c = f32x2(cs[e], cs[e + 1]), d = f32x2(sn[e], sn[e + 1]), m = f32x2(-sn[e], -sn[e + 1]);
            f32x2_split(f32x2_fma(b, m, f32x2_mul(a, c)), v[e], v[e + 1]);
            f32x2_split(f32x2_fma(a, d, f32x2_mul(b, c)), v[e + 4], v[e + 5]);
        }
    }
}

// Scale byte of a block: 2^(s - 127) with the least e >= -127 such that top <= 127 * 2^e; 255
// where a value is not finite (top: the bits of the largest magnitude, NaN above all).
W4_DEV uint32_t block_scale(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    // top = 1.f * 2^(E - 127): E - 6 where 1.f <= 127/64, else one more; what is below 2^-121 has 0
    const int s = (int)(top >> 23) - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return (uint32_t)max(s, 0);
}

// 2^(127 - s) for s = 0 .. 254, in two factors that f32 has.
struct Inverse {
    float a, b;
};
W4_DEV Inverse inverse_of(uint32_t s) {
    const int e = 127 - (int)s, half = e / 2;
    return {__uint_as_float((uint32_t)(127 + half) << 23), __uint_as_float((uint32_t)(127 + e - half) << 23)};
}

// Keys and values: a CTA takes a block of 16 tokens of a request and a head, so that the
// block's scale is one CTA's affair.  Place i of all blocks belongs to the last request b
// with floor(cu_new[b] / 16) + 2 b <= i: a request's blocks are no more than the places up to
// the next one's, whatever the offsets, and no scan over the requests is needed.
template <typename TI, int PASSES>
W4_DEV void store_block(const StoreParams &p) {
    __shared__ uint32_t s_top[2][kStoreWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int64_t place = blockIdx.x / (unsigned)p.Hkv;
    int64_t b = 0, hi = p.B;
    while (hi - b > 1) {
        const int64_t step = ceil_div(hi - b, 32), at = b + lane * step;
        const bool below = at < hi && ((int64_t)max(__ldg(p.cu_new + at), 0) >> kKvBlockLog) + 2 * at <= place;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        const int64_t next = b + max(n - 1, 0) * step;
        hi = min(hi, next + step);
        b = next;
    }
    const KvRequest r = kv_request(p.cu_new, p.ctx_len, b, p.T, p.width, p.page_shift);
    const int64_t p0 = ((r.ctx >> kKvBlockLog) + place - ((r.t0 >> kKvBlockLog) + 2 * b)) << kKvBlockLog;  // the block's first position
    if (r.n == 0 || p0 >= r.len || p0 + kKvBlock <= r.ctx) return;
    const int32_t page = __ldg(p.table + b * p.width + (p0 >> p.page_shift));
    if (page < 0 || page >= p.pages) return;
    const int off = (int)(p0 & ((1 << p.page_shift) - 1));
    const int64_t blocks = 1 << (p.page_shift - kKvBlockLog);
    const int64_t scale_at = ((int64_t)page * p.Hkv + head) * blocks + (off >> kKvBlockLog);
    const int kept = (int)max((int64_t)0, r.ctx - p0);  // tokens of the block that stay
    const uint32_t old_k = kept ? p.ks[scale_at] : 0u, old_v = kept ? p.vs[scale_at] : 0u;

    const int per_warp = 32 / p.lanes2, sub = lane / p.lanes2, l = lane & (p.lanes2 - 1);
    const Runs run = runs_of(p, l);
    float k[PASSES][8], v[PASSES][8];
    Raw4<TI> raw[PASSES][4];
    bool on[PASSES];
    uint32_t top_k = 0u, top_v = 0u;
    // every token of the block is asked for before the first is worked on
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int tok = (i * kStoreWarps + warp) * per_warp + sub;
        const int64_t pos = p0 + tok, t = r.t0 + pos - r.ctx;
        on[i] = l < p.lanes && tok >= kept && tok < kKvBlock && pos < r.len;
#pragma unroll
        for (int e = 0; e < (int)sizeof(TI); ++e) raw[i][0].r[e] = raw[i][1].r[e] = raw[i][2].r[e] = raw[i][3].r[e] = 0u;
        if (on[i]) {
            const TI *in = static_cast<const TI *>(p.qkv) + t * p.ld + (int64_t)(p.Hq + head) * p.D;
            raw[i][0] = load4(in + run.i0);
            raw[i][1] = load4(in + run.i1);
            raw[i][2] = load4(in + (int64_t)p.Hkv * p.D + run.i0);
            raw[i][3] = load4(in + (int64_t)p.Hkv * p.D + run.i1);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int tok = (i * kStoreWarps + warp) * per_warp + sub;
        const int64_t t = r.t0 + p0 + tok - r.ctx;
        unpack4<TI>(raw[i][0], k[i]);
        unpack4<TI>(raw[i][1], k[i] + 4);
        unpack4<TI>(raw[i][2], v[i]);
        unpack4<TI>(raw[i][3], v[i] + 4);
        float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (on[i]) {
            const int32_t pos = __ldg(p.positions + t);
            on[i] = pos >= 0 && pos < p.max_pos;  // else the token is left out
            if (on[i]) angles_of(p, run, pos, cs, sn);
        }
        norm_turn(p, run, p.wk, on[i], cs, sn, k[i]);
        if (on[i]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                top_k = max(top_k, __float_as_uint(k[i][e]) & 0x7FFFFFFFu);
                top_v = max(top_v, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
            }
        }
    }
    top_k = __reduce_max_sync(0xffffffffu, top_k);
    top_v = __reduce_max_sync(0xffffffffu, top_v);
    if (lane == 0) {
        s_top[0][warp] = top_k;
        s_top[1][warp] = top_v;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStoreWarps; ++w) {
        top_k = max(top_k, s_top[0][w]);
        top_v = max(top_v, s_top[1][w]);
    }
    const uint32_t sk = max(block_scale(top_k), old_k), sv = max(block_scale(top_v), old_v);
    if (threadIdx.x == 0) {
        p.ks[scale_at] = (uint8_t)sk;
        p.vs[scale_at] = (uint8_t)sv;
    }
    const int64_t base = (int64_t)page * p.page_stride + (int64_t)head * p.head_stride + (int64_t)off * p.token_stride;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint32_t s = kv ? sv : sk, old = kv ? old_v : old_k;
        int8_t *to = (kv ? p.vc : p.kc) + base;
        const Inverse inv = inverse_of(min(s, 254u));
        // of kept tokens: 2^(old - s), in one factor (beyond 2^-126 every code goes to 0 all the same)
        const float shrink = s == 255u ? 0.0f : __uint_as_float((uint32_t)max(127 - (int)(s - old), 1) << 23);
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int tok = (i * kStoreWarps + warp) * per_warp + sub;
            int8_t *d = to + (int64_t)tok * p.token_stride;
            if (on[i]) {
                const float *x = kv ? v[i] : k[i];
                int c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = s == 255u ? 0 : __float2int_rn(x[e] * inv.a * inv.b);
                *reinterpret_cast<uint32_t *>(d + run.i0) = pack_codes(c[0], c[1], c[2], c[3]);
                *reinterpret_cast<uint32_t *>(d + run.i1) = pack_codes(c[4], c[5], c[6], c[7]);
            } else if (tok < kept && l < p.lanes && s != old) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t *at = reinterpret_cast<uint32_t *>(d + (h ? run.i1 : run.i0));
                    const uint32_t w = *at;
                    int c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = __float2int_rn((float)(int8_t)(w >> (8 * e)) * shrink);
                    *at = pack_codes(c[0], c[1], c[2], c[3]);
                }
            }
        }
    }
}

template <typename TI, typename TQ, int PASSES>
__global__ void __launch_bounds__(32 * kStoreWarps) kv8_store_kernel(const StoreParams p) {
    griddep_wait();
    if (blockIdx.x < p.kv_ctas) {
        store_block<TI, PASSES>(p);
        return;
    }
    // Queries: a warp takes head groups of a token, all of them requested first.
    const int lane = threadIdx.x & 31;
    const uint32_t item = (blockIdx.x - (uint32_t)p.kv_ctas) * kStoreWarps + (threadIdx.x >> 5);
    const int64_t t = item / (uint32_t)p.groups;
    const int group = (int)(item - (uint32_t)t * (uint32_t)p.groups);
    if (t >= p.T || t >= __ldg(p.cu_new + p.B)) return;
    const int per_warp = 32 / p.lanes2, sub = lane / p.lanes2, l = lane & (p.lanes2 - 1);
    const Runs run = runs_of(p, l);
    const TI *in = static_cast<const TI *>(p.qkv) + t * p.ld;
    Raw4<TI> raw[kQPasses][2];
#pragma unroll
    for (int i = 0; i < kQPasses; ++i) {
        const int h = (group + i * p.groups) * per_warp + sub;
#pragma unroll
        for (int e = 0; e < (int)sizeof(TI); ++e) raw[i][0].r[e] = raw[i][1].r[e] = 0u;
        if (l < p.lanes && h < p.Hq) {
            raw[i][0] = load4(in + (int64_t)h * p.D + run.i0);
            raw[i][1] = load4(in + (int64_t)h * p.D + run.i1);
        }
    }
    const int32_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_pos) return;
    float cs[4], sn[4];
    angles_of(p, run, pos, cs, sn);
    TQ *q_row = static_cast<TQ *>(p.q_out) + t * p.Hq * p.D;
#pragma unroll
    for (int i = 0; i < kQPasses; ++i) {
        const int h0 = (group + i * p.groups) * per_warp, h = h0 + sub;
        if (h0 >= p.Hq) break;
        float v[8];
        unpack4<TI>(raw[i][0], v);
        unpack4<TI>(raw[i][1], v + 4);
        const bool live = l < p.lanes && h < p.Hq;
        norm_turn(p, run, p.wq, live, cs, sn, v);
        if (!live) continue;
        store4(q_row + (int64_t)h * p.D + run.i0, v);
        store4(q_row + (int64_t)h * p.D + run.i1, v + 4);
    }
}

template <typename TI, typename TQ>
cudaError_t store_launch(const StoreParams &p, const cudaLaunchConfig_t &cfg) {
    if (p.lanes2 <= 8) return cudaLaunchKernelEx(&cfg, kv8_store_kernel<TI, TQ, 1>, p);
    if (p.lanes2 == 16) return cudaLaunchKernelEx(&cfg, kv8_store_kernel<TI, TQ, 2>, p);
    return cudaLaunchKernelEx(&cfg, kv8_store_kernel<TI, TQ, 4>, p);
}

template <typename TI>
cudaError_t store_launch_q(const StoreParams &p, int q_type, const cudaLaunchConfig_t &cfg) {
    return q_type == W4_BF16 ? store_launch<TI, __nv_bfloat16>(p, cfg) : store_launch<TI, __half>(p, cfg);
}

// ---------------------------------------------------------------- reading back

struct ReadParams {
    const int8_t *c[2];
    const uint8_t *s[2];
    void *out[2];
    int64_t page_stride, token_stride, head_stride;
    uint32_t heads, chunks, page_shift;  // chunks of 16 values of a row
    uint32_t items, parts;               // chunks of a page, CTAs of one
};

constexpr int kReads = 4;  // chunks of a thread

// A thread turns 16 codes into values, four times; the output is dense.  Bound by memory: 25 MB of codes
// to bf16 in 12.2 us, 6.1 TB/s (18.1 with 64-bit divisions for each 16 codes; places are counted within
// a page, in 32 bits).
template <typename TO>
__global__ void __launch_bounds__(256) kv8_read_kernel(const ReadParams p) {
    griddep_wait();
    const bool values = blockIdx.y != 0;
    const int8_t *codes = values ? p.c[1] : p.c[0];
    const uint8_t *scales = values ? p.s[1] : p.s[0];
    TO *out = static_cast<TO *>(values ? p.out[1] : p.out[0]);
    const int64_t page = blockIdx.x / p.parts;
    const uint32_t first = (blockIdx.x - (uint32_t)page * p.parts) * (256 * kReads) + threadIdx.x;
    uint4 w[kReads];
    float f[kReads];
#pragma unroll
    for (int u = 0; u < kReads; ++u) {
        const uint32_t i = first + 256 * u;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        f[u] = 0.0f;
        if (i < p.items) {
            const uint32_t row = i / p.chunks, chunk = i - row * p.chunks, tok = row / p.heads, head = row - tok * p.heads;
            w[u] = __ldcs(reinterpret_cast<const uint4 *>(codes + page * p.page_stride + tok * p.token_stride +
                                                          head * p.head_stride + 16 * chunk));
            f[u] = scale_of(__ldg(scales + ((page * p.heads + head) << (p.page_shift - kKvBlockLog)) + (tok >> kKvBlockLog)));
        }
    }
#pragma unroll
    for (int u = 0; u < kReads; ++u) {
        const uint32_t i = first + 256 * u;
        if (i >= p.items) continue;
        const uint32_t c[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = (float)(int8_t)(c[e / 4] >> (8 * (e % 4))) * f[u];
        TO *to = out + (page * p.items + i) * 16;
        if constexpr (sizeof(TO) == 4) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) store4(to + e, v + e);
        } else {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4 *>(to + e) = make_uint4(pack_pair<TO>(v[e], v[e + 1]), pack_pair<TO>(v[e + 2], v[e + 3]),
                                                                pack_pair<TO>(v[e + 4], v[e + 5]), pack_pair<TO>(v[e + 6], v[e + 7]));
        }
    }
}

cudaLaunchAttribute *pdl(cudaLaunchAttribute *a) {
    a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a->val.programmaticStreamSerializationAllowed = 1;
    return a;
}

// Lanes of a head (8 values each), rounded up to a power of two.
int lanes_of(int32_t head_dim) {
    int n = 1;
    while (n < head_dim / 8) n *= 2;
    return n;
}

// Warps of a token's query heads: kQPasses groups each; few tokens are spread over more, until
// the machine (152 SMs x 64 warps) has one round.
int query_groups(int64_t T, int32_t q_heads, int lanes) {
    const int64_t iters = ceil_div((int64_t)q_heads, 32 / lanes);
    return (int)std::max<int64_t>(ceil_div(iters, kQPasses), std::min<int64_t>(iters, 152 * 64 / T));
}

int64_t read_items(const w4_kv8_cache &c) { return (int64_t)c.page_size * c.heads * (c.head_dim / 16); }

}  // namespace

int64_t kv8_store_ctas(int64_t T, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return ((T >> kKvBlockLog) + 2 * B) * kv_heads + ceil_div(T * query_groups(T, q_heads, lanes_of(head_dim)), kStoreWarps);
}

bool kv8_read_fits(const w4_kv8_cache &c) {
    return read_items(c) < (1ll << 31) && c.pages * ceil_div(read_items(c), 256 * kReads) < (1ll << 31);
}

cudaError_t launch_qk_norm_rope_kv8(const void *qkv, int32_t x_type, int64_t ld, int64_t T, int32_t q_heads, const float *wq,
                                    const float *wk, float eps, const int32_t *positions, const float *cos_sin,
                                    int64_t max_pos, int32_t rot, int32_t interleaved, const int32_t *table, int64_t width,
                                    const int32_t *ctx_len, const int32_t *cu_new, int64_t B, const w4_kv8_cache &c,
                                    void *q_out, int32_t q_type, cudaStream_t st) {
    StoreParams p = {};
    p.qkv = qkv; p.wq = wq; p.wk = wk; p.cos_sin = cos_sin; p.positions = positions; p.table = table;
    p.ctx_len = ctx_len; p.cu_new = cu_new; p.q_out = q_out; p.kc = c.k; p.vc = c.v; p.ks = c.k_scale; p.vs = c.v_scale;
    p.ld = ld; p.T = T; p.B = B; p.max_pos = max_pos; p.width = width; p.pages = c.pages;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.D = c.head_dim; p.rot = rot; p.inter = interleaved != 0; p.Hq = q_heads; p.Hkv = c.heads;
    p.page_shift = log2_of(c.page_size);
    p.eps = eps;
    p.inv_d = 1.0f / (float)c.head_dim;
    p.lanes = c.head_dim / 8;
    p.lanes2 = lanes_of(c.head_dim);
    p.groups = query_groups(T, q_heads, p.lanes2);
    p.kv_ctas = ((T >> kKvBlockLog) + 2 * B) * c.heads;
    const int64_t ctas = kv8_store_ctas(T, B, q_heads, c.heads, c.head_dim);
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(32 * kStoreWarps, 1, 1);
    cfg.stream = st;
    cfg.attrs = pdl(&attr);
    cfg.numAttrs = 1;
    switch (x_type) {
        case W4_F32: return store_launch_q<float>(p, q_type, cfg);
        case W4_BF16: return store_launch_q<__nv_bfloat16>(p, q_type, cfg);
        default: return store_launch_q<__half>(p, q_type, cfg);
    }
}

cudaError_t launch_dequantize_kv8(const w4_kv8_cache &c, void *k_out, void *v_out, int32_t type, cudaStream_t st) {
    ReadParams p = {};
    p.c[0] = c.k; p.c[1] = c.v; p.s[0] = c.k_scale; p.s[1] = c.v_scale; p.out[0] = k_out; p.out[1] = v_out;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.heads = (uint32_t)c.heads; p.chunks = (uint32_t)c.head_dim / 16; p.page_shift = (uint32_t)log2_of(c.page_size);
    p.items = (uint32_t)read_items(c);
    p.parts = (uint32_t)ceil_div(read_items(c), 256 * kReads);
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.pages * p.parts), 2, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = pdl(&attr);
    cfg.numAttrs = 1;
    switch (type) {
        case W4_F32: return cudaLaunchKernelEx(&cfg, kv8_read_kernel<float>, p);
        case W4_BF16: return cudaLaunchKernelEx(&cfg, kv8_read_kernel<__nv_bfloat16>, p);
        default: return cudaLaunchKernelEx(&cfg, kv8_read_kernel<__half>, p);
    }
}

}  // namespace w4
