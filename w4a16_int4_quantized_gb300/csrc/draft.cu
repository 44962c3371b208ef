// draft.cu -- what stands around the attention of a step of drafted tokens:
// the plan (block tables, slots, positions, ancestor masks) and the head norms
// with the rotation and the store into the paged cache.
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

// ---------------------------------------------------------------- plan

constexpr int kPlanWarps = 8;  // requests per block, one warp each
constexpr int kMaxDraft = W4_MAX_DRAFT;

W4_DEV int plan_new(const int32_t *new_len, int64_t b) { return min(max(__ldg(new_len + b), 0), kMaxDraft); }

// Table entries a request has and needs, as the header defines them (32-bit
// unsigned: ctx_len + new_len + page_size - 1 stays below 2^32).
W4_DEV void plan_blocks(uint32_t ctx, uint32_t n, uint32_t page, uint32_t width, uint32_t &have, uint32_t &need) {
    have = (uint32_t)(((uint64_t)ctx + page - 1) / page);
    need = min((uint32_t)(((uint64_t)ctx + n + page - 1) / page), width);
}

// One launch for the whole plan.  Every block sums the lengths and the page
// needs of all requests before its own (and of all of them, for the padding):
// 8 bytes a request from L2, instead of a second launch or blocks that wait on
// one another.  A warp then closes its request's parent relation by pointer
// doubling: after round r, mask(i) holds the first 2^r tokens of the path from
// i to its root and anc(i) the 2^r-th ancestor, so 7 rounds reach 128.
// Bound by a launch and its rounds of latency (lengths, parents, table): 2.8 us
// for one request, 5.1 us for 256 of 64 tokens.
__global__ void __launch_bounds__(32 * kPlanWarps)
draft_plan_kernel(const int32_t *__restrict__ ctx_len, const int32_t *__restrict__ new_len,
                  const int32_t *__restrict__ parents, const int32_t *__restrict__ free_pages, int64_t n_free,
                  int32_t *__restrict__ table, int64_t B, uint32_t width, uint32_t page, int64_t max_tokens,
                  int32_t *__restrict__ cu_new, int64_t *__restrict__ slots, int32_t *__restrict__ positions,
                  uint4 *__restrict__ mask, int32_t *__restrict__ taken) {
    __shared__ uint4 s_mask[kPlanWarps][kMaxDraft];
    __shared__ int16_t s_anc[kPlanWarps][kMaxDraft];
    __shared__ int64_t s_sum[kPlanWarps][3];
    __shared__ int32_t s_n[kPlanWarps];
    __shared__ int64_t s_take[kPlanWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t b0 = (int64_t)blockIdx.x * kPlanWarps, b = b0 + warp;

    // this warp's request
    const bool mine = b < B;
    const uint32_t ctx = mine ? (uint32_t)max(__ldg(ctx_len + b), 0) : 0u;
    const int n = mine ? plan_new(new_len, b) : 0;
    uint32_t have, need;
    plan_blocks(ctx, (uint32_t)n, page, width, have, need);
    const int64_t take = mine && need > have ? (int64_t)(need - have) : 0;
    if (lane == 0) {
        s_n[warp] = n;
        s_take[warp] = take;
    }

    // sums over the requests before this block's, and the total of new_len
    int64_t tok = 0, pages = 0, all = 0;
    for (int64_t i = tid; i < B; i += 32 * kPlanWarps) {
        const int ni = plan_new(new_len, i);
        all += ni;
        if (i < b0) {
            uint32_t h, q;
            plan_blocks((uint32_t)max(__ldg(ctx_len + i), 0), (uint32_t)ni, page, width, h, q);
            tok += ni;
            pages += q > h ? q - h : 0u;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        tok += __shfl_xor_sync(0xffffffffu, tok, o);
        pages += __shfl_xor_sync(0xffffffffu, pages, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 0) {
        s_sum[warp][0] = tok;
        s_sum[warp][1] = pages;
        s_sum[warp][2] = all;
    }
    __syncthreads();
    tok = pages = all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        tok += s_sum[w][0];
        pages += s_sum[w][1];
        all += s_sum[w][2];
        if (w < warp) {
            tok += s_n[w];
            pages += s_take[w];
        }
    }

    // unused places at the end of the per-token outputs
    for (int64_t t = all + (int64_t)blockIdx.x * blockDim.x + tid; t < max_tokens; t += (int64_t)gridDim.x * blockDim.x) {
        slots[t] = -1;
        positions[t] = 0;
        mask[t] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (b == 0 && lane == 0) cu_new[0] = 0;
    if (!mine) return;
    if (lane == 0) {
        cu_new[b + 1] = (int32_t)(tok + n);
        if (b == B - 1) taken[0] = (int32_t)(pages + take);
    }

    int32_t *row = table + b * (int64_t)width;
    for (int64_t j = lane; j < take; j += 32) row[have + j] = pages + j < n_free ? __ldg(free_pages + pages + j) : -1;

    // ancestors
    uint4 m[kMaxDraft / 32];
    int anc[kMaxDraft / 32];
#pragma unroll
    for (int c = 0; c < kMaxDraft / 32; ++c) {
        const int i = 32 * c + lane;
        int p = -1;
        if (i < n) {
            p = i - 1;
            if (parents) p = tok + i < max_tokens ? __ldg(parents + tok + i) : -1;
        }
        anc[c] = p >= 0 && p < i ? p : -1;
        const uint32_t bit = i < n ? 1u << lane : 0u;
        m[c] = make_uint4(c == 0 ? bit : 0u, c == 1 ? bit : 0u, c == 2 ? bit : 0u, c == 3 ? bit : 0u);
        s_mask[warp][i] = m[c];
        s_anc[warp][i] = (int16_t)anc[c];
    }
    __syncwarp();
    bool more = true;
    for (int r = 0; r < 7 && more; ++r) {
        bool any = false;
#pragma unroll
        for (int c = 0; c < kMaxDraft / 32; ++c) {
            if (anc[c] >= 0) {
                const uint4 o = s_mask[warp][anc[c]];
                m[c].x |= o.x;
                m[c].y |= o.y;
                m[c].z |= o.z;
                m[c].w |= o.w;
                anc[c] = s_anc[warp][anc[c]];
                any |= anc[c] >= 0;
            }
        }
        more = __any_sync(0xffffffffu, any);
        __syncwarp();  // all reads of this round before its writes
        if (more) {
#pragma unroll
            for (int c = 0; c < kMaxDraft / 32; ++c) {
                s_mask[warp][32 * c + lane] = m[c];
                s_anc[warp][32 * c + lane] = (int16_t)anc[c];
            }
            __syncwarp();
        }
    }
#pragma unroll
    for (int c = 0; c < kMaxDraft / 32; ++c) {
        const int i = 32 * c + lane;
        const int64_t t = tok + i;
        if (i >= n || t >= max_tokens) continue;
        const uint32_t at = ctx + (uint32_t)i, blk = at / page;
        int32_t id = -1;
        if (blk < width) {
            if (blk < have) id = __ldg(row + blk);  // entries the launch only reads
            else if (pages + (blk - have) < n_free) id = __ldg(free_pages + pages + (blk - have));
        }
        slots[t] = id >= 0 ? (int64_t)id * page + at % page : -1;
        positions[t] = (int32_t)(ctx + __popc(m[c].x) + __popc(m[c].y) + __popc(m[c].z) + __popc(m[c].w) - 1);
        mask[t] = m[c];
    }
}

// ---------------------------------------------------------------- norm, rotation, store

constexpr int kPasses = 4;  // head groups of a warp: they share its angles, addresses and checks

struct RopeParams {
    const void *qkv;
    const float *wq, *wk, *cos_sin;
    const int32_t *positions;
    const int64_t *slots;
    void *q_out, *kc, *vc;
    int64_t ld, T, max_pos, n_slots;
    int64_t page_stride, token_stride, head_stride;
    int D, rot, inter, Hq, Hkv;
    uint32_t page_size;
    int lanes, lanes2;  // lanes of a head (8 values each), and that rounded up to a power of two
    int groups;         // warps that share a token's heads
    float eps;
};

// A lane holds two runs of 4 values of a head, lanes2 lanes a head, so that a
// warp holds 1 to 32 heads of one token.  The two runs are rot/2 apart in the
// rotated part, so a half-split pair lies in one lane (an interleaved pair does
// anyway); only the sum of squares takes shuffles.  The cosines and sines stay
// in registers over the heads that a warp walks.  Bound by the instructions it
// issues (70 % of the issue slots), then by memory: 8 values a lane in packed
// pairs, no per-value shuffle, no branch in the sum, values copied without
// arithmetic.  4096 tokens of 48 heads of 128, bf16: 23.7 us, 4.3 TB/s (one
// shuffle for each value of a half-split pair: 28.7 us; 8 head groups a warp in
// place of 4: 27.2 us).
template <typename TI, typename TO>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeParams p) {
    const int lane = threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.z + threadIdx.z;
    const int group = blockIdx.y * blockDim.y + threadIdx.y;
    if (t >= p.T || group >= p.groups) return;
    const int per_warp = 32 / p.lanes2, sub = lane / p.lanes2, l = lane & (p.lanes2 - 1);
    const bool live = l < p.lanes;
    const int heads = p.Hq + 2 * p.Hkv;
    // first values of the lane's runs: the rotated part in halves, then the rest in halves
    const int rl = p.rot / 8;
    const bool rotated = l < rl;
    const int i0 = rotated ? 4 * l : p.rot + 4 * (l - rl);
    const int i1 = i0 + (rotated ? p.rot / 2 : (p.D - p.rot) / 2);

    // the token's heads (queries, keys, values) dealt to its warps in turn, at most kPasses a
    // warp (the launch sees to that), all of them requested before the first is worked on
    const TI *in = static_cast<const TI *>(p.qkv) + t * p.ld;
    Raw4<TI> raw[kPasses][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int h = (group + i * p.groups) * per_warp + sub;
#pragma unroll
        for (int e = 0; e < (int)sizeof(TI); ++e) raw[i][0].r[e] = raw[i][1].r[e] = 0u;
        if (live && h < heads) {
            raw[i][0] = load4(in + h * p.D + i0);
            raw[i][1] = load4(in + h * p.D + i1);
        }
    }
    const int pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_pos) return;  // the token is left out
    const int64_t slot = __ldg(p.slots + t);
    const bool stored = slot >= 0 && slot < p.n_slots;
    int64_t cache_at = 0;
    if (stored) {
        const int64_t pg = p.n_slots <= 0xFFFFFFFFll ? (uint32_t)slot / p.page_size : slot / (int64_t)p.page_size;
        cache_at = pg * p.page_stride + (slot - pg * p.page_size) * p.token_stride;
    }
    // angles: half split, those of the pairs (i0 + e, i1 + e); interleaved, of the pairs in both runs
    float cs[4], sn[4];
    if (rotated) {
        const float *c = p.cos_sin + (int64_t)pos * p.rot, *s = c + p.rot / 2;
        if (p.inter) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(c + i0 / 2)), b = __ldg(reinterpret_cast<const float2 *>(c + i1 / 2));
            const float2 d = __ldg(reinterpret_cast<const float2 *>(s + i0 / 2)), e = __ldg(reinterpret_cast<const float2 *>(s + i1 / 2));
            cs[0] = a.x; cs[1] = a.y; cs[2] = b.x; cs[3] = b.y;
            sn[0] = d.x; sn[1] = d.y; sn[2] = e.x; sn[3] = e.y;
        } else {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(c + i0)), d = __ldg(reinterpret_cast<const float4 *>(s + i0));
            cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
            sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w;
        }
    }
    TO *q_row = static_cast<TO *>(p.q_out) + t * p.Hq * p.D;
    TO *k_row = static_cast<TO *>(p.kc) + cache_at, *v_row = static_cast<TO *>(p.vc) + cache_at;
    const float inv_d = 1.0f / (float)p.D;

#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int h0 = (group + i * p.groups) * per_warp, h = h0 + sub;
        if (h0 >= heads) break;
        const bool on = live && h < heads;
        float v[8];
        unpack4<TI>(raw[i][0], v);
        unpack4<TI>(raw[i][1], v + 4);
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        if (h0 < p.Hq + p.Hkv) {  // some head of the warp is a query or a key
            const float *w = is_q ? p.wq : p.wk;
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
            if (on && !is_v) {
                if (w) {
                    const float r = rsqrtf(ss * inv_d + p.eps);
                    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + i0)), w1 = __ldg(reinterpret_cast<const float4 *>(w + i1));
                    const uint64_t rr = f32x2(r, r);
                    const uint64_t ws[4] = {f32x2(w0.x, w0.y), f32x2(w0.z, w0.w), f32x2(w1.x, w1.y), f32x2(w1.z, w1.w)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f32x2_split(f32x2_mul(f32x2(v[2 * e], v[2 * e + 1]), f32x2_mul(rr, ws[e])), v[2 * e], v[2 * e + 1]);
                }
                if (!rotated) {
                } else if (p.inter) {
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
        }
        if (!on || !(is_q || stored)) continue;
        const int hk = h - p.Hq - (is_v ? p.Hkv : 0);
        TO *d = (is_q ? q_row : is_v ? v_row : k_row) + (is_q ? (int64_t)(h * p.D) : hk * p.head_stride);
        store4(d + i0, v);
        store4(d + i1, v + 4);
    }
}

template <typename TI>
cudaError_t rope_launch(const RopeParams &p, int out_type, dim3 grid, dim3 block, cudaStream_t st) {
    switch (out_type) {
        case W4_F32: qk_norm_rope_kernel<TI, float><<<grid, block, 0, st>>>(p); break;
        case W4_BF16: qk_norm_rope_kernel<TI, __nv_bfloat16><<<grid, block, 0, st>>>(p); break;
        default: qk_norm_rope_kernel<TI, __half><<<grid, block, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_draft_plan(const int32_t *ctx_len, const int32_t *new_len, const int32_t *parents,
                              const int32_t *free_pages, int64_t n_free, int32_t *table, int64_t B, int64_t width,
                              int32_t page_size, int64_t max_tokens, int32_t *cu_new, int64_t *slots,
                              int32_t *positions, uint32_t *mask, int32_t *taken, cudaStream_t st) {
    draft_plan_kernel<<<(unsigned)ceil_div(B, kPlanWarps), 32 * kPlanWarps, 0, st>>>(
        ctx_len, new_len, parents, free_pages, n_free, table, B, (uint32_t)width, (uint32_t)page_size, max_tokens,
        cu_new, slots, positions, reinterpret_cast<uint4 *>(mask), taken);
    return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const void *qkv, int32_t x_type, int64_t ld, int64_t T, int32_t q_heads,
                                const float *wq, const float *wk, float eps, const int32_t *positions,
                                const float *cos_sin, int64_t max_pos, int32_t rot, int32_t interleaved,
                                const int64_t *slots, const w4_paged_cache &c, void *q_out, cudaStream_t st) {
    RopeParams p = {};
    p.qkv = qkv; p.wq = wq; p.wk = wk; p.cos_sin = cos_sin; p.positions = positions; p.slots = slots;
    p.q_out = q_out; p.kc = c.k; p.vc = c.v;
    p.ld = ld; p.T = T; p.max_pos = max_pos; p.n_slots = c.pages * (int64_t)c.page_size;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.D = c.head_dim; p.rot = rot; p.inter = interleaved != 0; p.Hq = q_heads; p.Hkv = c.heads;
    p.page_size = (uint32_t)c.page_size;
    p.eps = eps;
    p.lanes = c.head_dim / 8;
    p.lanes2 = 1;
    while (p.lanes2 < p.lanes) p.lanes2 *= 2;
    // kPasses head groups a warp; few tokens are spread over more warps, until the machine
    // (152 SMs x 64 warps) has one round.
    const int64_t iters = ceil_div((int64_t)q_heads + 2 * (int64_t)c.heads, 32 / p.lanes2);
    p.groups = (int)std::max<int64_t>(ceil_div(iters, kPasses), std::min<int64_t>(iters, 152 * 64 / std::max<int64_t>(1, T)));
    const unsigned by = (unsigned)std::min(p.groups, 8), bz = 8 / by;
    const dim3 block(32, by, bz), grid((unsigned)ceil_div(T, bz), (unsigned)ceil_div(p.groups, by));
    if (grid.y > 65535) return cudaErrorInvalidConfiguration;
    switch (x_type) {
        case W4_F32: return rope_launch<float>(p, c.type, grid, block, st);
        case W4_BF16: return rope_launch<__nv_bfloat16>(p, c.type, grid, block, st);
        default: return rope_launch<__half>(p, c.type, grid, block, st);
    }
}

}  // namespace w4
