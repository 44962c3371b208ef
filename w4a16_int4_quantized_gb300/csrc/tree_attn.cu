// tree_attn.cu -- attention of drafted token trees over a paged cache (tcgen05).
//
// A unit of work is (request, key head, row tiles, split): the rows are (drafted
// token, query head of the key head's group), 128 at most to a tile, and a
// split is a range of keys.  Its CTA runs over the range in tiles of 64 keys:
//   softmax warps  four to a row tile, one thread a row: S to registers, the
//                  mask where the tile reaches the drafted tokens, the running
//                  maximum and sum, P in 16 bits back over S;
//   TMA producers  the query tiles once, then the key and the value tiles (their
//                  pages through the block table), a ring and a warp for each;
//   MMA issuers    a warp for each row tile: S = Q K^T (M = 128 rows, N = 64
//                  keys) into one of two TMEM buffers, O += P V with P read
//                  from TMEM.
// Up to 128 rows a request and key head: one row tile to a CTA, two CTAs an SM
// (head_dim <= 128), so one's softmax runs under the other's products.  More:
// two row tiles to a CTA, one CTA an SM, which halves the reads of keys and
// values (both from L2 and into shared memory).
// O is rescaled only when a row's maximum has grown by more than 2^8: P then
// stays below 2^8, exact up to its rounding, and the common factor cancels in O / l.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kRows = 128;  // rows of a tile (TMEM lanes)
constexpr int kKeys = 64;   // keys of a tile
constexpr float kGrow = 8.0f;  // log2 by which a maximum may grow before O is rescaled
constexpr int kMaxSplits = 64;

struct AttnParams {
    CUtensorMap qmap;  // [T][Hq][D], box {64, G, tokens of a tile}
    CUtensorMap kmap, vmap;  // pages, then tokens and heads in the order of their strides, D; a box: 64 values, min(page, 64) tokens
    const int32_t *table, *ctx_len, *cu_new;
    const uint4 *mask;
    const uint16_t *v;  // for the exact treatment of NaN and infinities in drafted values
    uint16_t *out;
    float *part_o;   // [unit][split][rows of a tile][DP]
    float2 *part_ml; // [unit][split][rows of a tile]: maximum (log2), sum
    uint32_t *status;
    int64_t width, T, pages, page_stride, token_stride, head_stride;
    int B, Hq, Hkv, G, D;
    int page_shift;
    int tok_inner;  // the token stride is the smaller one
    int tpt;     // drafted tokens of a row tile
    int mtiles, mgroups, splits, chunk;  // chunk: keys of a split, a multiple of kKeys
    int max_new;
    float scale_log2;
};

struct Ctl {
    uint64_t q_full;
    uint64_t full[2][8], empty[2][8];  // [keys, values][stage]
    uint64_t s_full[2][2], p_full[2][2], o_done[2], o_last[2];  // [row tile][S buffer]; o_last: the last product
    uint64_t v_clean[2];  // the values of an edge tile have been gone over (edge tiles in turn)
    uint32_t tmem_base;
    int abort;
    int bad;  // a drafted value of this range is not finite
};

// DP: head_dim rounded up to whole chunks of 64; RT: row tiles of a CTA.
template <int DP, int RT>
struct Cfg {
    static_assert(RT == 1 || DP <= 128, "TMEM holds two row tiles up to 128 values");
    static constexpr int kChunks = DP / 64;
    static constexpr int kQTile = kRows * DP * 2;
    static constexpr int kTile = kKeys * DP * 2;
    static constexpr int kCtas = RT == 1 && DP <= 128 ? 2 : 1;
    static constexpr int kSmemMost = 233472 / kCtas - 1024;
    static constexpr int kFit = (kSmemMost - RT * kQTile - (int)sizeof(Ctl)) / kTile;
    // a ring for the keys, and a longer one for the values, which wait for the softmax
    static constexpr int kKStages = kFit / 2 < 8 ? kFit / 2 : 8, kVStages = kFit - kKStages < 8 ? kFit - kKStages : 8;
    static constexpr int kSmem = RT * kQTile + (kKStages + kVStages) * kTile + (int)sizeof(Ctl);
    static constexpr uint32_t kTmem = kCtas == 2 ? 256 : 512;
    static constexpr uint32_t kOCol = RT * 2 * kKeys;  // the S buffers first, then the O of each row tile
    static_assert(kOCol + RT * DP <= kTmem, "TMEM");
    static constexpr int kSoftWarps = 4 * RT, kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 2;
    static constexpr int kThreads = 32 * (kSoftWarps + 2 + RT);
};

W4_DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two f32 in one register pair, for the packed arithmetic.
W4_DEV uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
W4_DEV void f32x2_split(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
W4_DEV uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
W4_DEV uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <bool BF>
W4_DEV uint32_t pack2(float a, float b) {
    if constexpr (BF) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

template <bool BF>
W4_DEV float to_f32(uint16_t u) {
    if constexpr (BF) return __uint_as_float((uint32_t)u << 16);
    else return __half2float(__ushort_as_half(u));
}

// All exponent bits set: NaN or infinity.  Of the two values in a word, any.
template <bool BF>
W4_DEV bool any_nonfinite(uint32_t w) {
    constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

// Request b's drafted tokens and keys, in bounds whatever the arrays hold.
struct Request {
    int64_t t0;  // its first drafted token
    int n, ctx, len;
};
W4_DEV Request request_of(const AttnParams &p, int b) {
    Request r;
    const int64_t c0 = max(__ldg(p.cu_new + b), 0), c1 = min((int64_t)__ldg(p.cu_new + b + 1), p.T);
    r.t0 = c0;
    r.n = (int)max((int64_t)0, min(c1 - c0, (int64_t)W4_MAX_DRAFT));
    const int64_t top = min(p.width << p.page_shift, (int64_t)0x7FFFFF00);
    r.ctx = (int)min((int64_t)max(__ldg(p.ctx_len + b), 0), top);
    r.len = (int)min((int64_t)r.ctx + r.n, top);
    return r;
}

template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(Cfg<DP, RT>::kThreads, Cfg<DP, RT>::kCtas)
tree_attn_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<DP, RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tile = smem;
    uint8_t *k_ring = smem + RT * C::kQTile, *v_ring = k_ring + C::kKStages * C::kTile;
    Ctl *ctl = reinterpret_cast<Ctl *>(v_ring + C::kVStages * C::kTile);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // block -> (request, key head, split, row tiles); row tiles of a split next to
    // one another, so that they read its keys from L2 together
    int u = blockIdx.x;
    const int mg = u % p.mgroups;
    u /= p.mgroups;
    const int split = u % p.splits;
    u /= p.splits;
    const int h = u % p.Hkv, b = u / p.Hkv;
    griddep_launch_dependents();
    const Request rq = request_of(p, b);
    const int drafted = min(rq.n, p.max_new), tok_first = mg * RT * p.tpt;  // of the CTA
    const int k_begin = split * p.chunk;
    const int k_end = split == p.splits - 1 ? rq.len : min(rq.len, k_begin + p.chunk);
    if (tok_first >= drafted || k_begin >= k_end) return;
    const int tiles = RT == 1 || tok_first + p.tpt >= drafted ? 1 : 2;  // row tiles with rows
    const int nt = (k_end - k_begin + kKeys - 1) / kKeys;

    if (tid == 0) {
        mbar_init(&ctl->q_full, 1);
        for (int i = 0; i < 2; ++i)
            for (int s = 0; s < 8; ++s) {
                mbar_init(&ctl->full[i][s], 1);
                mbar_init(&ctl->empty[i][s], tiles);  // each row tile's products release a stage
            }
        for (int r = 0; r < RT; ++r) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl->s_full[r][i], 1);
                mbar_init(&ctl->p_full[r][i], 4);
            }
            mbar_init(&ctl->o_done[r], 1);
            mbar_init(&ctl->o_last[r], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&ctl->v_clean[i], 4 * tiles);
        ctl->abort = 0;
        ctl->bad = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&ctl->tmem_base, C::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    int *abort = &ctl->abort;

    if (warp == C::kLoadWarp || warp == C::kLoadWarp + 1) {
        // ---------------- TMA producers, one for the keys and one for the values (issuing a tile's boxes takes
        // about half of the tile's time): the whole warp walks, one lane issues
        const bool keys = warp == C::kLoadWarp;
        const uint32_t lead = elect_lead();
        const int page_rows = min(1 << p.page_shift, kKeys), page_log = min(p.page_shift, 6);  // rows of a box
        const int pages = kKeys >> page_log;                                                   // of a tile
        if (keys && lane == 0) {
            mbar_arrive_expect_tx(&ctl->q_full, (uint32_t)(tiles * C::kChunks * p.G * p.tpt * 128));
            for (int r = 0; r < tiles; ++r)
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load_3d(q_tile + r * C::kQTile + c * (kRows * 128), &p.qmap, 64 * c, h * p.G,
                                (int)(rq.t0 + tok_first + r * p.tpt), &ctl->q_full);
        }
        __syncwarp();
        // lane i: the block-table entry of box i of tile j, -1 where there is none; read two
        // tiles ahead and looked at only when it is used, or each tile would wait for it
        const int32_t *row = p.table + (int64_t)b * p.width;
        auto entry_of = [&](int j) {
            const int key = k_begin + j * kKeys + lane * page_rows;
            return lane < pages && j < nt && key < rq.len ? __ldg(row + (key >> p.page_shift)) : -1;
        };
        const CUtensorMap *map = keys ? &p.kmap : &p.vmap;
        uint64_t *full = ctl->full[keys ? 0 : 1], *empty = ctl->empty[keys ? 0 : 1];
        const uint32_t ring = smem_u32(keys ? k_ring : v_ring);
        const int stages = keys ? C::kKStages : C::kVStages;
        int stage = 0, round = 0;
        int now = entry_of(0), next = entry_of(1);
        for (int j = 0; j < nt; ++j) {
            if (round > 0 && !wait_warp(&empty[stage], (round - 1) & 1, abort, p.status)) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::kTile);
            __syncwarp();
            // no page: the page count, which is out of the map and read as zeros
            const int id = now < 0 || now >= p.pages ? (int)p.pages : now;
            now = next;
            next = entry_of(j + 2);
            const uint32_t dst = ring + (uint32_t)(stage * C::kTile), bar = smem_u32(&full[stage]);
            // a page of 64 or more: the tile's place in it; else its boxes are whole pages
            const int off = (k_begin + j * kKeys) & ((1 << p.page_shift) - 1);
            const int c1 = p.tok_inner ? off : h, c2 = p.tok_inner ? h : off;
            for (int i = 0; i < pages; ++i) {
                const int page = __shfl_sync(0xffffffffu, id, i);
#pragma unroll
                for (int ch = 0; ch < C::kChunks; ++ch)
                    tma_load_4d_lead(dst + (uint32_t)(ch * (kKeys * 128) + ((i << page_log) * 128)), map, 64 * ch, c1, c2, page,
                                     bar, lead);
            }
            if (++stage == stages) stage = 0, ++round;
        }
    } else if (warp >= C::kMmaWarp) {
        // ---------------- MMA issuers, one for each row tile: the whole warp walks, one lane issues
        const int r = warp - C::kMmaWarp;
        if (r < tiles) {
            const uint32_t lead = elect_lead();
            constexpr uint32_t fmt = BF ? 1u : 0u;
            constexpr uint32_t id_s = idesc_f16(fmt, kRows, kKeys);
            constexpr uint32_t id_o = idesc_f16(fmt, kRows, DP) | (1u << 16);  // B (the values) with its N axis contiguous
            const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tile + r * C::kQTile)), k_desc = smem_desc_sw128(smem_u32(k_ring)),
                           v_desc = smem_desc_mn_sw128(smem_u32(v_ring), kKeys * 128);
            const uint32_t s_col = tmem + (uint32_t)(2 * r * kKeys), o_col = tmem + C::kOCol + (uint32_t)(r * DP);
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                ok = ok && wait_warp(bar, parity, abort, p.status);
            };
            int ks = 0, kr = 0, vs = 0, vr = 0, edges = 0;  // the rings' stages and rounds
            auto issue_s = [&](int j) {
                wait(&ctl->full[0][ks], kr & 1);
                // it goes where P of tile j - 2 stood, whose product must be through
                if (j >= 2) wait(&ctl->o_done[r], j & 1);
                if (!ok) return;
                tc_fence_after();
                const uint64_t kd = desc_at(k_desc, (uint32_t)(ks * C::kTile));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    umma_f16_lead(s_col + (uint32_t)((j & 1) * kKeys), desc_at(q_desc, (k / 4) * (kRows * 128) + (k % 4) * 32),
                                  desc_at(kd, (k / 4) * (kKeys * 128) + (k % 4) * 32), id_s, k > 0 ? 1u : 0u, lead);
                umma_commit_lead(&ctl->s_full[r][j & 1], lead);
                umma_commit_lead(&ctl->empty[0][ks], lead);
                if (++ks == C::kKStages) ks = 0, ++kr;
            };
            wait(&ctl->q_full, 0);
            if (ok) issue_s(0);
            for (int j = 0; j < nt && ok; ++j) {
                if (j + 1 < nt) issue_s(j + 1);
                wait(&ctl->full[1][vs], vr & 1);
                if (k_begin + (j + 1) * kKeys > rq.ctx) {
                    wait(&ctl->v_clean[edges & 1], (edges >> 1) & 1);
                    ++edges;
                }
                wait(&ctl->p_full[r][j & 1], (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = desc_at(v_desc, (uint32_t)(vs * C::kTile));
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    umma_f16_ts_lead(o_col, s_col + (uint32_t)((j & 1) * kKeys + 8 * k), desc_at(vd, k * 2048), id_o,
                                     (j > 0 || k > 0) ? 1u : 0u, lead);
                umma_commit_lead(&ctl->o_done[r], lead);
                if (j == nt - 1) umma_commit_lead(&ctl->o_last[r], lead);
                umma_commit_lead(&ctl->empty[1][vs], lead);
                if (++vs == C::kVStages) vs = 0, ++vr;
            }
        }
        __syncwarp();
    } else if ((warp >> 2) < tiles) {
        // ---------------- softmax: thread = row
        const int rt = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
        const int tok0 = tok_first + rt * p.tpt, mt = mg * RT + rt;
        const int rows = min(p.tpt, drafted - tok0) * p.G;
        const bool active = 32 * quad < rows;  // of the warp
        const int tok = row / p.G, g = row - tok * p.G;
        const bool mine = row < rows;
        const int64_t t = rq.t0 + tok0 + tok;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
        const uint32_t o_col = C::kOCol + (uint32_t)(rt * DP);
        // the row's mask over its request's drafted tokens, later bits cleared (read where it
        // is needed: the few tiles that reach them)
        auto row_mask = [&](uint64_t &lo, uint64_t &hi) {
            lo = hi = 0;
            if (!mine) return;
            const uint4 m = __ldg(p.mask + t);
            lo = m.x | ((uint64_t)m.y << 32);
            hi = m.z | ((uint64_t)m.w << 32);
            const int kept = rq.len - rq.ctx;  // drafted tokens with a place in the block table
            if (kept < 64) {
                lo &= (1ull << kept) - 1;
                hi = 0;
            } else if (kept < 128) {
                hi &= (1ull << (kept - 64)) - 1;
            }
        };
        float mx = -INFINITY, l = 0.0f;  // the maximum that P is relative to (log2 units), the sum
        int edges = 0;  // edge tiles so far
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            ok = wait_warp(&ctl->s_full[rt][j & 1], (j >> 1) & 1, abort, p.status);
            if (!ok) break;
            tc_fence_after();
            const int key0 = k_begin + j * kKeys;
            const bool edge = key0 + kKeys > rq.ctx;  // reaches the drafted tokens or the end
            if (edge) {
                // Values that no row may see become zeros (P is zero there, but 0 * NaN is
                // not); drafted values that are not finite too, and are added at the end.
                const int s = j % C::kVStages;
                ok = wait_warp(&ctl->full[1][s], (j / C::kVStages) & 1, abort, p.status);
                if (!ok) break;
                uint8_t *vt = v_ring + s * C::kTile;
                bool bad = false;
                for (int i = tid; i < C::kChunks * kKeys * 8; i += 128 * tiles) {
                    const int key = key0 + ((i >> 3) & (kKeys - 1));
                    uint4 *at = reinterpret_cast<uint4 *>(vt + i * 16);
                    if (key >= rq.len) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (key >= rq.ctx) {
                        uint4 w = *at;
                        if (any_nonfinite<BF>(w.x) || any_nonfinite<BF>(w.y) || any_nonfinite<BF>(w.z) ||
                            any_nonfinite<BF>(w.w)) {
                            bad = true;
                            uint32_t *e = reinterpret_cast<uint32_t *>(&w);
                            constexpr uint32_t x = BF ? 0x7F80u : 0x7C00u;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                if ((e[c] & x) == x) e[c] &= 0xFFFF0000u;
                                if (((e[c] >> 16) & x) == x) e[c] &= 0x0000FFFFu;
                            }
                            *at = w;
                        }
                    }
                }
                if (bad) ctl->bad = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->v_clean[edges & 1]);
                ++edges;
            }
            if (active) {
                uint32_t sr[kKeys];
                tmem_ld64(tmem + lane_off + (uint32_t)((2 * rt + (j & 1)) * kKeys), sr);
                float top;
                if (edge) {
                    // which of the tile's 64 keys this row sees
                    uint64_t mlo, mhi;
                    row_mask(mlo, mhi);
                    const int j0 = key0 - rq.ctx;
                    uint64_t see;
                    if (j0 >= 64) see = j0 < 128 ? mhi >> (j0 - 64) : 0ull;
                    else if (j0 > 0) see = (mlo >> j0) | (mhi << (64 - j0));
                    else if (j0 == 0) see = mlo;
                    else see = (mlo << -j0) | ((1ull << -j0) - 1);  // -64 < j0 < 0
#pragma unroll
                    for (int c = 0; c < kKeys; ++c)
                        if (!((see >> c) & 1)) sr[c] = 0xFF800000u;
                }
                {
                    float part[4];  // four chains
#pragma unroll
                    for (int c = 0; c < 4; ++c) part[c] = fmaxf(__uint_as_float(sr[c]), __uint_as_float(sr[c + 4]));
#pragma unroll
                    for (int c = 8; c < kKeys; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            part[i] = fmaxf(part[i], fmaxf(__uint_as_float(sr[c + i]), __uint_as_float(sr[c + i + 4])));
                    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                }
                // scale > 0: the maximum scales along
                const float now = fmaxf(mx, top * p.scale_log2);
                const bool grow = mine && now > mx + kGrow;  // true for the first finite maximum: mx is -inf
                if (__any_sync(0xffffffffu, grow)) {
                    if (j > 0) {
                        // every product so far is through, then O *= 2^(old - new)
                        ok = wait_warp(&ctl->o_done[rt], (j - 1) & 1, abort, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        const float f = now == -INFINITY ? 1.0f : exp2_fast(mx - now);
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tmem + lane_off + o_col + 32 * c, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tmem + lane_off + o_col + 32 * c, o);
                        }
                    }
                    mx = now;
                }
                const float base = mx == -INFINITY ? 0.0f : mx;
                const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2), base2 = f32x2(-base, -base);
                uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < kKeys; c += 2) {
                    float a, e;
                    f32x2_split(f32x2_fma(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, base2), a, e);
                    a = exp2_fast(a);
                    e = exp2_fast(e);
                    sum2[(c / 2) & 3] = f32x2_add(sum2[(c / 2) & 3], f32x2(a, e));
                    sr[c / 2] = pack2<BF>(a, e);
                }
                float sa, sb;
                f32x2_split(f32x2_add(f32x2_add(sum2[0], sum2[1]), f32x2_add(sum2[2], sum2[3])), sa, sb);
                l += sa + sb;
                tmem_st32(tmem + lane_off + (uint32_t)((2 * rt + (j & 1)) * kKeys), sr);
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->p_full[rt][j & 1]);
        }
        // ---------------- the range's result
        if (ok) {
            ok = wait_or_abort(&ctl->o_last[rt], 0, abort, p.status);
            // the other warps' word on `bad` (already there: the last product followed it)
            if (ok && edges) ok = wait_warp(&ctl->v_clean[(edges - 1) & 1], ((edges - 1) >> 1) & 1, abort, p.status);
        }
        if (ok && active) {
            tc_fence_after();
            const bool bad = *reinterpret_cast<volatile int *>(&ctl->bad) != 0;
            const float inv = p.splits > 1 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
            const int64_t unit = (int64_t)(b * p.Hkv + h) * p.mtiles + mt;
            const int64_t prow = (unit * p.splits + split) * (p.tpt * p.G) + row;
            if (p.splits > 1 && mine) p.part_ml[prow] = make_float2(mx, l);
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_off + o_col + 32 * c, o);
                if (!mine) continue;
                // a row that sees nothing: O is a sum of zeros, P having been zero throughout
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                if (bad) {
                    uint64_t mlo, mhi;
                    row_mask(mlo, mhi);
                    for (int jd = max(0, k_begin - rq.ctx); jd < k_end - rq.ctx; ++jd) {
                        if (!((jd < 64 ? mlo >> jd : mhi >> (jd - 64)) & 1)) continue;
                        const int key = rq.ctx + jd;
                        const int64_t id = __ldg(p.table + (int64_t)b * p.width + (key >> p.page_shift));
                        if (id < 0 || id >= p.pages) continue;
                        const uint16_t *vr = p.v + id * p.page_stride + h * p.head_stride +
                                             (int64_t)(key & ((1 << p.page_shift) - 1)) * p.token_stride;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int d = 32 * c + i;
                            const float x = d < p.D ? to_f32<BF>(vr[d]) : 0.0f;
                            if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                        }
                    }
                }
                if (p.splits > 1) {
                    float4 *d = reinterpret_cast<float4 *>(p.part_o + prow * DP + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                           __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                } else {
                    uint16_t *d = p.out + (t * p.Hq + h * p.G + g) * (int64_t)p.D + 32 * c;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (32 * c + 8 * i < p.D) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2<BF>(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
                            *reinterpret_cast<uint4 *>(d + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Joins the splits of a row: out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
// A warp a row, a lane every 32nd pair of values.
template <bool BF>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const __grid_constant__ AttnParams p, int DP) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int hq = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int b = blockIdx.x / p.max_new, i = blockIdx.x % p.max_new;
    const Request rq = request_of(p, b);
    if (hq >= p.Hq || i >= rq.n) return;
    const int h = hq / p.G, g = hq - h * p.G;
    const int mt = i / p.tpt;
    const int row = (i - mt * p.tpt) * p.G + g;
    const int used = min(p.splits, (rq.len + p.chunk - 1) / p.chunk);
    const int64_t unit = (int64_t)(b * p.Hkv + h) * p.mtiles + mt;
    const int64_t stride = (int64_t)p.tpt * p.G, r0 = unit * p.splits * stride + row;

    // lanes over the splits: kMaxSplits is two a lane
    float2 a = make_float2(-INFINITY, 0.0f), c = a;
    if (lane < used) a = p.part_ml[r0 + lane * stride];
    if (lane + 32 < used) c = p.part_ml[r0 + (lane + 32) * stride];
    float m = fmaxf(a.x, c.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.0f : m;
    const float wa = exp2_fast(a.x - base), wc = exp2_fast(c.x - base);
    float l = wa * a.y + wc * c.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;

    float2 acc[4] = {};
    for (int s = 0; s < used; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? wa : wc, s & 31);
        const float *o = p.part_o + (r0 + s * stride) * DP;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 2 * lane + 64 * e;
            if (d < p.D) {
                const float2 v = *reinterpret_cast<const float2 *>(o + d);
                // a split that the row sees nothing of has weight 0 and O = 0
                acc[e].x = fmaf(w, v.x, acc[e].x);
                acc[e].y = fmaf(w, v.y, acc[e].y);
            }
        }
    }
    uint16_t *d = p.out + ((rq.t0 + i) * p.Hq + hq) * (int64_t)p.D;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (2 * lane + 64 * e < p.D)
            *reinterpret_cast<uint32_t *>(d + 2 * lane + 64 * e) = pack2<BF>(acc[e].x * inv, acc[e].y * inv);
}

struct Split {
    int rt, tpt, mtiles, mgroups, splits, chunk;
    int64_t units;  // row tiles of all requests and key heads
};

int dp_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

Split split_of(int64_t B, int G, int Hkv, int D, int64_t max_len, int max_new) {
    Split s;
    s.mtiles = (int)ceil_div(max_new, kRows / G);
    s.tpt = (int)ceil_div(max_new, s.mtiles);  // even tiles
    s.mtiles = (int)ceil_div(max_new, s.tpt);
    s.rt = s.mtiles > 1 && D <= 128 ? 2 : 1;
    s.mgroups = (int)ceil_div(s.mtiles, s.rt);
    s.units = B * Hkv * s.mtiles;
    // The makespan of `n` splits on the machine's CTA slots, in keys: whole rounds
    // of a split's keys and a CTA's fixed cost (set-up and the write of its part).
    const int64_t slots = 152 * (D <= 128 && s.rt == 1 ? 2 : 1), tiles = ceil_div(max_len, kKeys);
    double best = 0;
    s.splits = 1;
    s.chunk = (int)(tiles * kKeys);
    for (int n = 1; n <= kMaxSplits; ++n) {
        const int64_t per = ceil_div(tiles, n);
        if (n > 1 && per < 2) break;
        const int64_t real = ceil_div(tiles, per);
        const double cost = (double)ceil_div(B * Hkv * s.mgroups * real, slots) * ((double)per * kKeys + 160) + (real > 1 ? 96 : 0);
        if (n == 1 || cost < best) {
            best = cost;
            s.splits = (int)real;
            s.chunk = (int)(per * kKeys);
        }
    }
    return s;
}

template <int DP, int RT, bool BF>
cudaError_t launch_attn(const AttnParams &p, cudaStream_t st) {
    using C = Cfg<DP, RT>;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [] {
        attr = cudaFuncSetAttribute(tree_attn_kernel<DP, RT, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (attr != cudaSuccess) return attr;
    const int64_t blocks = (int64_t)p.B * p.Hkv * p.mgroups * p.splits;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    tree_attn_kernel<DP, RT, BF><<<(unsigned)blocks, C::kThreads, C::kSmem, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.max_new), (unsigned)ceil_div(p.Hq, 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<BF>, p, DP);
}

template <bool BF>
cudaError_t launch_attn(const AttnParams &p, int rt, cudaStream_t st) {
    switch (dp_of(p.D)) {
        case 64: return rt == 2 ? launch_attn<64, 2, BF>(p, st) : launch_attn<64, 1, BF>(p, st);
        case 128: return rt == 2 ? launch_attn<128, 2, BF>(p, st) : launch_attn<128, 1, BF>(p, st);
        default: return launch_attn<256, 1, BF>(p, st);
    }
}

}  // namespace

size_t tree_attention_workspace(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t D, int64_t max_len,
                                int32_t max_new) {
    const Split s = split_of(B, q_heads / kv_heads, kv_heads, D, max_len, max_new);
    if (s.splits == 1) return 0;
    const int64_t rows = s.units * s.splits * s.tpt * (q_heads / kv_heads);
    return (size_t)rows * ((size_t)dp_of(D) * 4 + 8);
}

cudaError_t launch_tree_attention(const void *q, int64_t ld, const w4_paged_cache &c, const int32_t *table,
                                  int64_t width, const int32_t *ctx_len, const int32_t *cu_new, const uint32_t *mask,
                                  int64_t B, int64_t T, int32_t q_heads, float scale, int64_t max_len, int32_t max_new,
                                  void *out, void *workspace, uint32_t *status, cudaStream_t st) {
    AttnParams p = {};
    const int G = q_heads / c.heads, D = c.head_dim, DP = dp_of(D);
    const Split s = split_of(B, G, c.heads, D, max_len, max_new);
    if (B * max_new > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    p.table = table; p.ctx_len = ctx_len; p.cu_new = cu_new; p.mask = reinterpret_cast<const uint4 *>(mask);
    p.v = static_cast<const uint16_t *>(c.v);
    p.out = static_cast<uint16_t *>(out);
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.part_o + s.units * s.splits * s.tpt * G * DP);
    p.status = status;
    p.width = width; p.T = T; p.pages = c.pages;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.B = (int)B; p.Hq = q_heads; p.Hkv = c.heads; p.G = G; p.D = D;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.tpt = s.tpt; p.mtiles = s.mtiles; p.mgroups = s.mgroups; p.splits = s.splits; p.chunk = s.chunk;
    p.max_new = max_new;
    p.scale_log2 = scale * 1.44269504f;  // log2(e)
    const CUtensorMapDataType ty = c.type == W4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    {
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)q_heads, (uint64_t)T};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)ld * 2};
        const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)s.tpt};
        if (!encode_tmap(&p.qmap, ty, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    }
    // a tensor map's strides grow from dimension to dimension
    const int ti = c.token_stride < c.head_stride ? 1 : 2, hi = 3 - ti;
    p.tok_inner = ti == 1;
    uint64_t dims[4] = {(uint64_t)D, 0, 0, (uint64_t)c.pages}, strides[3] = {0, 0, (uint64_t)c.page_stride * 2};
    uint32_t box[4] = {64, 1, 1, 1};
    dims[ti] = (uint64_t)c.page_size;
    dims[hi] = (uint64_t)c.heads;
    strides[ti - 1] = (uint64_t)c.token_stride * 2;
    strides[hi - 1] = (uint64_t)c.head_stride * 2;
    box[ti] = (uint32_t)std::min(c.page_size, kKeys);
    if (!encode_tmap(&p.kmap, ty, 4, c.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap(&p.vmap, ty, 4, c.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return c.type == W4_BF16 ? launch_attn<true>(p, s.rt, st) : launch_attn<false>(p, s.rt, st);
}

}  // namespace w4
