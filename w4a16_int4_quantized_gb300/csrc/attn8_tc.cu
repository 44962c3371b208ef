// attn8_tc.cu -- the 8-bit attention of many rows (a prompt, or drafted tokens times query
// heads), on the tensor cores of the fifth generation.
//
// A unit of work is (request, key head, row tiles): rows are (new token, query head of the key
// head's group), 128 to a tile, two tiles to a CTA where there are more.  It is worked in steps of
// 64 keys (four blocks of 16), and the steps of all units, in one line, are dealt out evenly to
// persistent CTAs, one an SM; parts of units that were cut are joined by a second kernel.
// The roles of a CTA, each walking its segments on its own:
//   softmax warps  four to a row tile, one thread a row: the queries to f16 at a segment's start, S to
//                  registers, the mask, the running maximum and sum, P in f16 back over S; at the
//                  end O from TMEM to memory;
//   converters     four warps: codes to f16 (u = code + 128 under the byte 0x64 is 1024 + u, minus 1152:
//                  exact) in the layout that the products read;
//   producer       codes by TMA (a box for the 64 keys, or for each page of less), a step's scales beside them (the
//                  softmax reads them when S has come: no barrier of their own);
//   MMA issuers    a warp for each row tile: S = Q K^T into one of two TMEM buffers, O += P V with P
//                  read from TMEM.
// Scales are powers of two: a block's scale of the keys goes into the factor of its scores, that
// of the values into its weights, relative to the largest met so far in the segment (a new
// largest one moves O as a new maximum does).
// Measured: 2 requests of 1,024 and 2,048 tokens behind 3,000 and 6,000 (32 query and 8 key heads of 128, bf16)
// 340 us, 0.87 PFLOP/s (with `mma.sync`, 32 rows to a warp, 1,320).  A step takes about 2,900 cycles: the products
// 1,306 of the tensor pipe (S reads Q from shared memory for each 64 keys, 384 cycles a tile), the
// softmax of a tile about 1,950 beside the converters.  On the way: the values' scales in the exponent in
// place of a product for each weight 624 -> 423, one box for 64 keys in place of four 423 -> 381, parts
// written 32 rows at a time and a row's query asked for at once 381 -> 339.  Requests of few rows cost whole steps
// here: 63 of one token over 16,000 keys beside one of 512 tokens behind 4,000 take 1,185 us together, apart (the
// 63 by attn8.cu) 324 and 70.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attn8.cuh"
#include "common.cuh"
#include "smem_limit.h"
#include "tcgen05.cuh"

namespace w4 {
namespace {

constexpr int kTcRows = 128;  // of a tile (TMEM lanes)
constexpr int kTcKeys = 64;   // of a step
constexpr int kTcBlocks = kTcKeys / kKvBlock;
// Steps whose scales are kept: more than a softmax warp can be behind the producer, which writes step s + 8 when
// step s + 4 has been converted, and so the product of step s + 1 issued for both tiles.  Ahead of it the warps
// of a tile without rows may be any number of steps; they read a step's scales when its S has come.
constexpr int kScaleSlots = 8;

// A segment of a CTA's part of the line (it lies in one unit), and where the part goes on.
struct SegTc {
    int64_t at, end, base, t0;  // the next step, the part's end, the item's first step; the request's first row
    int item, b, h, k0, nt, tiles, whole, slot, row0, rows, ctx, len, sink, skip, blocks, inner0, inner1;
};

struct CtlTc {
    SegTc seg[16];  // a warp's
    uint64_t raw_full[4], raw_empty[4];
    uint64_t k_full[2], k_empty[2], v_full[3], v_empty[3];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2], o_last[2], o_free[2];  // [row tile][S buffer]
    uint64_t drained[2];
    float4 k_scale[kScaleSlots];  // of the step's blocks: the keys' scales (0 for NaN and none)
    int4 v_scale[kScaleSlots];    // the values' bytes, 0 for none
    int odd[kScaleSlots];         // bits n: keys or values of block n are NaN; 4 + n: no such page; 8 and on: the largest of the values' bytes below 255
    uint32_t tmem_base;
    int abort, begun;
    int64_t sums[16], base;
    int item;
};

// DP: head_dim rounded up; RT: row tiles of a CTA.
template <int DP, int RT>
struct CfgTc {
    static_assert(RT == 1 || DP <= 128, "TMEM holds two row tiles up to 128 values");
    static constexpr int kQTile = kTcRows * DP * 2, kTile = kTcKeys * DP * 2, kRaw = kTcKeys * DP * 2;  // raw: keys, then values
    static constexpr int kRawStages = DP == 256 ? 2 : 4, kKStages = DP == 256 ? 1 : 2, kVStages = DP == 256 ? 1 : 3;
    static constexpr int kSmem = RT * kQTile + (kKStages + kVStages) * kTile + kRawStages * kRaw + (int)sizeof(CtlTc);
    static_assert(kSmem <= 232448 - 1024, "shared memory");
    static constexpr uint32_t kTmem = 512, kOCol = RT * 2 * kTcKeys;
    static_assert(kOCol + RT * DP <= kTmem, "TMEM");
    static constexpr int kSoftWarps = 4 * RT, kConvWarp = kSoftWarps, kLoadWarp = kConvWarp + 4, kMmaWarp = kLoadWarp + 1;
    static constexpr int kThreads = 32 * (kMmaWarp + RT);
};

// The next segment of the CTA's part of the line, in the warp's place; false behind the last one.
// By a converged warp, every warp for itself.
template <int RT>
W4_DEV bool next_segment(const Attn8Params &p, SegTc *s, int lane) {
    __syncwarp();  // what was there has been read
    if (lane == 0) {
        int nt = 0;
        if (s->at < s->end) {
            int64_t at = s->at, base = s->base;
            Item it = item_of<kTcRows * RT>(p, s->item);
            while (at >= base + (int64_t)p.Hkv * it.nb) {  // (there are steps left, so there is an item with some)
                base += (int64_t)p.Hkv * it.nb;
                it = item_of<kTcRows * RT>(p, ++s->item);
            }
            const int off = (int)(at - base), h = (int)((unsigned)off / (unsigned)it.nb), k0 = off - h * it.nb;
            nt = (int)min((int64_t)(it.nb - k0), s->end - at);
            s->at = at + nt;
            s->base = base;
            s->t0 = it.r.t0;
            s->b = it.b; s->h = h; s->k0 = k0;
            s->tiles = RT == 1 || it.rows <= kTcRows ? 1 : 2;
            s->whole = nt == it.nb;
            s->slot = k0 > 0 ? 0 : 1;
            s->row0 = it.row0; s->rows = it.rows; s->ctx = it.r.ctx; s->len = it.r.len;
            s->sink = it.span.sink; s->skip = it.span.first - it.span.sink; s->blocks = it.span.blocks();
            // steps from `inner0` up to `inner1` have only keys that all rows see
            const int full = ((min(it.pos0, it.r.len - 1) + 1) >> kKvBlockLog) - s->skip;
            int from = 0;
            if (p.window > 0) from = max(s->sink, max(it.pos1 - p.window, -1) / kKvBlock + 1 - s->skip);
            if (p.window > 0 && it.pos1 - p.window < 0) from = s->sink;
            s->inner0 = (from + kTcBlocks - 1) / kTcBlocks - k0;
            s->inner1 = (full < s->sink ? 0 : full / kTcBlocks) - k0;
        }
        s->nt = nt;
    }
    __syncwarp();
    return *(volatile int *)&s->nt > 0;
}
// First key of block n of step j of the segment, -1 behind the last block.
W4_DEV int key_of(const volatile SegTc &s, int j, int n) {
    const int i = (s.k0 + j) * kTcBlocks + n;
    return i < s.blocks ? (i < s.sink ? i : i + s.skip) << kKvBlockLog : -1;
}

// The largest of three, given as bits.
W4_DEV float max3(uint32_t a, uint32_t b, uint32_t c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}

// The n lowest of 16 bits.
W4_DEV uint32_t below(int n) { return (1u << min(max(n, 0), 16)) - 1u; }

// 16 codes as f16, in two runs of 8.
W4_DEV void codes16(const uint4 &raw, uint4 &lo, uint4 &hi) {
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t w[4] = {raw.x ^ 0x80808080u, raw.y ^ 0x80808080u, raw.z ^ 0x80808080u, raw.w ^ 0x80808080u};
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = prmt(w[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140);
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), bias);
        f[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
    lo = make_uint4(f[0], f[1], f[2], f[3]);
    hi = make_uint4(f[4], f[5], f[6], f[7]);
}

W4_DEV void sts128(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
W4_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(CfgTc<DP, RT>::kThreads, 1) attn8_tc_kernel(const __grid_constant__ Attn8Params p) {
    using C = CfgTc<DP, RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tile = smem, *k_ring = q_tile + RT * C::kQTile, *v_ring = k_ring + C::kKStages * C::kTile,
            *raw_ring = v_ring + C::kVStages * C::kTile;
    CtlTc *ctl = reinterpret_cast<CtlTc *>(raw_ring + C::kRawStages * C::kRaw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&ctl->raw_full[i], 1);
            mbar_init(&ctl->raw_empty[i], 4);
        }
        for (int i = 0; i < 3; ++i) {
            if (i < 2) {
                mbar_init(&ctl->k_full[i], 4);
                mbar_init(&ctl->k_empty[i], RT);
            }
            mbar_init(&ctl->v_full[i], 4);
            mbar_init(&ctl->v_empty[i], RT);
        }
        for (int r = 0; r < RT; ++r) {
            mbar_init(&ctl->q_full[r], 4);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl->s_full[r][i], 1);
                mbar_init(&ctl->p_full[r][i], 4);
            }
            mbar_init(&ctl->o_done[r], 1);
            mbar_init(&ctl->o_last[r], 1);
            mbar_init(&ctl->o_free[r], 4);
            mbar_init(&ctl->drained[r], 1);
        }
        ctl->abort = 0;
        ctl->begun = 0;
        fence_mbar_init();
    }
    // TMEM is asked for when the kernel before is through with its own, and the next kernel may
    // start only when it has been had here: neither can hold what the other waits for.
    griddep_wait();
    if (warp == C::kMmaWarp) tmem_alloc(&ctl->tmem_base, C::kTmem);

    // The line: steps before each item by a scan of the CTA, in rounds; the item of the part's first step.
    const int64_t items = (int64_t)p.B * p.tiles;
    auto scan = [&](int64_t carry, int64_t i, int64_t &before, int64_t &total) {
        const int64_t own = i < items ? (int64_t)p.Hkv * item_of<kTcRows * RT>(p, i).nb : 0;
        int64_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        __syncthreads();  // the sums of the round before are read
        if (lane == 31) ctl->sums[warp] = sum;
        __syncthreads();
        before = carry + sum - own;
        total = carry;
        for (int w = 0; w < C::kThreads / 32; ++w) {
            if (w < warp) before += ctl->sums[w];
            total += ctl->sums[w];
        }
        return own;
    };
    int64_t W = 0, before = 0, own = 0;
    for (int64_t i0 = 0; i0 < items; i0 += C::kThreads) {
        own = scan(W, i0 + tid, before, W);
        if (blockIdx.x == 0 && i0 + tid < items) p.first[i0 + tid] = before;
    }
    if (blockIdx.x == 0 && tid == 0) p.first[items] = W;
    const int64_t share = share_of(p, W), begin = min(W, share * blockIdx.x), end = min(W, begin + share);
    if (items <= C::kThreads) {
        if (begin >= before && begin < before + own) ctl->item = tid, ctl->base = before;
    } else {
        int64_t sum = 0;
        for (int64_t i0 = 0; i0 < items; i0 += C::kThreads) {
            own = scan(sum, i0 + tid, before, sum);
            if (begin >= before && begin < before + own) ctl->item = (int)(i0 + tid), ctl->base = before;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = ctl->tmem_base;
    int *abort = &ctl->abort;
    SegTc *my = &ctl->seg[warp];
    if (lane == 0) {
        my->at = begin;
        my->end = end;
        my->item = begin < end ? ctl->item : 0;
        my->base = begin < end ? ctl->base : 0;
    }
    const volatile SegTc &seg = *my;

    if (warp == C::kLoadWarp) {
        // ---------------- producer: the whole warp walks, one lane issues; lane n has block n of a step
        const uint32_t lead = elect_lead();
        const int page_mask = (1 << p.page_shift) - 1;
        const uint32_t ring = smem_u32(raw_ring);
        int stage = 0, round = 0, step = 0;
        bool ok = true;
        while (ok && next_segment<RT>(p, my, lane)) {
            const int32_t *row = p.table + (int64_t)seg.b * p.width;
            const int64_t per_head = 1 << (p.page_shift - kKvBlockLog);
            const int nt = seg.nt, h = seg.h;
            auto page_of = [&](int j) {
                const int key = lane < kTcBlocks && j < nt ? key_of(seg, j, lane) : -1;
                const int id = key >= 0 ? __ldg(row + (key >> p.page_shift)) : -1;
                return id >= 0 && id < p.pages ? id : -1;
            };
            auto scales_of = [&](int j, int page) {
                if (page < 0) return 256 | 256 << 16;
                const int64_t s = ((int64_t)page * p.Hkv + h) * per_head + ((key_of(seg, j, lane) & page_mask) >> kKvBlockLog);
                return (int)__ldg(p.ks + s) | (int)__ldg(p.vs + s) << 16;
            };
            // entries two steps ahead, scales one: neither load is waited for when it is made
            int now = page_of(0), next = page_of(1), sc = scales_of(0, now);
            for (int j = 0; j < nt; ++j) {
                const int sc_next = j + 1 < nt ? scales_of(j + 1, next) : 0;
                const int after = page_of(j + 2);
                if (round > 0) ok = wait_warp(&ctl->raw_empty[stage], (round - 1) & 1, abort, p.status);
                if (!ok) break;
                const int slot = step % kScaleSlots;
                const int kb = sc & 0xFFFF, vb = sc >> 16;
                const uint32_t nan = __ballot_sync(0xffffffffu, lane < kTcBlocks && (kb == 255 || vb == 255));
                const uint32_t none = __ballot_sync(0xffffffffu, lane < kTcBlocks && kb > 255);
                const int vtop = (int)__reduce_max_sync(0xffffffffu, lane < kTcBlocks && vb < 255 ? vb : 0);
                if (lane < kTcBlocks) {
                    reinterpret_cast<float *>(&ctl->k_scale[slot])[lane] = kb < 255 ? scale_of((uint32_t)kb) : 0.0f;
                    reinterpret_cast<int *>(&ctl->v_scale[slot])[lane] = vb < 255 ? vb : 0;
                    if (lane == 0) ctl->odd[slot] = (int)(nan | none << 4) | vtop << 8;
                }
                __syncwarp();
                // boxes whose first block has a page (the others of it are on the same page)
                const uint32_t have = __ballot_sync(0xffffffffu, now >= 0) & (p.box == 4 ? 1u : p.box == 2 ? 5u : 15u);
                if (lane == 0) mbar_arrive_expect_tx(&ctl->raw_full[stage], (uint32_t)(__popc(have) * p.box * 32 * DP));
                __syncwarp();
                const uint32_t bar = smem_u32(&ctl->raw_full[stage]), dst = ring + (uint32_t)(stage * C::kRaw);
#pragma unroll 1
                for (int n = 0; n < kTcBlocks; n += p.box) {
                    const int page = __shfl_sync(0xffffffffu, now, n);
                    if (page < 0) continue;
                    const int tok = key_of(seg, j, n) & page_mask;
                    const int c1 = p.tok_inner ? tok : h, c2 = p.tok_inner ? h : tok;
                    constexpr int kWide = DP < 128 ? DP : 128;
#pragma unroll
                    for (int c = 0; c < DP / kWide; ++c) {
                        const uint32_t to = dst + (uint32_t)(c * kTcKeys * 128 + n * 16 * kWide);
                        tma_load_4d_lead(to, &p.kmap, 128 * c, c1, c2, page, bar, lead);
                        tma_load_4d_lead(to + (uint32_t)(C::kRaw / 2), &p.vmap, 128 * c, c1, c2, page, bar, lead);
                    }
                }
                now = next;
                next = after;
                sc = sc_next;
                ++step;
                if (++stage == C::kRawStages) stage = 0, ++round;
            }
        }
        if (lane == 0) ctl->begun = round * C::kRawStages + stage;
    } else if (warp >= C::kMmaWarp) {
        // ---------------- MMA issuers, one for each row tile: the whole warp walks, one lane issues
        const int r = warp - C::kMmaWarp;
        const uint32_t lead = elect_lead();
        constexpr uint32_t id_s = idesc_f16(0u, kTcRows, kTcKeys);
        constexpr uint32_t id_o = idesc_f16(0u, kTcRows, DP) | (1u << 16);  // B (the values) with its N axis contiguous
        const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tile + r * C::kQTile)), k_desc = smem_desc_sw128(smem_u32(k_ring)),
                       v_desc = smem_desc_mn_sw128(smem_u32(v_ring), kTcKeys * 128);
        const uint32_t s_col = tmem + (uint32_t)(2 * r * kTcKeys), o_col = tmem + C::kOCol + (uint32_t)(r * DP);
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) { ok = ok && wait_warp(bar, parity, abort, p.status); };
        int ks = 0, kr = 0, vs = 0, vr = 0;  // the rings' stages and rounds
        int sj = 0, oj = 0, mine = 0;        // S and O products of this row tile so far; segments with rows in it
        while (ok && next_segment<RT>(p, my, lane)) {
            const int nt = seg.nt;
            const bool on = r < seg.tiles;
            auto issue_s = [&](int j) {
                wait(&ctl->k_full[ks], kr & 1);
                if (on) {
                    // it goes where P of two steps before stood, whose product must be through (at a
                    // segment's start it is known to be)
                    if (C::kKStages > 1 && j > 0 && sj >= 2) wait(&ctl->o_done[r], sj & 1);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t kd = desc_at(k_desc, (uint32_t)(ks * C::kTile));
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        umma_f16_lead(s_col + (uint32_t)((sj & 1) * kTcKeys), desc_at(q_desc, (k / 4) * (kTcRows * 128) + (k % 4) * 32),
                                      desc_at(kd, (k / 4) * (kTcKeys * 128) + (k % 4) * 32), id_s, k > 0 ? 1u : 0u, lead);
                    umma_commit_lead(&ctl->s_full[r][sj & 1], lead);
                    umma_commit_lead(&ctl->k_empty[ks], lead);
                    ++sj;
                } else if (ok && lane == 0) {
                    mbar_arrive(&ctl->k_empty[ks]);
                }
                if (++ks == C::kKStages) ks = 0, ++kr;
            };
            if (on) wait(&ctl->q_full[r], mine & 1);
            if (ok) issue_s(0);
            for (int j = 0; j < nt && ok; ++j) {
                if (C::kKStages > 1 && j + 1 < nt) issue_s(j + 1);
                wait(&ctl->v_full[vs], vr & 1);
                if (on) {
                    wait(&ctl->p_full[r][oj & 1], (oj >> 1) & 1);
                    // the first product of a segment writes over the O of the one before, which has been read
                    if (j == 0 && mine > 0) wait(&ctl->o_free[r], (mine - 1) & 1);
                    // No product but the last one is open when a segment ends, nor where S of the next step
                    // comes after this product (a barrier's parity tells a phase only from the next one)
                    if ((C::kKStages == 1 || j == nt - 1) && oj > 0) wait(&ctl->o_done[r], (oj - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = desc_at(v_desc, (uint32_t)(vs * C::kTile));
#pragma unroll
                    for (int k = 0; k < kTcKeys / 16; ++k)
                        umma_f16_ts_lead(o_col, s_col + (uint32_t)((oj & 1) * kTcKeys + 8 * k), desc_at(vd, k * 2048), id_o,
                                         (j > 0 || k > 0) ? 1u : 0u, lead);
                    umma_commit_lead(&ctl->o_done[r], lead);
                    if (j == nt - 1) umma_commit_lead(&ctl->o_last[r], lead);
                    umma_commit_lead(&ctl->v_empty[vs], lead);
                    ++oj;
                } else if (ok && lane == 0) {
                    mbar_arrive(&ctl->v_empty[vs]);
                }
                if (++vs == C::kVStages) vs = 0, ++vr;
                if (C::kKStages == 1 && j + 1 < nt && ok) issue_s(j + 1);
            }
            mine += on;
        }
        __syncwarp();
    } else if (warp >= C::kConvWarp) {
        // ---------------- converters
        const int t = tid - 32 * C::kConvWarp;
        const uint32_t raw = smem_u32(raw_ring), kt = smem_u32(k_ring), vt = smem_u32(v_ring);
        constexpr int kItems = kTcKeys * DP / 16;  // runs of 16 codes of a tile
        auto convert = [&](uint32_t from, uint32_t to) {
#pragma unroll
            for (int i0 = 0; i0 < kItems; i0 += 128) {
                const int i = i0 + t;
                const uint4 w = lds_u128(from + 16 * i);
                uint4 lo, hi;
                codes16(w, lo, hi);
                // (128 values of the head,) token, run
                constexpr int kRuns = DP < 128 ? DP / 16 : 8;
                const int row = i / kRuns % kTcKeys, c16 = i / (kRuns * kTcKeys) * 8 + i % kRuns;
                const uint32_t at = to + (uint32_t)((c16 >> 2) * (kTcKeys * 128) + row * 128);
                const int e = (c16 & 3) * 2, odd = (c16 >> 2) & 1;  // lanes of odd chunks begin with the second run: no two to a bank
                sts128(at + (uint32_t)(((e + odd) ^ (row & 7)) << 4), odd ? hi : lo);
                sts128(at + (uint32_t)(((e + 1 - odd) ^ (row & 7)) << 4), odd ? lo : hi);
            }
            fence_async_shared();
            __syncwarp();
        };
        int rs = 0, rr = 0, ks = 0, kr = 0, vs = 0, vr = 0;
        bool ok = true;
        while (ok && next_segment<RT>(p, my, lane)) {
            const int nt = seg.nt;
            for (int j = 0; j < nt; ++j) {
                ok = wait_warp(&ctl->raw_full[rs], rr & 1, abort, p.status);
                if (ok && kr > 0) ok = wait_warp(&ctl->k_empty[ks], (kr - 1) & 1, abort, p.status);
                if (!ok) break;
                convert(raw + (uint32_t)(rs * C::kRaw), kt + (uint32_t)(ks * C::kTile));
                if (lane == 0) mbar_arrive(&ctl->k_full[ks]);
                if (vr > 0) ok = wait_warp(&ctl->v_empty[vs], (vr - 1) & 1, abort, p.status);
                if (!ok) break;
                convert(raw + (uint32_t)(rs * C::kRaw + C::kRaw / 2), vt + (uint32_t)(vs * C::kTile));
                if (lane == 0) {
                    mbar_arrive(&ctl->v_full[vs]);
                    mbar_arrive(&ctl->raw_empty[rs]);
                }
                if (++rs == C::kRawStages) rs = 0, ++rr;
                if (++ks == C::kKStages) ks = 0, ++kr;
                if (++vs == C::kVStages) vs = 0, ++vr;
            }
        }
    } else {
        // ---------------- softmax: thread = row
        const int rt = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16, o_at = tmem + lane_off + C::kOCol + (uint32_t)(rt * DP);
        int sj = 0, step = 0, n_mine = 0;  // steps of this row tile, of all; segments of this row tile
        bool ok = true;
        while (ok && next_segment<RT>(p, my, lane)) {
            const int nt = seg.nt;
            if (rt >= seg.tiles) {
                step += nt;
                continue;
            }
            const int rows = seg.rows - rt * kTcRows;
            const bool active = 32 * quad < rows, mine = row < rows;
            const int inner0 = seg.inner0, inner1 = seg.inner1;
            // ---- the row's query, as f16 (all products that read the one before are through)
            float kq = p.scale_log2;
            {
                const int at_row = seg.row0 + rt * kTcRows + row, tok = (int)((unsigned)at_row / (unsigned)p.G);
                const uint16_t *src = static_cast<const uint16_t *>(p.q) + (seg.t0 + tok) * p.ld + (seg.h * (int64_t)p.G + (at_row - tok * p.G)) * p.D;
                uint4 w[DP / 8];  // (all of it asked for at once)
#pragma unroll
                for (int c = 0; c < DP / 8; ++c)
                    w[c] = mine && 8 * c < p.D ? __ldg(reinterpret_cast<const uint4 *>(src + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
                float f = 1.0f;
                if constexpr (BF) {
                    uint32_t top = 0u;
#pragma unroll
                    for (int c = 0; c < DP / 8; ++c) {
                        const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(max(top, u[e] & 0x7FFFu), (u[e] >> 16) & 0x7FFFu);
                    }
                    // times 2^k, which takes the largest exponent to 13 (tiny rows: as far as f32 goes)
                    const int k = min(140 - (int)(top >> 7), 126);
                    f = __uint_as_float((uint32_t)(127 + k) << 23);
                    kq *= __uint_as_float((uint32_t)(127 - k) << 23);
                }
                const uint32_t to = smem_u32(q_tile + rt * C::kQTile) + (uint32_t)(row * 128);
#pragma unroll
                for (int c = 0; c < DP / 8; ++c) {
                    if constexpr (BF) {
                        uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = pack_pair<__half>(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f);
                        w[c] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    sts128(to + (uint32_t)((c >> 3) * (kTcRows * 128) + (((c & 7) ^ (row & 7)) << 4)), w[c]);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->q_full[rt]);
            }
            float mx = -INFINITY, l = 0.0f;  // the maximum that P is relative to (log2 units), the sum times 2^kLift
            float far = 1.0f;                // by which the scores were scaled down (kFarScore)
            float eref = 0.0f;               // scale byte that the row's weights are relative to: the largest that it saw
            for (int j = 0; j < nt; ++j, ++step) {
                // A step's scales are read when its S has come, whose count is the tile's own: warps that skipped
                // segments may be far ahead of the producer, where a barrier of the scales' own would not tell a
                // phase from one two before it.  The producer writes them before its copies, which the converters
                // wait for, and for those the product.
                ok = wait_warp(&ctl->s_full[rt][sj & 1], (sj >> 1) & 1, abort, p.status);
                if (!ok) break;
                tc_fence_after();
                const float4 ks4 = ctl->k_scale[step % kScaleSlots];
                const int4 vs4 = ctl->v_scale[step % kScaleSlots];
                const int odd = ctl->odd[step % kScaleSlots];
                // (not 0: -infinity must stay what it is)
                float kf[4] = {fmaxf(kq * ks4.x, 0x1p-126f), fmaxf(kq * ks4.y, 0x1p-126f), fmaxf(kq * ks4.z, 0x1p-126f), fmaxf(kq * ks4.w, 0x1p-126f)};
                const float vs[4] = {(float)vs4.x, (float)vs4.y, (float)vs4.z, (float)vs4.w};
                float vtop = (float)(odd >> 8);  // of the blocks that the row sees
                const uint32_t s_at = tmem + lane_off + (uint32_t)((2 * rt + (sj & 1)) * kTcKeys);
                if (active) {
                    uint32_t sr[kTcKeys];
                    tmem_ld64(s_at, sr);
                    if ((odd & 255) || j < inner0 || j >= inner1) {
                        uint64_t see = 0ull;
                        vtop = 0.0f;
                        const int pos = mine ? seg.ctx + (int)((unsigned)(seg.row0 + rt * kTcRows + row) / (unsigned)p.G) : -1, len = seg.len;
#pragma unroll
                        for (int n = 0; n < kTcBlocks; ++n) {
                            const int key0 = key_of(seg, j, n);
                            uint32_t bits = 0u;
                            if (key0 >= 0 && !(odd >> (4 + n) & 1)) {
                                // keys up to the row's own, from the window's first on or among the first tokens
                                bits = below(min(pos + 1, len) - key0);
                                if (p.window > 0) bits &= ~below(pos - p.window + 1 - key0) | below(p.sinks - key0);
                                if (bits) vtop = fmaxf(vtop, vs[n]);
                                if (bits && (odd >> n & 1)) l = __uint_as_float(0x7FC00000u);  // and so is the row's output
                            }
                            see |= (uint64_t)bits << (16 * n);
                        }
#pragma unroll
                        for (int c = 0; c < kTcKeys; ++c)
                            if (!((see >> c) & 1)) sr[c] = 0xFF800000u;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < kTcBlocks; ++n) {
                        const uint32_t *x = sr + 16 * n;
                        float m0 = max3(x[0], x[1], x[2]), m1 = max3(x[3], x[4], x[5]);
                        m0 = max3(__float_as_uint(m0), x[6], x[7]);
                        m1 = max3(__float_as_uint(m1), x[8], x[9]);
                        m0 = max3(__float_as_uint(m0), x[10], x[11]);
                        m1 = max3(__float_as_uint(m1), x[12], x[13]);
                        m0 = max3(__float_as_uint(m0), x[14], x[15]);
                        top = fmaxf(top, fmaxf(m0, m1) * kf[n]);
                    }
                    vtop = fmaxf(vtop, eref);
                    const bool up = mine && top > fmaxf(mx + kGrow8, -kFarScore);  // also the first finite one: mx is -inf
                    if (__any_sync(0xffffffffu, up || vtop > eref)) {
                        const float f = up ? ex2(mx - top) : 1.0f, fo = f * ex2(eref - vtop);
                        l *= f;
                        if (j > 0) {
                            // every product so far is through, then O is moved
                            ok = wait_warp(&ctl->o_done[rt], (sj - 1) & 1, abort, p.status);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DP / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(o_at + 32 * c, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
                                tmem_st32(o_at + 32 * c, o);
                            }
                        }
                        eref = vtop;
                        if (up) {
                            mx = top;
                            if (top > kFarScore && top < INFINITY) {
                                const float down = far_scale(top);
                                mx *= down;
                                kq *= down;
                                far *= down;
#pragma unroll
                                for (int n = 0; n < kTcBlocks; ++n) kf[n] = fmaxf(kf[n] * down, 0x1p-126f);  // (not 0, as above)
                            }
                        }
                    }
                    // The weights come with their block's scale (in the exponent), and the sum takes it out
                    // of a block at a time; a scale 2^60 below the largest leaves nothing of a weight in f16
                    // as it is.
                    const float minus = mx == -INFINITY ? kLift : kLift - mx;
#pragma unroll
                    for (int n = 0; n < kTcBlocks; ++n) {
                        const float lift = fmaxf(vs[n] - eref, -60.0f), off = minus + lift;
                        const uint64_t kf2 = f32x2(kf[n], kf[n]), off2 = f32x2(off, off);
                        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                        for (int c = 16 * n; c < 16 * n + 16; c += 2) {
                            float a, e;
                            f32x2_split(f32x2_fma(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), kf2, off2), a, e);
                            a = ex2(a);
                            e = ex2(e);
                            sum2[(c / 2) & 1] = f32x2_add(sum2[(c / 2) & 1], f32x2(a, e));
                            sr[c / 2] = pack_pair<__half>(a, e);
                        }
                        float sa, sb;
                        f32x2_split(f32x2_add(sum2[0], sum2[1]), sa, sb);
                        l = fmaf(sa + sb, ex2(-lift), l);
                    }
                    tmem_st32(s_at, sr);
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[rt][sj & 1]);
                ++sj;
            }
            if (!ok) break;
            // ---------------- the segment's result
            ok = wait_warp(&ctl->o_last[rt], n_mine & 1, abort, p.status);
            if (!ok) break;
            ++n_mine;
            if (active) {
                tc_fence_after();
                const bool whole = seg.whole != 0;
                const float unit = scale_of((uint32_t)eref), inv = !whole ? 0x1p-7f : l == 0.0f ? 0.0f : 1.0f / l;
                // parts: [CTA][2][DP / 4][rows][4], so that 32 rows write 512 bytes in one piece
                constexpr int kRows = kTcRows * RT;
                const int64_t part = (int64_t)blockIdx.x * 2 + seg.slot;
                const int unit_row = rt * kTcRows + row;
                if (!whole && mine) p.part_ml[part * kRows + unit_row] = make_float2(mx / far, l * 0x1p-7f);
                using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
                const int at_row = seg.row0 + rt * kTcRows + row, tok = (int)((unsigned)at_row / (unsigned)p.G);
                uint16_t *to = static_cast<uint16_t *>(p.out) + ((seg.t0 + tok) * p.Hq + seg.h * (int64_t)p.G + (at_row - tok * p.G)) * p.D;
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_at + c, o);
                    if (!mine) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * unit * inv);
                    if (!whole) {
                        float4 *d = reinterpret_cast<float4 *>(p.part_o) + (part * (DP / 4) + c / 4) * kRows + unit_row;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[i * kRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                                       __uint_as_float(o[4 * i + 3]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 8 * i < p.D) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack_pair<TO>(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
                                *reinterpret_cast<uint4 *>(to + c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->o_free[rt]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(*reinterpret_cast<volatile int *>(abort), 0)) {  // of all threads alike
        if (warp == C::kLoadWarp && lane == 0) drain_ring(ctl->raw_full, C::kRawStages, ctl->begun);
        if (warp >= C::kMmaWarp) drain_products(&ctl->drained[warp - C::kMmaWarp]);
        __syncthreads();
    }
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Joins the parts of units that were cut: a thread a row and 32 of its values.
template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(128) attn8_tc_join_kernel(const __grid_constant__ Attn8Params p) {
    constexpr int kRows = kTcRows * RT;
    griddep_wait();
    const int c0 = (int)blockIdx.x, row = (int)blockIdx.y * 32 + ((int)threadIdx.x & 31), col = ((int)blockIdx.z * 4 + ((int)threadIdx.x >> 5)) * 32;
    if (col >= p.D) return;
    const Cut cut = cut_of(p, c0, (int)threadIdx.x & 31);
    if (!cut.is) return;
    const Item it = item_of<kRows>(p, cut.item);
    if (row >= it.rows) return;
    float top = -INFINITY, z = 0.0f, sum[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[i] = 0.0f;
#pragma unroll 1
    for (int c = c0; c <= cut.c1; ++c) {
        const int64_t part = 2 * (int64_t)c + (c > c0 ? 0 : 1);
        const float4 *src = reinterpret_cast<const float4 *>(p.part_o) + (part * (DP / 4) + col / 4) * kRows + row;
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __ldcs(src + i * kRows);
        const float2 x = p.part_ml[part * kRows + row];
        const float now = fmaxf(top, x.x);
        const float f0 = now == -INFINITY ? 1.0f : ex2(top - now), f = now == -INFINITY ? 1.0f : ex2(x.x - now);
        top = now;
        z = fmaf(x.y, f, z * f0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum[4 * i] = fmaf(v[i].x, f, sum[4 * i] * f0);
            sum[4 * i + 1] = fmaf(v[i].y, f, sum[4 * i + 1] * f0);
            sum[4 * i + 2] = fmaf(v[i].z, f, sum[4 * i + 2] * f0);
            sum[4 * i + 3] = fmaf(v[i].w, f, sum[4 * i + 3] * f0);
        }
    }
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    const int at_row = it.row0 + row, tok = (int)((unsigned)at_row / (unsigned)p.G);
    uint16_t *to = static_cast<uint16_t *>(p.out) + ((it.r.t0 + tok) * p.Hq + cut.head * (int64_t)p.G + (at_row - tok * p.G)) * p.D + col;
    using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (col + i < p.D)
            *reinterpret_cast<uint4 *>(to + i) =
                make_uint4(pack_pair<TO>(sum[i] * inv, sum[i + 1] * inv), pack_pair<TO>(sum[i + 2] * inv, sum[i + 3] * inv),
                           pack_pair<TO>(sum[i + 4] * inv, sum[i + 5] * inv), pack_pair<TO>(sum[i + 6] * inv, sum[i + 7] * inv));
}

template <int DP, int RT, bool BF>
cudaError_t tc_launch(const Attn8Params &p, const Plan8Tc &c, cudaStream_t st) {
    using C = CfgTc<DP, RT>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)attn8_tc_kernel<DP, RT, BF>, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.ctas, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t k = cudaLaunchKernelEx(&cfg, attn8_tc_kernel<DP, RT, BF>, p);
    if (k != cudaSuccess || c.ctas == 1) return k;
    cfg.gridDim = dim3((unsigned)(c.ctas - 1), kTcRows * RT / 32, (DP + 127) / 128);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn8_tc_join_kernel<DP, RT, BF>, p);
}

template <bool BF>
cudaError_t tc_launch_type(const Attn8Params &p, const Plan8Tc &c, cudaStream_t st) {
    if (c.dp == 64) return c.rt == 2 ? tc_launch<64, 2, BF>(p, c, st) : tc_launch<64, 1, BF>(p, c, st);
    if (c.dp == 128) return c.rt == 2 ? tc_launch<128, 2, BF>(p, c, st) : tc_launch<128, 1, BF>(p, c, st);
    return tc_launch<256, 1, BF>(p, c, st);
}

constexpr int kTcLeast = 2;  // steps of a CTA

}  // namespace

Plan8Tc attn8_tc_plan(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len, int64_t max_new,
                      int64_t window, int64_t sinks) {
    Plan8Tc c;
    const int64_t rows = max_new * (q_heads / kv_heads);
    c.dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    c.rt = rows > kTcRows && c.dp <= 128 ? 2 : 1;
    c.tiles = (int)ceil_div(rows, kTcRows * c.rt);
    c.items = B * c.tiles;
    int64_t blocks = ceil_div(max_len, kKvBlock);
    if (window > 0) blocks = std::min(blocks, ceil_div(window + kTcRows * c.rt, kKvBlock) + 1 + ceil_div(sinks, kKvBlock));
    const int64_t steps = c.items * kv_heads * ceil_div(blocks, kTcBlocks);
    c.ctas = (int)std::min<int64_t>(152, std::max<int64_t>(1, steps / kTcLeast));
    c.bytes = (size_t)c.ctas * 2 * kTcRows * c.rt * (c.dp + 2) * 4 + (size_t)(c.items + 2) / 2 * 16;
    return c;
}

cudaError_t launch_attn8_tc(Attn8Params p, const Plan8Tc &c, bool bf16, cudaStream_t st) {
    p.step = kTcBlocks;
    p.least = kTcLeast;
    p.cluster = 1;
    return bf16 ? tc_launch_type<true>(p, c, st) : tc_launch_type<false>(p, c, st);
}

}  // namespace w4
