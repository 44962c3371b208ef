// tree_attn.cu -- attention of drafted token trees over a paged cache (tcgen05).
//
// A unit of work is (request, key head, row tiles): its rows are (drafted
// token, query head of the key head's group), 128 at most to a row tile.  It
// is worked in steps of 64 keys, and the steps of all units, in one line, are
// dealt out evenly: persistent CTA c of G takes steps W c / G to W (c + 1) / G,
// whatever the lengths, found from them on the device.  A unit that lies in one
// CTA's part is finished there; the parts of one that was cut are joined by a
// second kernel.  The roles of a CTA, each walking its segments on its own, so
// that one unit's end lies under the next one's loads and first products:
//   softmax warps  four to a row tile, one thread a row: S to registers, the
//                  mask where the step reaches the drafted tokens, the running
//                  maximum and sum, P in 16 bits back over S; at a segment's
//                  end O from TMEM to memory;
//   TMA producers  the query tiles, and the key and the value tiles (their
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
// P is rounded to the cache's type, which the tensor cores want of both
// operands; l sums the unrounded values.  In f16, P and l carry a factor 2^7 that
// cancels too: P then reaches 2^15, and what f16 loses of a small weight is at most 2^-32
// of the largest (without it 2^-25: a tail of 128k such keys beside one dominant key lost 0.4 %).
// Measured with the join (bf16, 32 requests, 32 query and 8 key heads of 128, up to
// 8,192 keys each): one token 133 us, 6.1 TB/s of keys and values; 64 tokens, two row
// tiles, 194 us, 4.3 TB/s and 0.84 PFLOP/s.  The latter takes 267 us with one row tile
// to a CTA, 222 with units dealt out whole, 206 with a join of a block a row.
// A step of two row tiles takes about 1,850 cycles (5.1 TB/s); the rest is the
// first copies, the write of O at a unit's end and the join.  None of memory (3.7 TB/s), tensor
// pipe (44 %) and issue (33 %) is full over the kernel at 8 requests (a step's own chain of
// product, softmax and product is the likely wait; not measured).  One row tile spills 25 of the 128 registers that
// two CTAs an SM leave.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "smem_limit.h"
#include "tcgen05.cuh"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kRows = 128;  // rows of a tile (TMEM lanes)
constexpr int kKeys = 64;   // keys of a tile
constexpr float kGrow = 8.0f;  // log2 by which a maximum may grow before O is rescaled
constexpr float kLiftF16 = 7.0f;  // log2 of the factor of P in f16: 2^(8 + 7) is below f16's largest value
// Barriers for the edge steps in turn: more than an MMA warp that is behind can be passed by
// (the other row tile gets no further than the ring of keys, at most 8 stages, lets it).
constexpr int kClean = 16;
constexpr int kMinSteps = 2;   // of a CTA, if there are as many: a part costs its write and its join

struct AttnParams {
    CUtensorMap qmap;  // [T][Hq][D], box {64, G, tokens of a tile}
    CUtensorMap kmap, vmap;  // pages, then tokens and heads in the order of their strides, D; a box: 64 values, min(page, 64) tokens
    const int32_t *table, *ctx_len, *cu_new;
    const uint4 *mask;
    const uint16_t *v;  // for the exact treatment of NaN and infinities in drafted values
    uint16_t *out;
    float *part_o;   // [CTA][2][row tile of the CTA][DP / 4][128 rows][4]
    float2 *part_ml; // [CTA][2][row tile of the CTA][128 rows]: maximum (log2), sum
    int64_t *first;  // [B + 1]: first step of each request, and their number
    uint32_t *status;
    int64_t width, T, pages, page_stride, token_stride, head_stride;
    int B, Hq, Hkv, G, D;
    int page_shift;
    int tok_inner;  // the token stride is the smaller one
    int tpt;     // drafted tokens of a row tile
    int max_new;
    int ctas;
    float scale_log2;
};

struct Ctl {
    uint64_t q_full, q_empty;
    uint64_t full[2][8], empty[2][8];  // [keys, values][stage]
    uint64_t s_full[2][2], p_full[2][2], o_done[2];  // [row tile][S buffer]
    uint64_t o_last[2], o_free[2];  // a segment's last product; its O has been read
    uint64_t v_clean[kClean];  // the values of an edge step have been gone over (edge steps in turn)
    uint32_t tmem_base;
    int abort;
    int bad;  // a drafted value that is not finite has been met
    int first_b;
    int64_t first_at, sums[16];
    uint64_t drained[2];  // [row tile], after an abort: its products are through
    int begun[2], queries;  // fills of the rings, copies of query tiles
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

template <bool BF>
W4_DEV uint32_t drop_nonfinite(uint32_t w) {
    constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
    return ((w & e) == e ? 0u : w & 0xFFFFu) | (((w >> 16) & e) == e ? 0u : w & 0xFFFF0000u);
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

// Requests in steps: b's units are (key head, group of row tiles), each of nt steps.
struct Steps {
    Request rq;
    int drafted, groups, nt;
    int64_t all;
};
template <int RT>
W4_DEV Steps steps_of(const AttnParams &p, int b) {
    Steps s;
    s.rq = request_of(p, b);
    s.drafted = min(s.rq.n, p.max_new);
    const int rows = RT * p.tpt;
    s.groups = (s.drafted + rows - 1) / rows;
    s.nt = (s.rq.len + kKeys - 1) / kKeys;
    s.all = (int64_t)p.Hkv * s.groups * s.nt;
    return s;
}

// CTAs that share W steps: each has some (the launch knows only a bound of W).
W4_DEV int ctas_of(const AttnParams &p, int64_t W) { return (int)min((int64_t)p.ctas, max((int64_t)1, W / kMinSteps)); }

// A CTA's part of the steps, segment by segment (a segment lies in one unit).
template <int RT>
struct Walk {
    const AttnParams &p;
    int64_t at, end, base;  // the next step, the part's end, the request's first step
    int b;
    Steps st;
    // the segment
    int h, k0, nt;       // key head, first key, steps
    int tok0, tiles;     // its first drafted token, row tiles with rows
    bool whole;          // all of the unit
    int slot;            // of its part, if not: 0 where the unit began in an earlier CTA, 1 where it ends in a later one

    W4_DEV Walk(const AttnParams &p_, int64_t begin, int64_t end_, int b_, int64_t base_)
        : p(p_), at(begin), end(end_), base(base_), b(b_) {
        if (at < end) st = steps_of<RT>(p, b);
    }
    W4_DEV bool next() {
        if (at >= end) return false;
        while (at >= base + st.all) {  // (there are steps left, so there is a request with some)
            base += st.all;
            st = steps_of<RT>(p, ++b);
        }
        const int64_t off = at - base;
        const int unit = (int)(off / st.nt), k = (int)(off - (int64_t)unit * st.nt);
        h = unit / st.groups;
        tok0 = (unit - h * st.groups) * RT * p.tpt;
        tiles = RT == 1 || tok0 + p.tpt >= st.drafted ? 1 : 2;
        nt = (int)min((int64_t)(st.nt - k), end - at);
        k0 = k * kKeys;
        whole = nt == st.nt;
        slot = k > 0 ? 0 : 1;
        at += nt;
        return true;
    }
    W4_DEV int k_end() const { return min(st.rq.len, k0 + nt * kKeys); }
    // Step j reaches the drafted tokens or the end; such steps are a segment's last.
    W4_DEV bool edge(int j) const { return k0 + (j + 1) * kKeys > st.rq.ctx; }
    W4_DEV int edges() const { return nt - min(max((st.rq.ctx - k0) / kKeys, 0), nt); }
};

template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(Cfg<DP, RT>::kThreads, Cfg<DP, RT>::kCtas)
tree_attn_kernel(const __grid_constant__ AttnParams p) {
    using C = Cfg<DP, RT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tile = smem;
    uint8_t *k_ring = smem + RT * C::kQTile, *v_ring = k_ring + C::kKStages * C::kTile;
    Ctl *ctl = reinterpret_cast<Ctl *>(v_ring + C::kVStages * C::kTile);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    griddep_launch_dependents();
    if (tid == 0) {
        mbar_init(&ctl->q_full, 1);
        mbar_init(&ctl->q_empty, RT);
        for (int i = 0; i < 2; ++i)
            for (int s = 0; s < 8; ++s) {
                mbar_init(&ctl->full[i][s], 1);
                mbar_init(&ctl->empty[i][s], RT);  // each row tile's products release a stage
            }
        for (int r = 0; r < RT; ++r) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl->s_full[r][i], 1);
                mbar_init(&ctl->p_full[r][i], 4);
            }
            mbar_init(&ctl->o_done[r], 1);
            mbar_init(&ctl->o_last[r], 1);
            mbar_init(&ctl->o_free[r], 4);
            mbar_init(&ctl->drained[r], 1);
        }
        for (int i = 0; i < kClean; ++i) mbar_init(&ctl->v_clean[i], 4 * RT);
        ctl->abort = 0;
        ctl->bad = 0;
        ctl->first_b = 0;
        ctl->first_at = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(&ctl->tmem_base, C::kTmem);

    // All steps before each request, by a scan of the block over the requests: their number W
    // first (more requests than threads: in rounds), then the request of the part's first step.
    constexpr int kWarps = C::kThreads / 32;
    auto scan = [&](int64_t carry, int b, int64_t &before, int64_t &total) {
        const int64_t own = b < p.B ? steps_of<RT>(p, b).all : 0;
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += ctl->sums[w];
            total += ctl->sums[w];
        }
        return own;
    };
    int64_t before = 0, W = 0, own = 0;
    for (int b0 = 0; b0 < p.B; b0 += C::kThreads) {
        own = scan(W, b0 + tid, before, W);
        if (blockIdx.x == 0 && b0 + tid < p.B) p.first[b0 + tid] = before;
    }
    if (blockIdx.x == 0 && tid == 0) p.first[p.B] = W;
    const int G = ctas_of(p, W);
    const int64_t begin = min(W, W * blockIdx.x / G), end = min(W, W * (blockIdx.x + 1) / G);
    if (p.B <= C::kThreads) {
        if (begin >= before && begin < before + own) ctl->first_b = tid, ctl->first_at = before;
    } else {
        int64_t sum = 0;
        for (int b0 = 0; b0 < p.B; b0 += C::kThreads) {
            own = scan(sum, b0 + tid, before, sum);
            if (begin >= before && begin < before + own) ctl->first_b = b0 + tid, ctl->first_at = before;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    int *abort = &ctl->abort;
    Walk<RT> seg(p, begin, end, ctl->first_b, ctl->first_at);

    if (warp == C::kLoadWarp || warp == C::kLoadWarp + 1) {
        // ---------------- TMA producers, one for the keys (and the queries) and one for the values (issuing a
        // tile's boxes takes about half of the tile's time): the whole warp walks, one lane issues
        const bool keys = warp == C::kLoadWarp;
        const uint32_t lead = elect_lead();
        const int page_rows = min(1 << p.page_shift, kKeys), page_log = min(p.page_shift, 6);  // rows of a box
        const int pages = kKeys >> page_log;                                                   // of a tile
        const CUtensorMap *map = keys ? &p.kmap : &p.vmap;
        uint64_t *full = ctl->full[keys ? 0 : 1], *empty = ctl->empty[keys ? 0 : 1];
        const uint32_t ring = smem_u32(keys ? k_ring : v_ring);
        const int stages = keys ? C::kKStages : C::kVStages;
        int stage = 0, round = 0, n_seg = 0;
        bool ok = true;
        for (; ok && seg.next(); ++n_seg) {
            if (keys) {
                // the queries, once the products of the segment before are through with theirs
                if (n_seg > 0) ok = wait_warp(&ctl->q_empty, (n_seg - 1) & 1, abort, p.status);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ctl->q_full, (uint32_t)(seg.tiles * C::kChunks * p.G * p.tpt * 128));
                    for (int r = 0; r < seg.tiles; ++r)
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_3d(q_tile + r * C::kQTile + c * (kRows * 128), &p.qmap, 64 * c, seg.h * p.G,
                                        (int)(seg.st.rq.t0 + seg.tok0 + r * p.tpt), &ctl->q_full);
                }
                __syncwarp();
            }
            // lane i: the block-table entry of box i of step j, -1 where there is none; read two
            // steps ahead and looked at only when it is used, or each step would wait for it
            const int32_t *row = p.table + (int64_t)seg.b * p.width;
            const int k0 = seg.k0, nt = seg.nt, len = seg.st.rq.len;
            auto entry_of = [&](int j) {
                const int key = k0 + j * kKeys + lane * page_rows;
                return lane < pages && j < nt && key < len ? __ldg(row + (key >> p.page_shift)) : -1;
            };
            int now = entry_of(0), next = entry_of(1);
            for (int j = 0; j < nt; ++j) {
                if (round > 0) ok = wait_warp(&empty[stage], (round - 1) & 1, abort, p.status);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::kTile);
                __syncwarp();
                // no page: the page count, which is out of the map and read as zeros
                const int id = now < 0 || now >= p.pages ? (int)p.pages : now;
                now = next;
                next = entry_of(j + 2);
                const uint32_t dst = ring + (uint32_t)(stage * C::kTile), bar = smem_u32(&full[stage]);
                // a page of 64 or more: the tile's place in it; else its boxes are whole pages
                const int off = (k0 + j * kKeys) & ((1 << p.page_shift) - 1);
                const int c1 = p.tok_inner ? off : seg.h, c2 = p.tok_inner ? seg.h : off;
                for (int i = 0; i < pages; ++i) {
                    const int page = __shfl_sync(0xffffffffu, id, i);
#pragma unroll
                    for (int ch = 0; ch < C::kChunks; ++ch)
                        tma_load_4d_lead(dst + (uint32_t)(ch * (kKeys * 128) + ((i << page_log) * 128)), map, 64 * ch, c1, c2,
                                         page, bar, lead);
                }
                if (++stage == stages) stage = 0, ++round;
            }
        }
        if (lane == 0) {
            ctl->begun[keys ? 0 : 1] = round * stages + stage;
            if (keys) ctl->queries = n_seg;
        }
    } else if (warp >= C::kMmaWarp) {
        // ---------------- MMA issuers, one for each row tile: the whole warp walks, one lane issues
        const int r = warp - C::kMmaWarp;
        const uint32_t lead = elect_lead();
        constexpr uint32_t fmt = BF ? 1u : 0u;
        constexpr uint32_t id_s = idesc_f16(fmt, kRows, kKeys);
        constexpr uint32_t id_o = idesc_f16(fmt, kRows, DP) | (1u << 16);  // B (the values) with its N axis contiguous
        const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tile + r * C::kQTile)), k_desc = smem_desc_sw128(smem_u32(k_ring)),
                       v_desc = smem_desc_mn_sw128(smem_u32(v_ring), kKeys * 128);
        const uint32_t s_col = tmem + (uint32_t)(2 * r * kKeys), o_col = tmem + C::kOCol + (uint32_t)(r * DP);
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) { ok = ok && wait_warp(bar, parity, abort, p.status); };
        int ks = 0, kr = 0, vs = 0, vr = 0;  // the rings' stages and rounds
        int sj = 0, oj = 0;                  // S and O products of this row tile so far
        int edges = 0, mine = 0;             // edge steps of all segments; segments with rows in this tile
        for (int n_seg = 0; ok && seg.next(); ++n_seg) {
            const int nt = seg.nt;
            const bool on = r < seg.tiles;
            auto issue_s = [&](int j) {
                wait(&ctl->full[0][ks], kr & 1);
                if (on) {
                    // it goes where P of two steps before stood, whose product must be through (at a
                    // segment's start it is known to be)
                    if (j > 0 && sj >= 2) wait(&ctl->o_done[r], sj & 1);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t kd = desc_at(k_desc, (uint32_t)(ks * C::kTile));
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        umma_f16_lead(s_col + (uint32_t)((sj & 1) * kKeys), desc_at(q_desc, (k / 4) * (kRows * 128) + (k % 4) * 32),
                                      desc_at(kd, (k / 4) * (kKeys * 128) + (k % 4) * 32), id_s, k > 0 ? 1u : 0u, lead);
                    umma_commit_lead(&ctl->s_full[r][sj & 1], lead);
                    umma_commit_lead(&ctl->empty[0][ks], lead);
                    if (j == nt - 1) umma_commit_lead(&ctl->q_empty, lead);
                    ++sj;
                } else if (ok && lane == 0) {
                    mbar_arrive(&ctl->empty[0][ks]);
                    if (j == nt - 1) mbar_arrive(&ctl->q_empty);
                }
                if (++ks == C::kKStages) ks = 0, ++kr;
            };
            wait(&ctl->q_full, n_seg & 1);
            if (ok) issue_s(0);
            for (int j = 0; j < nt && ok; ++j) {
                if (j + 1 < nt) issue_s(j + 1);
                wait(&ctl->full[1][vs], vr & 1);
                if (seg.edge(j)) {
                    if (on) wait(&ctl->v_clean[edges % kClean], (edges / kClean) & 1);
                    ++edges;
                }
                if (on) {
                    wait(&ctl->p_full[r][oj & 1], (oj >> 1) & 1);
                    // the first product of a segment writes over the O of the one before, which has been read
                    if (j == 0 && mine > 0) wait(&ctl->o_free[r], (mine - 1) & 1);
                    // No product but the last one is open when a segment ends (a barrier's parity
                    // tells a phase only from the next one)
                    if (j == nt - 1 && oj > 0) wait(&ctl->o_done[r], (oj - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = desc_at(v_desc, (uint32_t)(vs * C::kTile));
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        umma_f16_ts_lead(o_col, s_col + (uint32_t)((oj & 1) * kKeys + 8 * k), desc_at(vd, k * 2048), id_o,
                                         (j > 0 || k > 0) ? 1u : 0u, lead);
                    umma_commit_lead(&ctl->o_done[r], lead);
                    if (j == nt - 1) umma_commit_lead(&ctl->o_last[r], lead);
                    umma_commit_lead(&ctl->empty[1][vs], lead);
                    ++oj;
                } else if (ok && lane == 0) {
                    mbar_arrive(&ctl->empty[1][vs]);
                }
                if (++vs == C::kVStages) vs = 0, ++vr;
            }
            mine += on;
        }
        __syncwarp();
    } else {
        // ---------------- softmax: thread = row
        const int rt = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
        const int tok = row / p.G, g = row - tok * p.G;
        const uint32_t lane_off = (uint32_t)(32 * quad) << 16, o_at = tmem + lane_off + C::kOCol + (uint32_t)(rt * DP);
        int sj = 0, vj = 0, edges = 0, n_mine = 0;  // steps of this row tile, of all; edge steps; segments of this row tile
        bool ok = true;
        while (ok && seg.next()) {
            const Request &rq = seg.st.rq;
            const int nt = seg.nt;
            const bool on = rt < seg.tiles;
            const int tok0 = seg.tok0 + rt * p.tpt;
            const int rows = min(p.tpt, seg.st.drafted - tok0) * p.G;
            const bool active = on && 32 * quad < rows;  // of the warp
            const bool mine = on && row < rows;
            const int64_t t = rq.t0 + tok0 + tok;
            // the row's mask over its request's drafted tokens, later bits cleared (read where it
            // is needed: the few steps that reach them)
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
            if (!on) {
                vj += nt;
                edges += seg.edges();
                continue;
            }
            float mx = -INFINITY, l = 0.0f;  // the maximum that P is relative to (log2 units), the sum
            for (int j = 0; j < nt; ++j) {
                const int key0 = seg.k0 + j * kKeys;
                const bool edge = seg.edge(j);
                ok = wait_warp(&ctl->s_full[rt][sj & 1], (sj >> 1) & 1, abort, p.status);
                if (!ok) break;
                tc_fence_after();
                if (edge) {
                    // Values that no row may see become zeros (P is zero there, but 0 * NaN is
                    // not); drafted values that are not finite too, and are added at the end.
                    // The softmax warps of the row tiles with rows share the work, and where there
                    // is one such tile of two, its warps arrive for the other's too.
                    const int s = (vj + j) % C::kVStages;
                    ok = wait_warp(&ctl->full[1][s], ((vj + j) / C::kVStages) & 1, abort, p.status);
                    if (!ok) break;
                    uint8_t *vt = v_ring + s * C::kTile;
                    bool bad = false;
                    for (int i = tid; i < C::kChunks * kKeys * 8; i += 128 * seg.tiles) {
                        const int key = key0 + ((i >> 3) & (kKeys - 1));
                        uint4 *at = reinterpret_cast<uint4 *>(vt + i * 16);
                        if (key >= rq.len) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else if (key >= rq.ctx) {
                            uint4 w = *at;
                            if (any_nonfinite<BF>(w.x) || any_nonfinite<BF>(w.y) || any_nonfinite<BF>(w.z) ||
                                any_nonfinite<BF>(w.w)) {
                                bad = true;
                                w.x = drop_nonfinite<BF>(w.x);
                                w.y = drop_nonfinite<BF>(w.y);
                                w.z = drop_nonfinite<BF>(w.z);
                                w.w = drop_nonfinite<BF>(w.w);
                                *at = w;
                            }
                        }
                    }
                    if (bad) ctl->bad = 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&ctl->v_clean[edges % kClean]);
                        if (seg.tiles < RT) mbar_arrive(&ctl->v_clean[edges % kClean]);
                    }
                    ++edges;
                }
                const uint32_t s_at = tmem + lane_off + (uint32_t)((2 * rt + (sj & 1)) * kKeys);
                if (active) {
                    uint32_t sr[kKeys];
                    tmem_ld64(s_at, sr);
                    if (edge) {
                        // which of the step's 64 keys this row sees
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
                    float part[4];  // four chains
#pragma unroll
                    for (int c = 0; c < 4; ++c) part[c] = fmaxf(__uint_as_float(sr[c]), __uint_as_float(sr[c + 4]));
#pragma unroll
                    for (int c = 8; c < kKeys; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            part[i] = fmaxf(part[i], fmaxf(__uint_as_float(sr[c + i]), __uint_as_float(sr[c + i + 4])));
                    const float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                    // scale > 0: the maximum scales along
                    const float now = fmaxf(mx, top * p.scale_log2);
                    const bool grow = mine && now > mx + kGrow;  // true for the first finite maximum: mx is -inf
                    if (__any_sync(0xffffffffu, grow)) {
                        if (j > 0) {
                            // every product so far is through, then O *= 2^(old - new)
                            ok = wait_warp(&ctl->o_done[rt], (sj - 1) & 1, abort, p.status);
                            if (!ok) break;
                            tc_fence_after();
                            const float f = now == -INFINITY ? 1.0f : exp2_fast(mx - now);
                            l *= f;
#pragma unroll 1
                            for (int c = 0; c < DP / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(o_at + 32 * c, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st32(o_at + 32 * c, o);
                            }
                        }
                        mx = now;
                    }
                    const float base = mx == -INFINITY ? 0.0f : mx;
                    const float off = BF ? -base : kLiftF16 - base;
                    const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2), base2 = f32x2(off, off);
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
                    tmem_st32(s_at, sr);
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[rt][sj & 1]);
                ++sj;
            }
            vj += nt;
            if (!ok) break;
            // ---------------- the segment's result (and the word on `bad`: the last product waited
            // for v_clean, before which it was written)
            ok = wait_warp(&ctl->o_last[rt], n_mine & 1, abort, p.status);
            if (!ok) break;
            ++n_mine;
            if (active) {
                tc_fence_after();
                const bool bad = *reinterpret_cast<volatile int *>(&ctl->bad) != 0;
                const float inv = !seg.whole ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
                const int64_t part = ((int64_t)blockIdx.x * 2 + seg.slot) * RT + rt;
                if (!seg.whole) p.part_ml[part * kRows + row] = make_float2(mx, l);
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_at + c, o);
                    if (!mine) continue;
                    // a row that sees nothing: O is a sum of zeros, P having been zero throughout
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                    if (bad) {
                        uint64_t mlo, mhi;
                        row_mask(mlo, mhi);
                        for (int jd = max(0, seg.k0 - rq.ctx); jd < seg.k_end() - rq.ctx; ++jd) {
                            if (!((jd < 64 ? mlo >> jd : mhi >> (jd - 64)) & 1)) continue;
                            const int key = rq.ctx + jd;
                            const int64_t id = __ldg(p.table + (int64_t)seg.b * p.width + (key >> p.page_shift));
                            if (id < 0 || id >= p.pages) continue;
                            const uint16_t *vr = p.v + id * p.page_stride + seg.h * p.head_stride +
                                                 (int64_t)(key & ((1 << p.page_shift) - 1)) * p.token_stride;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float x = c + i < p.D ? to_f32<BF>(vr[c + i]) : 0.0f;
                                if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                            }
                        }
                    }
                    if (!seg.whole) {
                        // four values of 32 rows to a store: 512 bytes in one piece
                        float4 *d = reinterpret_cast<float4 *>(p.part_o) + (part * (DP / 4) + c / 4) * kRows + row;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[i * kRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    } else {
                        uint16_t *d = p.out + (t * p.Hq + seg.h * p.G + g) * (int64_t)p.D + c;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 8 * i < p.D) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack2<BF>(__uint_as_float(o[8 * i + 2 * e]), __uint_as_float(o[8 * i + 2 * e + 1]));
                                *reinterpret_cast<uint4 *>(d + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
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
        if (warp == C::kLoadWarp && lane == 0) {
            drain_ring(ctl->full[0], C::kKStages, ctl->begun[0]);
            drain_ring(ctl->full[1], C::kVStages, ctl->begun[1]);
            drain_ring(&ctl->q_full, 1, ctl->queries);
        }
        if (warp >= C::kMmaWarp) drain_products(&ctl->drained[warp - C::kMmaWarp]);
        __syncthreads();
    }
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// The join of the parts of a unit that was cut, for each of its rows:
// out = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c over the CTAs c that share it.

// The CTAs that share the unit of request b, key head h and row tile mt.
struct Parts {
    int c0, c1, rt, rts;
    W4_DEV int64_t of(int c) const { return ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * rts + rt; }
};
template <int RT>
W4_DEV Parts parts_of(const AttnParams &p, const Steps &st, int b, int h, int mt) {
    Parts u;
    const int64_t W = p.first[p.B], from = p.first[b] + (int64_t)(h * st.groups + mt / RT) * st.nt;
    // CTA c has steps W c / G to W (c + 1) / G: those of the unit's first and last step
    const int G = ctas_of(p, W);
    u.c0 = (int)(((from + 1) * G - 1) / W);
    u.c1 = (int)(((from + st.nt) * G - 1) / W);
    u.rt = mt % RT;
    u.rts = RT;
    return u;
}

// Many rows: a thread a row and `cols` columns (the parts lie row
// beside row), two such column groups to a block.
template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(256) tree_attn_join_tiles_kernel(const __grid_constant__ AttnParams p, int mtiles, int cols) {
    const int row = threadIdx.x & (kRows - 1);
    int u = blockIdx.x;
    const int mt = u % mtiles;
    u /= mtiles;
    const int h = u % p.Hkv, b = u / p.Hkv;
    const Steps st = steps_of<RT>(p, b);  // the caller's arrays: no part of the kernel before
    const int tok = row / p.G, i = mt * p.tpt + tok, g = row - tok * p.G;
    griddep_wait();
    if (mt * p.tpt >= st.drafted) return;
    const Parts pt = parts_of<RT>(p, st, b, h, mt);
    if (pt.c0 == pt.c1 || tok >= p.tpt || i >= st.drafted) return;

    float m = -INFINITY;
#pragma unroll 4
    for (int c = pt.c0; c <= pt.c1; ++c) m = fmaxf(m, p.part_ml[pt.of(c) * kRows + row].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
#pragma unroll 4
    for (int c = pt.c0; c <= pt.c1; ++c) {
        const float2 ml = p.part_ml[pt.of(c) * kRows + row];
        l += exp2_fast(ml.x - base) * ml.y;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint16_t *d = p.out + ((st.rq.t0 + i) * p.Hq + h * p.G + g) * (int64_t)p.D;
    const int from = (blockIdx.y * 2 + (threadIdx.x >> 7)) * cols, to = min(from + cols, p.D);
    for (int at = from; at < to; at += 16) {  // 16 columns at a time (or the last 8), for loads in flight
        const bool two = at + 8 < to;
        float acc[16] = {};
#pragma unroll 2
        for (int c = pt.c0; c <= pt.c1; ++c) {
            const float4 *o = reinterpret_cast<const float4 *>(p.part_o) + (pt.of(c) * (DP / 4) + at / 4) * kRows + row;
            float4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = e < 2 || two ? __ldcs(o + e * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
            // a part that the row sees nothing of has weight 0 and O = 0
            const float w = exp2_fast(p.part_ml[pt.of(c) * kRows + row].x - base);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[4 * e] = fmaf(w, v[e].x, acc[4 * e]);
                acc[4 * e + 1] = fmaf(w, v[e].y, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(w, v[e].z, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(w, v[e].w, acc[4 * e + 3]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (e == 1 && !two) break;
            const float *x = acc + 8 * e;
            *reinterpret_cast<uint4 *>(d + at + 8 * e) =
                make_uint4(pack2<BF>(x[0] * inv, x[1] * inv), pack2<BF>(x[2] * inv, x[3] * inv),
                           pack2<BF>(x[4] * inv, x[5] * inv), pack2<BF>(x[6] * inv, x[7] * inv));
        }
    }
}

// Few rows: 8 warps (one block) a row, which take its parts in turn; a lane has
// four values of each 128.
template <int DP, int RT, bool BF>
__global__ void __launch_bounds__(256) tree_attn_join_rows_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kVecs = (DP + 127) / 128, kPer = 8;
    __shared__ float4 sums[kPer][32 * kVecs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hq = blockIdx.y, b = blockIdx.x / p.max_new, i = blockIdx.x % p.max_new;
    const Steps st = steps_of<RT>(p, b);
    const int h = hq / p.G, g = hq - h * p.G;
    const int mt = i / p.tpt, row = (i - mt * p.tpt) * p.G + g;
    griddep_wait();
    if (i >= st.drafted) return;
    const Parts pt = parts_of<RT>(p, st, b, h, mt);
    if (pt.c0 == pt.c1) return;
    auto ml_of = [&](int c) { return c <= pt.c1 ? p.part_ml[pt.of(c) * kRows + row] : make_float2(-INFINITY, 0.0f); };

    float2 ml = ml_of(pt.c0 + lane);
    float m = ml.x, l = 0.0f;
    for (int c = pt.c0 + 32 + lane; c <= pt.c1; c += 32) m = fmaxf(m, ml_of(c).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.0f : m;
    float4 acc[kVecs] = {};
    for (int cb = pt.c0; cb <= pt.c1; cb += 32) {
        if (cb > pt.c0) ml = ml_of(cb + lane);
        const float w = exp2_fast(ml.x - base);
        l += w * ml.y;
        const int n = min(32, pt.c1 - cb + 1);
#pragma unroll 4
        for (int k = warp; k < n; k += kPer) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float4 *o = reinterpret_cast<const float4 *>(p.part_o) + pt.of(cb + k) * (DP / 4) * kRows + row;
#pragma unroll
            for (int e = 0; e < kVecs; ++e) {
                const int d4 = 32 * e + lane;
                if (d4 * 4 < p.D) {
                    const float4 v = o[d4 * kRows];
                    acc[e].x = fmaf(wk, v.x, acc[e].x);
                    acc[e].y = fmaf(wk, v.y, acc[e].y);
                    acc[e].z = fmaf(wk, v.z, acc[e].z);
                    acc[e].w = fmaf(wk, v.w, acc[e].w);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int e = 0; e < kVecs; ++e) sums[warp][32 * e + lane] = acc[e];
    __syncthreads();
    if (warp > 0) return;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint16_t *d = p.out + ((st.rq.t0 + i) * p.Hq + hq) * (int64_t)p.D;
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
        for (int k = 1; k < kPer; ++k) {
            const float4 v = sums[k][32 * e + lane];
            acc[e].x += v.x;
            acc[e].y += v.y;
            acc[e].z += v.z;
            acc[e].w += v.w;
        }
        const int at = 4 * (32 * e + lane);
        if (at < p.D)
            *reinterpret_cast<uint2 *>(d + at) =
                make_uint2(pack2<BF>(acc[e].x * inv, acc[e].y * inv), pack2<BF>(acc[e].z * inv, acc[e].w * inv));
    }
}

struct Shape {
    int rt, tpt, ctas;
    int64_t o_floats, ml;  // of the workspace, in float and float2
};

int dp_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Even row tiles; two of them to a CTA where there are two; a CTA for every
// place on the machine (152 SMs; with one row tile two places, one token of 32 requests
// of 8,192 keys 133 us, in one place 148), fewer where not even kMinSteps are left for each.
Shape shape_of(int64_t B, int G, int Hkv, int D, int64_t max_len, int max_new) {
    Shape s;
    const int most = (int)ceil_div(max_new, kRows / G);
    s.tpt = (int)ceil_div(max_new, most);
    const int mtiles = (int)ceil_div(max_new, s.tpt);
    s.rt = mtiles > 1 && D <= 128 ? 2 : 1;
    const int64_t steps = B * Hkv * ceil_div(mtiles, s.rt) * ceil_div(max_len, kKeys);
    s.ctas = (int)std::min<int64_t>(D <= 128 && s.rt == 1 ? 304 : 152, ceil_div(steps, kMinSteps));
    s.ml = (int64_t)s.ctas * 2 * s.rt * kRows;
    s.o_floats = s.ml * dp_of(D);
    return s;
}

template <int DP, int RT, bool BF>
cudaError_t launch_attn(const AttnParams &p, cudaStream_t st) {
    using C = Cfg<DP, RT>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void *>(tree_attn_kernel<DP, RT, BF>), C::kSmem);
    if (e != cudaSuccess) return e;
    tree_attn_kernel<DP, RT, BF><<<p.ctas, C::kThreads, C::kSmem, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // a block a row while a row has about an eighth of an SM (152 of them): 32 requests of
    // one token, 1,024 rows, 132.9 us (138.4 with a thread a row); 4 of 16, 2,048 rows, 27.3
    // (26.7); 32 of 4, 4,096 rows, 140.6 (139.6); 8 of 24, 6,144 rows, 46.9 (36.5)
    if ((int64_t)p.B * p.max_new * p.Hq <= 152 * 16) {
        cfg.gridDim = dim3((unsigned)(p.B * p.max_new), (unsigned)p.Hq);
        return cudaLaunchKernelEx(&cfg, tree_attn_join_rows_kernel<DP, RT, BF>, p);
    }
    // the widest columns that leave three blocks an SM (152), in us with 8 / 16 / 32 of D = 128:
    // 64 tiles 36.5 / 38.7 / 42.8, 128 27.8 / 26.3 / 30.9, 512 200 / 195 / 192
    const int mtiles = (int)ceil_div(p.max_new, p.tpt);
    const int64_t tiles = (int64_t)p.B * p.Hkv * mtiles;
    const auto blocks = [&](int c) { return tiles * ceil_div(p.D, 2 * c); };
    const int cols = blocks(32) >= 3 * 152 ? 32 : blocks(16) >= 3 * 152 ? 16 : 8;
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)ceil_div(p.D, 2 * cols));
    return cudaLaunchKernelEx(&cfg, tree_attn_join_tiles_kernel<DP, RT, BF>, p, mtiles, cols);
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
    const Shape s = shape_of(B, q_heads / kv_heads, kv_heads, D, max_len, max_new);
    return (size_t)s.o_floats * 4 + (size_t)s.ml * 8 + (size_t)(B + 1) * 8;
}

cudaError_t launch_tree_attention(const void *q, int64_t ld, const w4_paged_cache &c, const int32_t *table,
                                  int64_t width, const int32_t *ctx_len, const int32_t *cu_new, const uint32_t *mask,
                                  int64_t B, int64_t T, int32_t q_heads, float scale, int64_t max_len, int32_t max_new,
                                  void *out, void *workspace, uint32_t *status, cudaStream_t st) {
    AttnParams p = {};
    const int G = q_heads / c.heads, D = c.head_dim;
    const Shape s = shape_of(B, G, c.heads, D, max_len, max_new);
    if (B * max_new > 0x7FFFFFFF || B * c.heads * max_new > 0x7FFFFFFF || q_heads > 65535) return cudaErrorInvalidConfiguration;
    p.table = table; p.ctx_len = ctx_len; p.cu_new = cu_new; p.mask = reinterpret_cast<const uint4 *>(mask);
    p.v = static_cast<const uint16_t *>(c.v);
    p.out = static_cast<uint16_t *>(out);
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.part_o + s.o_floats);
    p.first = reinterpret_cast<int64_t *>(p.part_ml + s.ml);
    p.status = status;
    p.width = width; p.T = T; p.pages = c.pages;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.B = (int)B; p.Hq = q_heads; p.Hkv = c.heads; p.G = G; p.D = D;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.tpt = s.tpt; p.ctas = s.ctas;
    p.max_new = max_new;
    p.scale_log2 = scale * kLog2e;
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
