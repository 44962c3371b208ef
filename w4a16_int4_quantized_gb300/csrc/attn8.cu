// attn8.cu -- causal attention over a paged cache held in 8 bits, whole or through a sliding
// window beside a few first tokens.
//
// Rows are (new token, query head of the key head's group), 16 to a tile and one or two tiles
// to a warp.  A unit of work is (request, tiles, key head) and consists of blocks of 16 keys.
// Either a cluster of CTAs shares a unit's blocks and joins what it found in shared memory; or
// the blocks of all units, in one line, are dealt out evenly, so many to a CTA, found from the
// lengths on the device, and a second kernel joins the parts of units that were cut.
// The warps of a CTA share the rows and take its blocks in turn, each with its own running
// maximum, sum and O.  A warp does not wait for others before a unit's end: it has a ring of its own in
// shared memory, which TMA fills a turn of two blocks ahead (one box for the 16 keys of a block
// and head, one for the values, in whatever order the cache has tokens and heads).
// Bound by memory where there are few rows: 64 requests of one token over up to 16,384 keys (32
// query and 8 key heads of 128, bf16) take 260 us, 6.2 TB/s; by cp.async, 16 bytes a lane, the copies
// alone took 318.  Where work is short, by its beginning and end (about 8 us: offsets, block table,
// first copies, the joins): 1,000 keys of one request 8.2 us.  With 17 to 32 rows by issue, 8 warps an SM:
// 32 requests of 32 rows over 8k keys 138 us.
//
// Operands without shuffles: which value of a head stands at which place of an operand is free
// as long as both factors agree.  For S = Q K^T a lane's quad index q takes values 64 i + 16 q
// .. + 15 of a key (a run of 16 bytes), for O = P V its group index g takes values g D/8 .. of the
// four keys whose weights S left in that lane.
// Codes become f16 exactly, by one byte permutation for two: u = code + 128 (the top bit
// flipped) under a byte of zeros is the f16 number u 2^-24.  The 128 is taken out of the sums:
// those of S begin with -128 times the query's sum, those of O have a column that multiplies
// the weights by 128.  Scales are powers of two, one for a block of 16 keys: the keys' multiplies
// the scores, the values' the weights, relative to the largest one that the row has met so far (a
// weight is then rounded to f16 with a factor 2^7: what it loses is at most 2^-32 of the largest).
// Queries in bf16 go to f16 with a power of two of their row, so that the largest lies in
// [2^13, 2^14): what a value loses is at most half of f16's least step, 2^-25, and so 2^-38 of the largest.
// O is rescaled only when a row's maximum has grown by more than 2^8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn8.cuh"
#include "common.cuh"
#include "smem_limit.h"
#include "tcgen05.cuh"

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kMinBlocks = 4 * kWarps;  // of a CTA, if there are as many: a part costs its write and its join
// What the second kernel and the scan cost, in blocks of a CTA: clusters / line, in us, 64 requests of 1,000
// keys 37 / 43 and of 2,000 57 / 58, 128 of 1,500 74 / 81, 32 of 4,000 68 / 51, 2 of 8,000 21 / 24, 1 of
// 20,000 35 / 30 (one token each, 32 query and 8 key heads of 128).
constexpr int kJoinBlocks = 80;
constexpr int kStages = 4;
constexpr int kMostCluster = 8;
constexpr int kFewRows = 32;  // of a request and key head; more go to the kernel of attn8_tc.cu

W4_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two biased codes (bytes `sel` of w) times 2^-24, as f16.
W4_DEV uint32_t codes_f16(uint32_t w, uint32_t sel) { return prmt(w, 0u, sel); }
constexpr uint32_t kBiasF16 = 0x00800080u;  // 128 * 2^-24, twice

W4_DEV float sum_f16(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return f.x + f.y;
}

// What a CTA works on: blocks b0 .. b1 - 1 of a unit.
struct Segment {
    int64_t t0, slot;  // slot: of its part, if it is not the whole unit
    int b, row0, all_rows, rows, pos0, pos1, ctx, len, head, b0, b1;
    int sink, skip;  // block i of the unit is block i, from `sink` on block i + skip
    bool whole;
};

// DP: head_dim rounded up to 64; MT: tiles of 16 rows.
template <int DP, int MT>
struct Cfg8 {
    static constexpr int kChunks = DP / 64;  // 16-byte runs of a key in a lane
    static constexpr int kSteps = DP / 16;   // of S along the head
    static constexpr int kVRun = DP / 8;     // bytes of a value in a lane
    static constexpr int kStage = 32 * DP;   // bytes of a block of a warp: 16 keys, then 16 values
    static constexpr int kRows = 16 * MT;
    static constexpr bool kQRegs = DP * MT <= 64;  // Q stays in registers, else in shared memory
    static constexpr int kBlocks = DP == 256 ? 1 : 2;  // of a warp's turn: their products and exponentials overlap
    static constexpr int kSlots = kStages / kBlocks;   // turns in the ring
    static constexpr int kPitch = DP < 128 ? 64 : 128, kBox = 16 * kPitch, kBoxes = DP / kPitch;  // of 16 tokens, swizzled over its pitch
    // 16-byte run `c` of a row of a box
    static W4_DEV uint32_t at(int row, int c) {
        return (uint32_t)(row * kPitch + ((kPitch == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4));
    }
    static constexpr int kQBytes = kQRegs ? 0 : MT * kSteps * 32 * 16;
    static constexpr int kSmem = kWarps * kStages * kStage + kQBytes;
    static constexpr int kCtas = DP * MT <= 128 ? 3 : DP <= 128 ? 2 : 1;  // an SM
    static_assert(kStages * kStage >= kRows * DP * 4, "a warp's O takes the place of its ring at the end");
};

template <int DP, int MT, bool BF>
__global__ void __launch_bounds__(32 * kWarps, Cfg8<DP, MT>::kCtas) attn8_kernel(const __grid_constant__ Attn8Params p) {
    using C = Cfg8<DP, MT>;
    extern __shared__ __align__(1024) uint8_t smem8[];
    __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
    __shared__ int64_t s_sum[kWarps], s_base;
    __shared__ int s_item;
    __shared__ Segment s_seg;
    __shared__ uint64_t s_full[kWarps][C::kSlots];
    __shared__ int s_failed;
    __shared__ float2 s_ml[C::kRows];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, qd = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < C::kSlots; ++i) mbar_init(&s_full[warp][i], 1);
        if (tid == 0) s_failed = 0;
        fence_mbar_init();
    }
    __syncwarp();
    const uint32_t lead = elect_lead();
    int turns = 0;  // of the warp, so far
    griddep_wait();

    // ---- the CTA's part of the line of blocks
    int64_t at, end, base;  // the next block, the part's end, the item's first block
    int64_t item;
    bool idle = false;
    if (p.ctas == 0) {  // a unit
        // (later tiles see more keys: they go first)
        const unsigned unit = blockIdx.x / (unsigned)p.cluster;
        item = unit / (unsigned)p.Hkv;
        item = item / p.tiles * p.tiles + (p.tiles - 1 - item % p.tiles);
        const int64_t nb = item_of<C::kRows>(p, item).nb, rank = blockIdx.x - unit * (unsigned)p.cluster;
        if (nb == 0) return;
        base = 0;
        at = (int64_t)(unit % (unsigned)p.Hkv) * nb;
        end = at + nb * (rank + 1) / p.cluster;
        at += nb * rank / p.cluster;
        idle = at == end;  // nothing to do, but for the join
        if (idle) end = at + 1;
    } else {
        // blocks before each item by a scan of the CTA, in rounds; the item of the part's first block
        const int64_t items = (int64_t)p.B * p.tiles;
        auto scan = [&](int64_t carry, int64_t i, int64_t &before, int64_t &total) {
            const int64_t own = i < items ? (int64_t)p.Hkv * item_of<C::kRows>(p, i).nb : 0;
            int64_t sum = own;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            __syncthreads();  // the sums of the round before are read
            if (lane == 31) s_sum[warp] = sum;
            __syncthreads();
            before = carry + sum - own;
            total = carry;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s_sum[w];
                total += s_sum[w];
            }
            return own;
        };
        int64_t W = 0, before = 0, own = 0;
        for (int64_t i0 = 0; i0 < items; i0 += 32 * kWarps) {
            own = scan(W, i0 + tid, before, W);
            if (blockIdx.x == 0 && i0 + tid < items) p.first[i0 + tid] = before;
        }
        if (blockIdx.x == 0 && tid == 0) p.first[items] = W;
        const int64_t share = share_of(p, W);
        at = share * blockIdx.x;
        end = min(W, at + share);
        if (at >= end) return;
        if (items <= 32 * kWarps) {
            if (at >= before && at < before + own) s_item = tid, s_base = before;
        } else {
            int64_t sum = 0;
            for (int64_t i0 = 0; i0 < items; i0 += 32 * kWarps) {
                own = scan(sum, i0 + tid, before, sum);
                if (at >= before && at < before + own) s_item = (int)(i0 + tid), s_base = before;
            }
        }
        __syncthreads();
        item = s_item;
        base = s_base;
    }

#pragma unroll 1
    while (at < end) {
    {
        // The unit: found by all, kept in shared memory (it would cost the loop its registers)
        Item it = item_of<C::kRows>(p, item);
        while (at >= base + (int64_t)p.Hkv * it.nb) {  // (there are blocks left, so there is an item with some)
            base += (int64_t)p.Hkv * it.nb;
            it = item_of<C::kRows>(p, ++item);
        }
        const int head = (int)((at - base) / (int64_t)it.nb), b0 = (int)(at - base - (int64_t)head * it.nb);
        const int b1 = (int)min((int64_t)it.nb, b0 + (end - at));
        at += b1 - b0;
        if (tid == 0) {
            s_seg.t0 = it.r.t0; s_seg.row0 = it.row0; s_seg.all_rows = it.all_rows; s_seg.b = it.b;
            s_seg.rows = it.rows; s_seg.pos0 = it.pos0; s_seg.pos1 = it.pos1; s_seg.ctx = it.r.ctx; s_seg.len = it.r.len;
            s_seg.head = head; s_seg.b0 = b0; s_seg.b1 = it.span.blocks() > 0 && !idle ? b1 : b0;
            s_seg.sink = it.span.sink; s_seg.skip = it.span.first - it.span.sink;
            s_seg.whole = p.cluster == 1 && b1 - b0 == it.nb;
            s_seg.slot = 2 * (int64_t)blockIdx.x + (b0 > 0 ? 0 : 1);
        }
        __syncthreads();
    }
    const volatile Segment &seg = s_seg;

    // ---- the warp's blocks: b0 + warp, then every fourth
    const int b0 = seg.b0 + warp, n_mine = seg.b1 > b0 ? (seg.b1 - b0 + kWarps - 1) / kWarps : 0;
    const int head = seg.head, sink = seg.sink, skip = seg.skip, pos0 = seg.pos0, pos1 = seg.pos1, len = seg.len;
    auto key_of = [&](int j) {
        const int i = b0 + kWarps * j;
        return (i < sink ? i : i + skip) << kKvBlockLog;
    };
    const int32_t *row_of = p.table + (int64_t)seg.b * p.width;
    const int page_mask = (1 << p.page_shift) - 1;
    const int64_t scale_head = (int64_t)head << (p.page_shift - kKvBlockLog);
    // lane i: the page and the scales of the warp's block j + i (-1: no such page)
    auto fetch = [&](int j, int &page, uint32_t &scales) {
        page = -1;
        scales = 0u;
        if (j + lane < n_mine) {
            const int key = key_of(j + lane);
            page = __ldg(row_of + (key >> p.page_shift));
            if (page >= p.pages) page = -1;
            if (page >= 0) {
                const int64_t s = page * ((int64_t)p.Hkv << (p.page_shift - kKvBlockLog)) + scale_head + ((key & page_mask) >> kKvBlockLog);
                scales = (uint32_t)__ldg(p.ks + s) | (uint32_t)__ldg(p.vs + s) << 8;
            }
        }
    };
    const uint32_t ring = smem_u32(smem8) + (uint32_t)(warp * kStages * C::kStage);
    constexpr int NB = C::kBlocks, NT = 2 * NB;
    // Turn i of the unit, blocks NB i and on: the whole warp calls, one lane issues
    const int n_turns = (n_mine + NB - 1) / NB;
    auto copy = [&](int i, int pages_now, int pages_next, int upto) {  // pages_now: of blocks before upto
        int page[NB], have = 0;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int j = (NB * i + n) & 31;
            const int a = __shfl_sync(0xffffffffu, pages_now, j), c = __shfl_sync(0xffffffffu, pages_next, j);
            page[n] = NB * i + n >= n_mine ? -1 : NB * i + n >= upto ? c : a;
            have += page[n] >= 0;
        }
        const int slot = (turns + i) % C::kSlots;
        if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][slot], (uint32_t)(have * C::kStage));
        __syncwarp();  // (what the slot held has been read by all lanes)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (page[n] < 0) continue;
            const int tok = key_of(NB * i + n) & page_mask;
            const int c1 = p.tok_inner ? tok : head, c2 = p.tok_inner ? head : tok;
            const uint32_t dst = ring + (uint32_t)((slot * NB + n) * C::kStage), bar = smem_u32(&s_full[warp][slot]);
#pragma unroll
            for (int c = 0; c < C::kBoxes; ++c) {
                tma_load_4d_lead(dst + (uint32_t)(c * C::kBox), &p.kmap, 128 * c, c1, c2, page[n], bar, lead);
                tma_load_4d_lead(dst + (uint32_t)((C::kBoxes + c) * C::kBox), &p.vmap, 128 * c, c1, c2, page[n], bar, lead);
            }
        }
    };

    float o[MT][DP / 8 + 1][4];  // the last column: 128 times the weights
    float mref[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int c = 0; c <= DP / 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[m][c][e] = 0.0f;
        mref[m][0] = mref[m][1] = -INFINITY;
        l[m][0] = l[m][1] = 0.0f;
    }
    float eref[MT][2];  // scale byte that a row's weights are relative to: the largest that it saw
#pragma unroll
    for (int m = 0; m < MT; ++m) eref[m][0] = eref[m][1] = 0.0f;
    float far[MT][2];  // by which a row's scores were scaled down (kFarScore)
#pragma unroll
    for (int m = 0; m < MT; ++m) far[m][0] = far[m][1] = 1.0f;

    // Lane i of now and next: blocks i of the warp's present 32 and of the next
    int page_now, page_next;
    uint32_t sc_now, sc_next;
    fetch(0, page_now, sc_now);
#pragma unroll
    for (int i = 0; i < C::kSlots - 1; ++i)
        if (i < n_turns) copy(i, page_now, page_now, 32);
    fetch(32, page_next, sc_next);

    // ---- queries: rows g and g + 8 of each tile, as operands
    int pos[MT][2];
    float kq[MT][2];  // from products times 2^24 to log2 units, without the keys' scale
    float bias[MT][2];  // what the sums begin with
    uint32_t qa[C::kQRegs ? MT * C::kSteps : 1][4];
    uint8_t *q_smem = smem8 + kWarps * kStages * C::kStage;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint2 raw[2][C::kSteps];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = seg.row0 + 16 * m + 8 * h + g;
            const bool on = row < seg.all_rows;
            const int tok = (int)((unsigned)row / (unsigned)p.G);
            pos[m][h] = on ? seg.ctx + tok : -1;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (seg.t0 + tok) * p.ld + (seg.head * (int64_t)p.G + (row - tok * p.G)) * p.D;
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                const int d = 64 * (s >> 2) + 16 * qd + 4 * (s & 3);
                raw[h][s] = on && d < p.D ? __ldg(reinterpret_cast<const uint2 *>(src + d)) : make_uint2(0u, 0u);
            }
            kq[m][h] = p.scale_log2;
            if constexpr (BF) {
                uint32_t top = 0u;
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
                    top = max(max(top, max(raw[h][s].x & 0x7FFFu, (raw[h][s].x >> 16) & 0x7FFFu)),
                              max(raw[h][s].y & 0x7FFFu, (raw[h][s].y >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // times 2^k, which takes the largest exponent to 13 (tiny rows: as far as f32 goes)
                const int k = min(140 - (int)(top >> 7), 126);
                const float f = __uint_as_float((uint32_t)(127 + k) << 23);
                kq[m][h] *= __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s) {
                    uint2 &w = raw[h][s];
                    w.x = pack_pair<__half>(__uint_as_float(w.x << 16) * f, __uint_as_float(w.x & 0xFFFF0000u) * f);
                    w.y = pack_pair<__half>(__uint_as_float(w.y << 16) * f, __uint_as_float(w.y & 0xFFFF0000u) * f);
                }
            }
            float sum = 0.0f;
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) sum += sum_f16(raw[h][s].x) + sum_f16(raw[h][s].y);
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            bias[m][h] = sum * -0x1p-17f;  // -128 * 2^-24
        }
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
            if constexpr (C::kQRegs) {
                qa[m * C::kSteps + s][0] = raw[0][s].x;
                qa[m * C::kSteps + s][1] = raw[1][s].x;
                qa[m * C::kSteps + s][2] = raw[0][s].y;
                qa[m * C::kSteps + s][3] = raw[1][s].y;
            } else if (warp == 0) {
                reinterpret_cast<uint4 *>(q_smem)[(m * C::kSteps + s) * 32 + lane] =
                    make_uint4(raw[0][s].x, raw[1][s].x, raw[0][s].y, raw[1][s].y);
            }
        }
    }
    if constexpr (!C::kQRegs) __syncthreads();

    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n_turns; ++i) {
        const int j = NB * i, ji = j & 31;
        if (j > 0 && ji == 0) {
            page_now = page_next;
            sc_now = sc_next;
            fetch(j + 32, page_next, sc_next);
        }
        // into the place of the turn before
        if (i + C::kSlots - 1 < n_turns) copy(i + C::kSlots - 1, page_now, page_next, (j | 31) + 1);
        int page[NB];
        uint32_t sc[NB];
        bool any = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            page[n] = __shfl_sync(0xffffffffu, page_now, ji + n);
            sc[n] = __shfl_sync(0xffffffffu, sc_now, ji + n);
            any |= page[n] >= 0;
        }
        const int slot = (turns + i) % C::kSlots;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][slot], (uint32_t)((turns + i) / C::kSlots) & 1u));
        if (!ok) break;
        if (!any) continue;  // keys of a page outside the cache are not seen
        uint32_t src[NB];
        int key0[NB];
        bool edge[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            src[n] = ring + (uint32_t)((slot * NB + n) * C::kStage);
            key0[n] = key_of(j + n);
            const int last = key0[n] + kKvBlock - 1;
            edge[n] = page[n] < 0 || last > pos0 || last >= len || (p.window > 0 && key0[n] <= pos1 - p.window && last >= p.sinks);
        }

        // S: tile t of NT is keys of block t >> 1
        float s[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][t][e] = bias[m][e >> 1];
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i) {
            uint32_t w[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = 8 * (t & 1) + g;
                const uint4 v = lds_u128(src[t >> 1] + (uint32_t)((64 * i / C::kPitch) * C::kBox) + C::at(row, 4 * (i & (C::kPitch / 64 - 1)) + qd));
                w[t][0] = v.x ^ 0x80808080u; w[t][1] = v.y ^ 0x80808080u;
                w[t][2] = v.z ^ 0x80808080u; w[t][3] = v.w ^ 0x80808080u;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t a[4];
                    if constexpr (C::kQRegs) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = qa[m * C::kSteps + 4 * i + q][e];
                    } else {
                        const uint4 v = lds_u128(smem_u32(q_smem) + (uint32_t)(((m * C::kSteps + 4 * i + q) * 32 + lane) * 16));
                        a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(s[m][t], a, codes_f16(w[t][q], 0x4140), codes_f16(w[t][q], 0x4342));
                }
            }
        }

        // weights: element e of tile t is row g + 8 (e >> 1), key key0 + 8 (t & 1) + 2 qd + (e & 1)
        float kf[MT][2][NB], top[MT][2], vs[NB], vtop[MT][2];  // vtop: the largest scale of values that a row sees
        float ks[NB], vmost = 0.0f;
        bool plain = true, grow = false;  // plain: all rows see all keys, and none is NaN
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const uint32_t kb = sc[n] & 255u, vb = sc[n] >> 8;
            ks[n] = kb == 255u ? 0.0f : __uint_as_float((kb + 1u) << 23);  // twice the scale: a normal number for byte 0 too
            vs[n] = vb == 255u ? 0.0f : (float)vb;
            vmost = fmaxf(vmost, vs[n]);
            plain = plain && !edge[n] && kb != 255u && vb != 255u;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) vtop[m][h] = fmaxf(eref[m][h], vmost);
        if (!plain) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at_row = pos[m][h];
                    vtop[m][h] = eref[m][h];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        bool seen = true;
                        if (edge[n]) {
                            seen = page[n] >= 0 && key0[n] <= at_row && key0[n] < len &&
                                   (p.window == 0 || at_row - (key0[n] + kKvBlock - 1) < p.window || key0[n] < p.sinks);
#pragma unroll
                            for (int t = 2 * n; t < 2 * n + 2; ++t)
#pragma unroll
                                for (int e = 2 * h; e < 2 * h + 2; ++e) {
                                    const int key = key0[n] + 8 * (t & 1) + 2 * qd + (e & 1);
                                    const bool see = page[n] >= 0 && key <= at_row && key < len &&
                                                     (p.window == 0 || at_row - key < p.window || key < p.sinks);
                                    if (!see) s[m][t][e] = -INFINITY;
                                }
                        }
                        if (seen) {
                            vtop[m][h] = fmaxf(vtop[m][h], vs[n]);
                            // a block of NaN that a row sees: so is the row
                            if ((sc[n] & 255u) == 255u || sc[n] >> 8 == 255u) l[m][h] = __uint_as_float(0x7FC00000u);
                        }
                    }
                }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[m][h] = -INFINITY;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    // (2^24 last: with kq, large queries would leave f32; not 0: -infinity must stay what it is)
                    kf[m][h][n] = fmaxf(kq[m][h] * ks[n] * 0x1p23f, 0x1p-126f);
                    const float most = fmaxf(fmaxf(s[m][2 * n][2 * h], s[m][2 * n][2 * h + 1]), fmaxf(s[m][2 * n + 1][2 * h], s[m][2 * n + 1][2 * h + 1]));
                    top[m][h] = fmaxf(top[m][h], most * kf[m][h][n]);
                }
                // (also the first finite one: the reference is -inf)
                grow |= top[m][h] > fmaxf(mref[m][h] + kGrow8, -kFarScore) || vtop[m][h] > eref[m][h];
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(top[m][h], __shfl_xor_sync(0xffffffffu, top[m][h], 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    f[h] = 1.0f;
                    if (x > fmaxf(mref[m][h] + kGrow8, -kFarScore)) {
                        f[h] = ex2(mref[m][h] - x);
                        mref[m][h] = x;
                        l[m][h] *= f[h];
                        if (x > kFarScore && x < INFINITY) {
                            const float down = far_scale(x);
                            mref[m][h] *= down;
                            kq[m][h] *= down;
                            far[m][h] *= down;
#pragma unroll
                            for (int n = 0; n < NB; ++n) kf[m][h][n] = fmaxf(kf[m][h][n] * down, 0x1p-126f);  // (not 0, as above)
                        }
                    }
                    f[h] *= ex2(eref[m][h] - vtop[m][h]);
                    eref[m][h] = vtop[m][h];
                }
#pragma unroll
                for (int c = 0; c <= DP / 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[m][c][e] *= f[e >> 1];
            }
        }
        // A weight comes with its block's scale (in the exponent), and the sum takes it out of a block at a
        // time; a scale 2^60 below the largest leaves nothing of a weight in f16 as it is.
        uint32_t pa[MT][NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float w[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float lift = fmaxf(vs[n] - eref[m][h], -60.0f), off = lift + (mref[m][h] == -INFINITY ? kLift : kLift - mref[m][h]);
                    float sum = 0.0f;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 2 * h; e < 2 * h + 2; ++e) {
                            w[t][e] = ex2(fmaf(s[m][2 * n + t][e], kf[m][h][n], off));
                            sum += w[t][e];
                        }
                    l[m][h] = fmaf(sum, ex2(-lift), l[m][h]);
                }
                pa[m][n][0] = pack_pair<__half>(w[0][0], w[0][1]);
                pa[m][n][1] = pack_pair<__half>(w[0][2], w[0][3]);
                pa[m][n][2] = pack_pair<__half>(w[1][0], w[1][1]);
                pa[m][n][3] = pack_pair<__half>(w[1][2], w[1][3]);
                mma_f16(o[m][DP / 8], pa[m][n], kBiasF16, kBiasF16);
            }

        // O: column 8 c + g of the operand is value kVRun g + c
#pragma unroll
        for (int c16 = 0; c16 < (DP + 127) / 128; ++c16) {
            constexpr int W = DP == 64 ? 2 : 4;  // words of 4 values
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint32_t vsrc = src[n] + (uint32_t)(C::kBoxes * C::kBox);
                uint32_t w[4][W];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 8 * (i >> 1) + 2 * qd + (i & 1);
                    if constexpr (DP == 64) {
                        const uint2 v = lds_u64(vsrc + C::at(row, g >> 1) + 8 * (g & 1));
                        w[i][0] = v.x; w[i][1] = v.y;
                    } else {
                        const int run = (DP / 128) * g + c16;
                        const uint4 v = lds_u128(vsrc + (uint32_t)((run >> 3) * C::kBox) + C::at(row, run & 7));
                        w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                    }
                }
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    // bytes of keys (0, 1) and (2, 3) side by side, for values 4 q .. 4 q + 3
                    const uint32_t a01 = prmt(w[0][q], w[1][q], 0x5140) ^ 0x80808080u, b01 = prmt(w[0][q], w[1][q], 0x7362) ^ 0x80808080u;
                    const uint32_t a23 = prmt(w[2][q], w[3][q], 0x5140) ^ 0x80808080u, b23 = prmt(w[2][q], w[3][q], 0x7362) ^ 0x80808080u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t sel = e & 1 ? 0x4342 : 0x4140;
                        const uint32_t f0 = codes_f16(e < 2 ? a01 : b01, sel), f1 = codes_f16(e < 2 ? a23 : b23, sel);
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma_f16(o[m][16 * c16 + 4 * q + e], pa[m][n], f0, f1);
                    }
                }
            }
        }
    }
    if (!ok) {
        // a copy did not come: what is still on its way is waited for, and the CTA gives up
        if (lane == 0) {
            atomicOr(p.status, kStatusCopyTimeout);
            s_failed = 1;
            for (int s = 0; s < C::kSlots; ++s) mbar_wait_bounded(&s_full[warp][s], (uint32_t)((turns + n_turns - 1) / C::kSlots) & 1u, kWaitLimitNs / 8);
        }
    }
    turns += n_turns;

    // ---- the warps' parts together, in order
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 1);
            l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 2);
            if (qd == 0) {
                s_m[warp][16 * m + 8 * h + g] = mref[m][h] / far[m][h];
                s_l[warp][16 * m + 8 * h + g] = l[m][h] * 0x1p-7f;  // without kLift
            }
        }
    __syncthreads();
    if (s_failed && p.cluster == 1) return;
    // maximum over the warps; a warp's factor (1 where nothing finite was seen: NaN stays NaN)
    auto top_of = [&](int row) {
        float x = s_m[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x = fmaxf(x, s_m[w][row]);
        return x;
    };
    auto factor = [&](int w, int row, float x) { return x == -INFINITY ? 1.0f : ex2(s_m[w][row] - x); };
    float *mine = reinterpret_cast<float *>(smem8 + warp * kStages * C::kStage);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 16 * m + 8 * h + g;
            const float unit = scale_of((uint32_t)eref[m][h]) * 0x1p17f;  // 2^24 / 2^7
            const float f = factor(warp, row, top_of(row)), w128 = o[m][DP / 8][2 * h];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < DP / 8; c += 4) {
                    const int d4 = ((2 * qd + e) * C::kVRun + c) / 4;
                    *reinterpret_cast<float4 *>(mine + row * DP + 4 * (d4 ^ g)) =
                        make_float4((o[m][c][2 * h + e] - w128) * unit * f, (o[m][c + 1][2 * h + e] - w128) * unit * f,
                                    (o[m][c + 2][2 * h + e] - w128) * unit * f, (o[m][c + 3][2 * h + e] - w128) * unit * f);
                }
        }
    __syncthreads();
    const int rows = seg.rows;
    const bool whole = seg.whole;
    const int row0 = seg.row0;
    const int64_t slot = seg.slot, t0 = seg.t0;
    auto write = [&](int row, int d4, const float4 &sum, float z) {
        if (4 * d4 >= p.D) return;
        const int at_row = row0 + row, tok = (int)((unsigned)at_row / (unsigned)p.G);
        const float inv = z == 0.0f ? 0.0f : 1.0f / z;
        uint16_t *to = static_cast<uint16_t *>(p.out) + ((t0 + tok) * p.Hq + head * (int64_t)p.G + (at_row - tok * p.G)) * p.D + 4 * d4;
        using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
        const float v[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
        store4(reinterpret_cast<TO *>(to), v);
    };
    for (int i = tid; i < rows * (DP / 4); i += 32 * kWarps) {
        const int row = i / (DP / 4), d4 = i - row * (DP / 4);
        const float x = top_of(row);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4 *>(smem8 + w * kStages * C::kStage + (row * DP + 4 * (d4 ^ (row & 7))) * 4);
            sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
            z = fmaf(s_l[w][row], factor(w, row, x), z);
        }
        if (whole) {
            write(row, d4, sum, z);
        } else if (p.cluster > 1) {
            // over what this thread has just read of the first warp
            *reinterpret_cast<float4 *>(smem8 + (row * DP + 4 * (d4 ^ (row & 7))) * 4) = sum;
            if (d4 == 0) s_ml[row] = make_float2(x, s_failed ? __uint_as_float(0x7FC00000u) : z);
        } else {
            *reinterpret_cast<float4 *>(p.part_o + (slot * C::kRows + row) * DP + 4 * d4) = sum;
            if (d4 == 0) p.part_ml[slot * C::kRows + row] = make_float2(x, z);
        }
    }
    if (p.cluster > 1) {
        // the unit's CTAs together, each for its share of the rows, in order
        __syncwarp();
        cluster_sync();
        const int rank = (int)cluster_ctarank();
        for (int i = tid + 32 * kWarps * rank; i < rows * (DP / 4); i += 32 * kWarps * p.cluster) {
            const int row = i / (DP / 4), d4 = i - row * (DP / 4);
            const uint32_t from = smem_u32(smem8) + (uint32_t)((row * DP + 4 * (d4 ^ (row & 7))) * 4), ml = smem_u32(&s_ml[row]);
            float4 v[kMostCluster];
            float2 x[kMostCluster];
            float top = -INFINITY, z = 0.0f;
#pragma unroll
            for (int c = 0; c < kMostCluster; ++c) {
                x[c] = make_float2(-INFINITY, 0.0f);
                v[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c < p.cluster) {
                    x[c] = dsmem_ld_f32x2(dsmem_at(ml, (uint32_t)c));
                    v[c] = dsmem_ld_f32x4(dsmem_at(from, (uint32_t)c));
                }
                top = fmaxf(top, x[c].x);
            }
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < kMostCluster; ++c) {
                const float f = top == -INFINITY ? 1.0f : ex2(x[c].x - top);
                z = fmaf(x[c].y, f, z);
                sum.x = fmaf(v[c].x, f, sum.x);
                sum.y = fmaf(v[c].y, f, sum.y);
                sum.z = fmaf(v[c].z, f, sum.z);
                sum.w = fmaf(v[c].w, f, sum.w);
            }
            write(row, d4, sum, z);
        }
        __syncwarp();
        cluster_sync();  // nobody's shared memory goes before it has been read
        return;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();  // the next unit's copies and queries go where this one's sums were
    }
}

// Joins the parts of units that were cut, a warp to a row.
template <int DP, int ROWS, bool BF>
__global__ void __launch_bounds__(32 * kWarps) attn8_join_kernel(const __grid_constant__ Attn8Params p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    constexpr int kPer = ROWS / kWarps;  // CTAs of a unit
    const int c0 = (int)(blockIdx.x / kPer), row = (int)(blockIdx.x - c0 * kPer) * kWarps + (int)(threadIdx.x >> 5);
    const Cut cut = cut_of(p, c0, lane);
    if (!cut.is) return;
    const Item it = item_of<ROWS>(p, cut.item);
    if (row >= it.rows) return;
    const int c1 = cut.c1, head = cut.head;
    auto slot_of = [&](int c) { return (int64_t)(2 * c + (c > c0 ? 0 : 1)) * ROWS + row; };
    constexpr int L = DP / 32;  // values a lane
    constexpr int kAtOnce = 8;  // parts in flight
    float top = -INFINITY, sum[L], z = 0.0f;
#pragma unroll
    for (int e = 0; e < L; ++e) sum[e] = 0.0f;
#pragma unroll 1
    for (int c = c0; c <= c1; c += kAtOnce) {
        float2 x[kAtOnce], v[kAtOnce][L / 2];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            x[i] = make_float2(-INFINITY, 0.0f);
            if (c + i <= c1) x[i] = p.part_ml[slot_of(c + i)];
#pragma unroll
            for (int e = 0; e < L / 2; ++e) {
                v[i][e] = make_float2(0.0f, 0.0f);
                if (c + i <= c1) v[i][e] = *reinterpret_cast<const float2 *>(p.part_o + slot_of(c + i) * DP + L * lane + 2 * e);
            }
        }
        float now = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) now = fmaxf(now, x[i].x);
        const float f0 = now == -INFINITY ? 1.0f : ex2(top - now);
        z *= f0;
#pragma unroll
        for (int e = 0; e < L; ++e) sum[e] *= f0;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float f = now == -INFINITY ? 1.0f : ex2(x[i].x - now);
            z = fmaf(x[i].y, f, z);
#pragma unroll
            for (int e = 0; e < L / 2; ++e) {
                sum[2 * e] = fmaf(v[i][e].x, f, sum[2 * e]);
                sum[2 * e + 1] = fmaf(v[i][e].y, f, sum[2 * e + 1]);
            }
        }
        top = now;
    }
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    const int at_row = it.row0 + row, tok = (int)((unsigned)at_row / (unsigned)p.G);
    uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) +
                                                ((it.r.t0 + tok) * p.Hq + head * (int64_t)p.G + (at_row - tok * p.G)) * p.D + L * lane);
    using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
#pragma unroll
    for (int e = 0; e < L; e += 2)
        if (L * lane + e < p.D) to[e / 2] = pack_pair<TO>(sum[e] * inv, sum[e + 1] * inv);
}

// How a call is cut.
struct Plan8 {
    int mt, dp, tiles, ctas, cluster, grid;
    int64_t units;  // (request, tile, head)
    size_t bytes;
};
Plan8 plan_of(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len, int64_t max_new, int64_t window,
              int64_t sinks) {
    Plan8 c;
    const int64_t rows = max_new * (q_heads / kv_heads);
    c.dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    c.mt = rows > 16 && c.dp <= 128 ? 2 : 1;
    c.tiles = (int)ceil_div(rows, 16 * c.mt);
    const int64_t items = B * c.tiles;
    c.units = items * kv_heads;
    int64_t blocks = ceil_div(max_len, kKvBlock);
    if (window > 0) blocks = std::min(blocks, ceil_div(window + 16 * c.mt, kKvBlock) + 1 + ceil_div(sinks, kKvBlock));
    const int64_t room = 152 * (c.dp * c.mt <= 128 ? 3 : c.dp <= 128 ? 2 : 1);
    // A unit to a cluster (one kernel): as many CTAs as have two blocks a warp and fill the machine once.
    c.cluster = 1;
    while (c.cluster < kMostCluster && c.units * c.cluster * 2 <= room && blocks >= 2 * kWarps * 2 * c.cluster) c.cluster *= 2;
    // Or the line of all units' blocks in even parts, which the second kernel and its launch make
    // dearer by about kJoinBlocks of a CTA.
    const int64_t clusters = ceil_div(c.units * c.cluster, room) * ceil_div(blocks, c.cluster);
    const int64_t line = std::max<int64_t>(ceil_div(c.units * blocks, room), kMinBlocks) + kJoinBlocks;
    c.ctas = 0;
    c.grid = (int)(c.units * c.cluster);
    c.bytes = 0;
    if (items <= kMostItems && line < clusters) {
        c.cluster = 1;
        c.ctas = c.grid = (int)std::min<int64_t>(room, ceil_div(c.units * blocks, kMinBlocks));
        c.bytes = (size_t)c.ctas * 2 * 16 * c.mt * (c.dp + 2) * 4 + (size_t)(items + 2) / 2 * 16;
    }
    return c;
}

template <int ROWS, bool BF>
cudaError_t join_launch(const Attn8Params &p, int dp, cudaStream_t st) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.ctas - 1) * (ROWS / kWarps)), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (dp == 64) return cudaLaunchKernelEx(&cfg, attn8_join_kernel<64, ROWS, BF>, p);
    if (dp == 128) return cudaLaunchKernelEx(&cfg, attn8_join_kernel<128, ROWS, BF>, p);
    return cudaLaunchKernelEx(&cfg, attn8_join_kernel<256, ROWS, BF>, p);
}

template <int DP, int MT, bool BF>
cudaError_t attn8_launch(const Attn8Params &p, const Plan8 &c, cudaStream_t st) {
    using C = Cfg8<DP, MT>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)attn8_kernel<DP, MT, BF>, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.grid, 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = c.cluster > 1 ? 2 : 1;
    const cudaError_t k = cudaLaunchKernelEx(&cfg, attn8_kernel<DP, MT, BF>, p);
    return k != cudaSuccess || c.ctas == 0 ? k : join_launch<C::kRows, BF>(p, DP, st);
}

template <bool BF>
cudaError_t attn8_launch_type(const Attn8Params &p, const Plan8 &c, cudaStream_t st) {
    if (c.dp == 64) return c.mt == 1 ? attn8_launch<64, 1, BF>(p, c, st) : attn8_launch<64, 2, BF>(p, c, st);
    if (c.dp == 128) return c.mt == 1 ? attn8_launch<128, 1, BF>(p, c, st) : attn8_launch<128, 2, BF>(p, c, st);
    return attn8_launch<256, 1, BF>(p, c, st);
}

}  // namespace

bool attn8_maps(Attn8Params &p, const w4_kv8_cache &c, int dp, int tokens, CUtensorMapSwizzle swizzle) {
    // a tensor map's strides grow from dimension to dimension
    const int ti = c.token_stride < c.head_stride ? 1 : 2, hi = 3 - ti;
    p.tok_inner = ti == 1;
    uint64_t dims[4] = {(uint64_t)c.head_dim, 0, 0, (uint64_t)c.pages}, strides[3] = {0, 0, (uint64_t)c.page_stride};
    uint32_t box[4] = {(uint32_t)std::min(dp, 128), 1, 1, 1};
    dims[ti] = (uint64_t)c.page_size;
    dims[hi] = (uint64_t)c.heads;
    strides[ti - 1] = (uint64_t)c.token_stride;
    strides[hi - 1] = (uint64_t)c.head_stride;
    box[ti] = (uint32_t)tokens;
    return encode_tmap(&p.kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.k, dims, strides, box, swizzle) &&
           encode_tmap(&p.vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.v, dims, strides, box, swizzle);
}

namespace {

// Rows of a request and key head from which on the tensor-core kernel is taken.
bool many_rows(int64_t max_new, int32_t G) { return max_new * G > kFewRows; }

}  // namespace

size_t attention_kv8_workspace(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len,
                               int64_t max_new, int64_t window, int64_t sinks) {
    if (many_rows(max_new, q_heads / kv_heads))
        return attn8_tc_plan(B, q_heads, kv_heads, head_dim, max_len, max_new, window, sinks).bytes;
    return plan_of(B, q_heads, kv_heads, head_dim, max_len, max_new, window, sinks).bytes;
}

cudaError_t launch_attention_kv8(const void *q, int32_t q_type, int64_t ld, const w4_kv8_cache &c, const int32_t *table,
                                 int64_t width, const int32_t *ctx_len, const int32_t *cu_new, int64_t B, int64_t T,
                                 int32_t q_heads, float scale, int64_t max_len, int64_t max_new, int64_t window,
                                 int64_t sinks, void *out, void *workspace, uint32_t *status, cudaStream_t st) {
    Attn8Params p = {};
    p.q = q; p.out = out; p.status = status; p.ks = c.k_scale; p.vs = c.v_scale;
    p.table = table; p.ctx_len = ctx_len; p.cu_new = cu_new;
    p.ld = ld; p.width = width; p.T = T; p.pages = c.pages;
    p.B = (int)B; p.Hq = q_heads; p.Hkv = c.heads; p.G = q_heads / c.heads; p.D = c.head_dim;
    p.page_shift = log2_of(c.page_size);
    p.window = (int)window; p.sinks = (int)sinks;
    p.max_new = (int)max_new;
    p.scale_log2 = scale * kLog2e;
    auto places = [&](int ctas, int tiles, int rows, int dp) {  // of the parts, in the workspace
        p.tiles = tiles;
        p.ctas = ctas;
        p.first = static_cast<int64_t *>(workspace);
        p.part_o = reinterpret_cast<float *>(p.first + (B * tiles + 2) / 2 * 2);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)ctas * 2 * rows * dp);
    };
    if (many_rows(max_new, p.G)) {
        const Plan8Tc plan = attn8_tc_plan(B, q_heads, c.heads, c.head_dim, max_len, max_new, window, sinks);
        places(plan.ctas, plan.tiles, 128 * plan.rt, plan.dp);
        p.box = std::min(c.page_size, 64) / kKvBlock;
        if (!attn8_maps(p, c, plan.dp, std::min(c.page_size, 64), CU_TENSOR_MAP_SWIZZLE_NONE)) return cudaErrorInvalidValue;
        return launch_attn8_tc(p, plan, q_type == W4_BF16, st);
    }
    const Plan8 plan = plan_of(B, q_heads, c.heads, c.head_dim, max_len, max_new, window, sinks);
    places(plan.ctas, plan.tiles, 16 * plan.mt, plan.dp);
    p.cluster = plan.cluster;
    p.step = 1;
    p.least = kMinBlocks;
    if (!attn8_maps(p, c, plan.dp, kKvBlock, plan.dp < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    return q_type == W4_BF16 ? attn8_launch_type<true>(p, plan, st) : attn8_launch_type<false>(p, plan, st);
}

}  // namespace w4
