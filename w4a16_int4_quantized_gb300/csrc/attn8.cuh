// attn8.cuh -- what the two kernels of the 8-bit attention share: what a row tile sees, and how
// the work is dealt out.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "rows.cuh"
#include "w4.h"

namespace w4 {

constexpr float kGrow8 = 8.0f;  // log2 by which a maximum may grow before O is rescaled
constexpr float kLift = 7.0f;   // log2 of the factor of the weights: 2^(8 + 7) is below f16's largest value
// Scores (log2 units) below this count as -infinity; where one is above its opposite, the row's scores are
// scaled down to half of it or more from there on.  An exponent is one fused product and sum, exact but for the
// rounding of the maximum, which beyond would not be small (the weights' 2^15 would leave f16).  The price: a
// score d times the largest below that counts as 2^21 d to 2^22 d below it, whatever its size.
constexpr float kFarScore = 0x1p22f;
W4_DEV float far_scale(float x) { return __uint_as_float((uint32_t)(127 + 127 + 21 - (int)(__float_as_uint(x) >> 23)) << 23); }  // x to 2^21 .. 2^22

constexpr int64_t kMostItems = 4096;  // (request, tile) whose steps are counted on the device; more are units enough

struct Attn8Params {
    CUtensorMap kmap, vmap;  // bytes: D, tokens and heads in the order of their strides, pages; a box: 128 (64) values of 16 tokens of a head
    uint32_t *status;
    const void *q;
    void *out;
    const uint8_t *ks, *vs;
    const int32_t *table, *ctx_len, *cu_new;
    float *part_o;    // [CTA][2][rows][DP]
    float2 *part_ml;  // [CTA][2][rows]: maximum (log2), sum
    int64_t *first;   // [items + 1]: blocks before each item, all of them
    int64_t ld, width, T, pages;
    int tok_inner;  // the token stride is the smaller one
    int B, Hq, Hkv, G, D, page_shift;
    int window, sinks;
    int tiles;      // of a request, at most
    int step;       // blocks that are worked on together; a unit's are counted so
    int box;        // of them in a box of the tensor maps
    int least;      // steps of a CTA, if there are as many: a part costs its write and its join
    int ctas;       // that share the line of blocks at most; 0: a unit to each cluster
    int cluster;    // CTAs of one, which share a unit's blocks
    int max_new;
    float scale_log2;
};

// The blocks of 16 keys that a row tile sees: those of the first tokens, then [first, end).
struct Span {
    int sink, first, end;
    W4_DEV int blocks() const { return sink + end - first; }
    W4_DEV int block(int i) const { return i < sink ? i : first + (i - sink); }
};
// Rows r0 .. r0 + rows - 1 of a request; pos0, pos1: the positions of the first and last one's tokens.
W4_DEV Span span_of(const Attn8Params &p, const KvRequest &r, int pos0, int pos1) {
    Span s;
    s.end = (min(pos1 + 1, r.len) + kKvBlock - 1) >> kKvBlockLog;
    // (in whole steps from the beginning of the request on, and in whole steps of first tokens: a
    // step's blocks then lie side by side)
    s.first = p.window > 0 ? (max(0, pos0 - p.window + 1) >> kKvBlockLog) / p.step * p.step : 0;
    s.first = min(s.first, s.end / p.step * p.step);
    s.sink = min(((p.sinks >> kKvBlockLog) + ((p.sinks & (kKvBlock - 1)) != 0) + p.step - 1) / p.step * p.step, s.first);
    return s;
}

// An item is (request, tile of its rows): its rows and the blocks that they see.
struct Item {
    KvRequest r;
    int b, row0, all_rows, rows, pos0, pos1;
    Span span;
    int nb;  // steps
};
template <int ROWS>
W4_DEV Item item_of(const Attn8Params &p, int64_t i) {
    Item t;
    t.b = (int)((unsigned)i / (unsigned)p.tiles);
    t.r = kv_request(p.cu_new, p.ctx_len, t.b, p.T, p.width, p.page_shift);
    t.row0 = ((int)i - t.b * p.tiles) * ROWS;
    t.all_rows = min(t.r.n, p.max_new) * p.G;
    t.rows = max(0, min(ROWS, t.all_rows - t.row0));
    t.nb = 0;
    t.pos0 = t.pos1 = 0;
    if (t.rows > 0) {
        t.pos0 = t.r.ctx + (int)((unsigned)t.row0 / (unsigned)p.G);
        t.pos1 = t.r.ctx + (int)((unsigned)(t.row0 + t.rows - 1) / (unsigned)p.G);
        t.span = span_of(p, t.r, t.pos0, t.pos1);
        t.nb = max((t.span.blocks() + p.step - 1) / p.step, 1);  // rows that see nothing have a block of nothing: zeros are written
    }
    return t;
}

// Steps of a CTA, of W in all.
W4_DEV int64_t share_of(const Attn8Params &p, int64_t W) { return max((W + p.ctas - 1) / p.ctas, (int64_t)p.least); }

// The unit that CTA c0's part of the line ends in, if that goes on in the next CTA and began in this one.
struct Cut {
    bool is;
    int head, c1;  // its key head, the last CTA that has some of it
    int64_t item;
};
W4_DEV Cut cut_of(const Attn8Params &p, int c0, int lane) {
    Cut cut = {};
    const int64_t items = (int64_t)p.B * p.tiles, W = p.first[items], share = share_of(p, W), s = share * (c0 + 1);
    if (s >= W) return cut;
    int64_t item = 0, hi = items;
    while (hi - item > 1) {  // 32 places at a time
        const int64_t step = ceil_div(hi - item, 32), i = item + lane * step;
        const int n = __popc(__ballot_sync(0xffffffffu, i < hi && p.first[i] <= s));
        const int64_t next = item + max(n - 1, 0) * step;
        hi = min(hi, next + step);
        item = next;
    }
    const int64_t u = p.first[item], nb = (p.first[item + 1] - u) / p.Hkv;
    cut.item = item;
    cut.head = (int)((s - u) / nb);
    const int64_t u0 = u + cut.head * nb;
    cut.is = u0 != s && u0 >= share * c0;
    cut.c1 = (int)((u0 + nb - 1) / share);
    return cut;
}

// attn8_tc.cu -- many rows: the tensor cores of the fifth generation.
struct Plan8Tc {
    int rt, dp, tiles, ctas;
    int64_t items;
    size_t bytes;
};
Plan8Tc attn8_tc_plan(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len, int64_t max_new,
                      int64_t window, int64_t sinks);
cudaError_t launch_attn8_tc(Attn8Params p, const Plan8Tc &c, bool bf16, cudaStream_t st);
// attn8.cu.
// Tensor maps of the codes: boxes of `tokens` of a head, dp values (128 at most) wide.
bool attn8_maps(Attn8Params &p, const w4_kv8_cache &c, int dp, int tokens, CUtensorMapSwizzle swizzle);

}  // namespace w4
