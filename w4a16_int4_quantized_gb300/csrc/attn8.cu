// attn8.cu -- causal attention over a paged cache held in 8 bits, whole or through a sliding
// window beside a few first tokens.
//
// Rows are (new token, query head of the key head's group), 16 to a tile and one or two tiles
// to a warp; the warps of a CTA share the rows and take blocks of 16 keys in turn, each with
// its own running maximum, sum and O, and the keys of a request are cut into parts for
// more CTAs.  A warp does not wait for others before its end: every lane copies (cp.async) the
// codes that it will itself put into the tensor-core operands, several blocks ahead, and reads
// nothing that another lane copied.
//
// Operands without shuffles: which of 16 keys and which value of a head stands at which place
// of an operand is free as long as both factors agree.  For S = Q K^T a lane's quad index q
// takes values 64 i + 16 q .. + 15 of a key (a run of 16 bytes), for O = P V its group
// index g takes values g D/8 .. of keys 4 q .. 4 q + 3, whose weights are what S left in that
// lane.
// Codes become f16 exactly: u = code + 128 under the exponent byte 0x64 is 1024 + u, from which
// 1152 is taken.  Scales are powers of two, one for a block of 16 keys: the keys' multiplies
// the scores, the values' the weights, relative to the largest one met so far (a weight
// is then rounded to f16 with a factor 2^7: what it loses is at most 2^-32 of the largest).
// Queries in bf16 go to f16 with a power of two of their row, so that the largest lies in
// [2^13, 2^14): what a value loses is at most 2^-39 of the largest.
// O is rescaled only when a row's maximum has grown by more than 2^8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "rows.cuh"
#include "smem_limit.h"
#include "w4.h"

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;
constexpr float kGrow8 = 8.0f;  // log2 by which a maximum may grow before O is rescaled
constexpr float kLift = 7.0f;   // log2 of the factor of the weights: 2^(8 + 7) is below f16's largest value

struct Attn8Params {
    const void *q;
    void *out;
    const int8_t *k, *v;
    const uint8_t *ks, *vs;
    const int32_t *table, *ctx_len, *cu_new;
    float *part_o;    // [request, tile][head][part][rows][DP]
    float2 *part_ml;  // the same without DP: maximum (log2), sum
    int64_t ld, width, T, pages, page_stride, token_stride, head_stride;
    int B, Hq, Hkv, G, D, page_shift;
    int window, sinks;
    int tiles;      // of a request, at most
    int parts;      // of its keys, at most
    int part_len;   // blocks of a part
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
    s.first = p.window > 0 ? max(0, pos0 - p.window + 1) >> kKvBlockLog : 0;
    s.first = min(s.first, s.end);
    s.sink = min((p.sinks >> kKvBlockLog) + ((p.sinks & (kKvBlock - 1)) != 0), s.first);
    return s;
}

W4_DEV void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
W4_DEV void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
W4_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
W4_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

W4_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

W4_DEV float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two biased codes (bytes `sel` of w) as f16.
W4_DEV uint32_t codes_f16(uint32_t w, uint32_t sel) {
    const uint32_t h = prmt(w, 0x64646464u, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));  // 1152
    return *reinterpret_cast<const uint32_t *>(&r);
}

// DP: head_dim rounded up to 64; MT: tiles of 16 rows.
template <int DP, int MT>
struct Cfg8 {
    static constexpr int kChunks = DP / 64;  // 16-byte runs of a key in a lane
    static constexpr int kSteps = DP / 16;   // of S along the head
    static constexpr int kVRun = DP / 8;     // bytes of a value in a lane
    static constexpr int kStage = 32 * DP;   // bytes of a block of a warp: 16 keys, then 16 values
    static constexpr int kRows = 16 * MT;
    static constexpr bool kQRegs = DP * MT <= 128;  // Q stays in registers, else in shared memory
    static constexpr int kQBytes = kQRegs ? 0 : MT * kSteps * 32 * 16;
    static constexpr int kSmem = kWarps * kStages * kStage + kQBytes;
    static constexpr int kCtas = DP * MT <= 128 ? 3 : DP <= 128 ? 2 : 1;  // an SM
    static_assert(kStages * kStage >= kRows * DP * 4, "a warp's O takes the place of its ring at the end");
};

template <int DP, int MT, bool BF>
__global__ void __launch_bounds__(32 * kWarps, Cfg8<DP, MT>::kCtas) attn8_kernel(const Attn8Params p) {
    using C = Cfg8<DP, MT>;
    extern __shared__ __align__(128) uint8_t smem8[];
    __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, qd = lane & 3;
    uint32_t at = blockIdx.x;
    const int part = (int)(at % (uint32_t)p.parts);
    at /= (uint32_t)p.parts;
    const int head = (int)(at % (uint32_t)p.Hkv);
    at /= (uint32_t)p.Hkv;
    const int tile = p.tiles - 1 - (int)(at % (uint32_t)p.tiles);  // later tiles see more keys: they go first
    const int b = (int)(at / (uint32_t)p.tiles);
    const KvRequest r = kv_request(p.cu_new, p.ctx_len, b, p.T, p.width, p.page_shift);
    const int64_t row0 = (int64_t)tile * C::kRows, all_rows = (int64_t)min(r.n, p.max_new) * p.G;
    if (row0 >= all_rows) return;
    const int rows = (int)min((int64_t)C::kRows, all_rows - row0);
    const int pos0 = r.ctx + (int)(row0 / p.G), pos1 = r.ctx + (int)((row0 + rows - 1) / p.G);
    const Span span = span_of(p, r, pos0, pos1);
    const int nb = span.blocks();
    // the part's blocks; the last part takes all that is left
    const int64_t from = (int64_t)part * p.part_len;
    if (from >= nb && part > 0) return;
    const int b0 = (int)from, b1 = part == p.parts - 1 ? nb : min(nb, b0 + p.part_len);

    // ---- queries: rows g and g + 8 of each tile, as operands
    int pos[MT][2];
    float kq[MT][2];  // from products to log2 units, without the keys' scale
    uint32_t qa[C::kQRegs ? MT * C::kSteps : 1][4];
    uint8_t *q_smem = smem8 + kWarps * kStages * C::kStage;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint2 raw[2][C::kSteps];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = row0 + 16 * m + 8 * h + g;
            const bool on = row < all_rows;
            const int tok = (int)(row / p.G);
            pos[m][h] = on ? r.ctx + tok : -1;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (r.t0 + tok) * p.ld + (head * (int64_t)p.G + (row - (int64_t)tok * p.G)) * p.D;
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

    // ---- the warp's blocks: b0 + warp, then every fourth
    const int n_mine = b1 - b0 > warp ? (b1 - b0 - warp + kWarps - 1) / kWarps : 0;
    const int32_t *row_of = p.table + (int64_t)b * p.width;
    const int64_t scale_head = (int64_t)head << (p.page_shift - kKvBlockLog);
    const int64_t scale_page = (int64_t)p.Hkv << (p.page_shift - kKvBlockLog);
    // lane i: the page and the scales of the warp's block j + i (-1: no such page)
    auto fetch = [&](int j, int &page, uint32_t &scales) {
        page = -1;
        scales = 0u;
        if (j + lane < n_mine) {
            const int key = span.block(b0 + warp + kWarps * (j + lane)) << kKvBlockLog;
            page = __ldg(row_of + (key >> p.page_shift));
            if (page >= p.pages) page = -1;
            if (page >= 0) {
                const int64_t s = page * scale_page + scale_head + ((key & ((1 << p.page_shift) - 1)) >> kKvBlockLog);
                scales = (uint32_t)__ldg(p.ks + s) | (uint32_t)__ldg(p.vs + s) << 8;
            }
        }
    };
    const uint32_t ring = smem_u32(smem8) + (uint32_t)(warp * kStages * C::kStage + lane * 16);
    const int8_t *k_lane = p.k + head * p.head_stride + (4 * (g >> 1) + (g & 1)) * p.token_stride + 16 * qd;
    const int8_t *v_lane = p.v + head * p.head_stride + 4 * qd * p.token_stride + C::kVRun * g;
    auto copy = [&](int j, int page) {
        if (j < n_mine && page >= 0) {
            const int key = span.block(b0 + warp + kWarps * j) << kKvBlockLog;
            const int64_t off = page * p.page_stride + (key & ((1 << p.page_shift) - 1)) * p.token_stride;
            const uint32_t dst = ring + (uint32_t)((j & (kStages - 1)) * C::kStage);
            const int8_t *k = k_lane + off, *v = v_lane + off;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < C::kChunks; ++i)
                    if (64 * i + 16 * qd < p.D)
                        cp_async16(dst + (uint32_t)((t * C::kChunks + i) * 512), k + 2 * t * p.token_stride + 64 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t to = dst + (uint32_t)(C::kChunks * 1024);
                if constexpr (DP == 64) {
                    if (8 * g < p.D) cp_async8(to + (uint32_t)((i >> 1) * 512 + (i & 1) * 8), v + i * p.token_stride);
                } else {
#pragma unroll
                    for (int c = 0; c < DP / 128; ++c)
                        if (C::kVRun * g + 16 * c < p.D)
                            cp_async16(to + (uint32_t)((i * (DP / 128) + c) * 512), v + i * p.token_stride + 16 * c);
                }
            }
        }
        cp_commit();
    };

    float o[MT][DP / 8][4];
    float mref[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int c = 0; c < DP / 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[m][c][e] = 0.0f;
        mref[m][0] = mref[m][1] = -INFINITY;
        l[m][0] = l[m][1] = 0.0f;
    }
    int eref = 0;  // scale byte that the weights are relative to

    int page_now, page_next;
    uint32_t sc_now, sc_next;
    fetch(0, page_now, sc_now);
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) copy(j, __shfl_sync(0xffffffffu, page_now, j));
    fetch(32, page_next, sc_next);

#pragma unroll 1
    for (int j = 0; j < n_mine; ++j) {
        const int ji = j & 31;
        if (j > 0 && ji == 0) {
            page_now = page_next;
            sc_now = sc_next;
            fetch(j + 32, page_next, sc_next);
        }
        const int page = __shfl_sync(0xffffffffu, page_now, ji);
        const uint32_t sc = __shfl_sync(0xffffffffu, sc_now, ji);
        {
            // the place of the block before, which this lane has read
            const int ahead = ji + kStages - 1;
            const int a0 = __shfl_sync(0xffffffffu, page_now, ahead & 31), a1 = __shfl_sync(0xffffffffu, page_next, ahead & 31);
            copy(j + kStages - 1, ahead < 32 ? a0 : a1);
        }
        cp_wait<kStages - 1>();
        if (page < 0) continue;  // keys of a page outside the cache are not seen
        const uint32_t src = ring + (uint32_t)((j & (kStages - 1)) * C::kStage);
        const int key0 = span.block(b0 + warp + kWarps * j) << kKvBlockLog;

        // S
        float s[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][t][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i) {
            uint32_t w[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4 v = lds_u128(src + (uint32_t)((t * C::kChunks + i) * 512));
                w[t][0] = v.x ^ 0x80808080u; w[t][1] = v.y ^ 0x80808080u;
                w[t][2] = v.z ^ 0x80808080u; w[t][3] = v.w ^ 0x80808080u;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t bf[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    bf[t][0] = codes_f16(w[t][q], 0x4140);
                    bf[t][1] = codes_f16(w[t][q], 0x4342);
                }
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
                    for (int t = 0; t < 2; ++t) mma_f16(s[m][t], a, bf[t][0], bf[t][1]);
                }
            }
        }

        // weights: element e of tile t is row g + 8 (e >> 1), key key0 + 4 qd + 2 t + (e & 1)
        const float ks = scale_of(sc & 255u);
        const uint32_t vs = sc >> 8;
        const int last = key0 + kKvBlock - 1;
        const bool edge = last > pos0 || last >= r.len ||
                          (p.window > 0 && key0 <= pos1 - p.window && last >= p.sinks);
        uint32_t hidden = 0u;  // bit 8 m + 4 t + e
        bool grow = vs != 255u && (int)vs > eref;
        float top[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[m][t][e] *= kq[m][e >> 1] * ks;
            if (edge) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + 4 * qd + 2 * t + (e & 1), at_row = pos[m][e >> 1];
                        const bool see = key <= at_row && key < r.len &&
                                         (p.window == 0 || at_row - key < p.window || key < p.sinks);
                        if (!see) {
                            s[m][t][e] = -INFINITY;
                            hidden |= 1u << (8 * m + 4 * t + e);
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[m][h] = fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]), fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1]));
                grow |= top[m][h] > mref[m][h] + kGrow8;  // also the first finite one: the reference is -inf
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
            float fe = 1.0f;
            if (vs != 255u && (int)vs > eref) {
                fe = ex2f((float)(eref - (int)vs));
                eref = (int)vs;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(top[m][h], __shfl_xor_sync(0xffffffffu, top[m][h], 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    f[h] = 1.0f;
                    if (x > mref[m][h] + kGrow8) {
                        f[h] = ex2f(mref[m][h] - x);
                        mref[m][h] = x;
                        l[m][h] *= f[h];
                    }
                    f[h] *= fe;
                }
#pragma unroll
                for (int c = 0; c < DP / 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[m][c][e] *= f[e >> 1];
            }
        }
        const float vf = vs == 255u ? __uint_as_float(0x7FC00000u) : ex2f((float)((int)vs - eref) + kLift);
        uint32_t pa[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float w[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float zero = mref[m][h] == -INFINITY ? 0.0f : mref[m][h];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 2 * h; e < 2 * h + 2; ++e) {
                        const float x = ex2f(s[m][t][e] - zero);
                        l[m][h] += x;
                        w[t][e] = x * vf;
                    }
            }
            if (edge) {  // 0 * NaN
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden >> (8 * m + 4 * t + e) & 1u) w[t][e] = 0.0f;
            }
            pa[m][0] = pack_pair<__half>(w[0][0], w[0][1]);
            pa[m][1] = pack_pair<__half>(w[0][2], w[0][3]);
            pa[m][2] = pack_pair<__half>(w[1][0], w[1][1]);
            pa[m][3] = pack_pair<__half>(w[1][2], w[1][3]);
        }

        // O: column 8 c + g of the operand is value kVRun g + c
        const uint32_t vsrc = src + (uint32_t)(C::kChunks * 1024);
#pragma unroll
        for (int c16 = 0; c16 < (DP + 127) / 128; ++c16) {
            constexpr int W = DP == 64 ? 2 : 4;  // words of 4 values
            uint32_t w[4][W];
            if constexpr (DP == 64) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = lds_u128(vsrc + (uint32_t)(i * 512));
                    w[2 * i][0] = v.x; w[2 * i][1] = v.y;
                    w[2 * i + 1][0] = v.z; w[2 * i + 1][1] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = lds_u128(vsrc + (uint32_t)((i * (DP / 128) + c16) * 512));
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
                    for (int m = 0; m < MT; ++m) mma_f16(o[m][16 * c16 + 4 * q + e], pa[m], f0, f1);
                }
            }
        }
    }
    cp_wait<0>();

    // ---- the warps' parts together, in order
    const float unit = scale_of((uint32_t)eref) * 0x1p-7f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 1);
            l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 2);
            if (qd == 0) {
                s_m[warp][16 * m + 8 * h + g] = mref[m][h];
                s_l[warp][16 * m + 8 * h + g] = l[m][h];
            }
        }
    __syncthreads();
    // maximum over the warps; a warp's factor (1 where nothing finite was seen: NaN stays NaN)
    auto top_of = [&](int row) {
        float x = s_m[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x = fmaxf(x, s_m[w][row]);
        return x;
    };
    auto factor = [&](int w, int row, float x) { return x == -INFINITY ? 1.0f : ex2f(s_m[w][row] - x); };
    float *mine = reinterpret_cast<float *>(smem8 + warp * kStages * C::kStage);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 16 * m + 8 * h + g;
            const float f = factor(warp, row, top_of(row));
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < DP / 8; c += 4) {
                    const int d4 = ((2 * qd + e) * C::kVRun + c) / 4;
                    *reinterpret_cast<float4 *>(mine + row * DP + 4 * (d4 ^ g)) =
                        make_float4(o[m][c][2 * h + e] * unit * f, o[m][c + 1][2 * h + e] * unit * f,
                                    o[m][c + 2][2 * h + e] * unit * f, o[m][c + 3][2 * h + e] * unit * f);
                }
        }
    __syncthreads();
    const bool whole = p.parts == 1 || nb <= p.part_len;
    const int64_t slot = (((int64_t)b * p.tiles + tile) * p.Hkv + head) * p.parts + part;
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
            if (4 * d4 >= p.D) continue;
            const int64_t at_row = row0 + row, tok = at_row / p.G;
            const float inv = z == 0.0f ? 0.0f : 1.0f / z;
            uint16_t *to = static_cast<uint16_t *>(p.out) + ((r.t0 + tok) * p.Hq + head * (int64_t)p.G + (at_row - tok * p.G)) * p.D + 4 * d4;
            using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
            const float v[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
            store4(reinterpret_cast<TO *>(to), v);
        } else {
            *reinterpret_cast<float4 *>(p.part_o + (slot * C::kRows + row) * DP + 4 * d4) = sum;
            if (d4 == 0) p.part_ml[slot * C::kRows + row] = make_float2(x, z);
        }
    }
}

// Joins the parts of rows whose keys were cut, a warp to a row.
template <int DP, int MT, bool BF>
__global__ void __launch_bounds__(32 * kWarps) attn8_join_kernel(const Attn8Params p) {
    using C = Cfg8<DP, MT>;
    griddep_wait();
    const int lane = threadIdx.x & 31;
    int64_t at = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int row = (int)(at % C::kRows);
    at /= C::kRows;
    const int64_t unit = at;
    const int head = (int)(at % p.Hkv);
    at /= p.Hkv;
    const int tile = (int)(at % p.tiles);
    const int64_t b = at / p.tiles;
    if (b >= p.B) return;
    const KvRequest r = kv_request(p.cu_new, p.ctx_len, b, p.T, p.width, p.page_shift);
    const int64_t row0 = (int64_t)tile * C::kRows, all_rows = (int64_t)min(r.n, p.max_new) * p.G;
    if (row0 + row >= all_rows) return;
    const int rows = (int)min((int64_t)C::kRows, all_rows - row0);
    const Span span = span_of(p, r, r.ctx + (int)(row0 / p.G), r.ctx + (int)((row0 + rows - 1) / p.G));
    const int nb = span.blocks();
    if (nb <= p.part_len) return;  // it was not cut
    const int n = (int)min((int64_t)p.parts, ceil_div(nb, p.part_len));
    const float2 *ml = p.part_ml + unit * p.parts * C::kRows + row;
    const float *po = p.part_o + (unit * p.parts * C::kRows + row) * DP;
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[(int64_t)i * C::kRows].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    constexpr int W = DP / 32;  // values a lane
    float sum[W], z = 0.0f;
#pragma unroll
    for (int e = 0; e < W; ++e) sum[e] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float2 x = ml[(int64_t)i * C::kRows];
        const float f = top == -INFINITY ? 1.0f : ex2f(x.x - top);
        z = fmaf(x.y, f, z);
        const float *src = po + (int64_t)i * C::kRows * DP + W * lane;
#pragma unroll
        for (int e = 0; e < W; e += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(src + e);
            sum[e] = fmaf(v.x, f, sum[e]);
            sum[e + 1] = fmaf(v.y, f, sum[e + 1]);
        }
    }
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    const int64_t at_row = row0 + row, tok = at_row / p.G;
    uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) +
                                                ((r.t0 + tok) * p.Hq + head * (int64_t)p.G + (at_row - tok * p.G)) * p.D + W * lane);
    using TO = typename std::conditional<BF, __nv_bfloat16, __half>::type;
#pragma unroll
    for (int e = 0; e < W; e += 2)
        if (W * lane + e < p.D) to[e / 2] = pack_pair<TO>(sum[e] * inv, sum[e + 1] * inv);
}

int log2_of(int32_t n) {
    int s = 0;
    while (1 << s < n) ++s;
    return s;
}

// How a call is cut: tiles of rows, parts of keys.
struct Plan8 {
    int mt, dp, tiles, parts, part_len;
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
    c.units = B * c.tiles * kv_heads;
    int64_t blocks = ceil_div(max_len, kKvBlock);
    if (window > 0) {
        const int64_t seen = ceil_div(window + 16 * c.mt, kKvBlock) + 1 + ceil_div(sinks, kKvBlock);
        blocks = std::min(blocks, seen);
    }
    // parts: about six rounds of the CTAs that the machine holds, so that uneven lengths
    // even out, but no fewer than four blocks a warp
    const int64_t want = ceil_div(152 * 3 * 6, c.units);
    c.part_len = (int)std::max<int64_t>(ceil_div(blocks, std::max<int64_t>(want, 1)), 4 * kWarps);
    c.parts = (int)std::max<int64_t>(1, ceil_div(blocks, c.part_len));
    c.bytes = c.parts == 1 ? 0 : (size_t)c.units * c.parts * 16 * c.mt * (c.dp + 2) * 4;
    return c;
}

template <int DP, int MT, bool BF>
cudaError_t attn8_launch(const Attn8Params &p, const Plan8 &c, cudaStream_t st) {
    using C = Cfg8<DP, MT>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)attn8_kernel<DP, MT, BF>, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.units * c.parts), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t k = cudaLaunchKernelEx(&cfg, attn8_kernel<DP, MT, BF>, p);
    if (k != cudaSuccess || c.parts == 1) return k;
    cfg.gridDim = dim3((unsigned)(c.units * C::kRows / kWarps), 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn8_join_kernel<DP, MT, BF>, p);
}

template <bool BF>
cudaError_t attn8_launch_type(const Attn8Params &p, const Plan8 &c, cudaStream_t st) {
    if (c.dp == 64) return c.mt == 1 ? attn8_launch<64, 1, BF>(p, c, st) : attn8_launch<64, 2, BF>(p, c, st);
    if (c.dp == 128) return c.mt == 1 ? attn8_launch<128, 1, BF>(p, c, st) : attn8_launch<128, 2, BF>(p, c, st);
    return attn8_launch<256, 1, BF>(p, c, st);
}

}  // namespace

size_t attention_kv8_workspace(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t max_len,
                               int64_t max_new, int64_t window, int64_t sinks) {
    return plan_of(B, q_heads, kv_heads, head_dim, max_len, max_new, window, sinks).bytes;
}

cudaError_t launch_attention_kv8(const void *q, int32_t q_type, int64_t ld, const w4_kv8_cache &c, const int32_t *table,
                                 int64_t width, const int32_t *ctx_len, const int32_t *cu_new, int64_t B, int64_t T,
                                 int32_t q_heads, float scale, int64_t max_len, int64_t max_new, int64_t window,
                                 int64_t sinks, void *out, void *workspace, cudaStream_t st) {
    const Plan8 plan = plan_of(B, q_heads, c.heads, c.head_dim, max_len, max_new, window, sinks);
    if (plan.units * plan.parts > 0x7FFFFFFF || plan.units * 32 > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    Attn8Params p = {};
    p.q = q; p.out = out; p.k = c.k; p.v = c.v; p.ks = c.k_scale; p.vs = c.v_scale;
    p.table = table; p.ctx_len = ctx_len; p.cu_new = cu_new;
    p.ld = ld; p.width = width; p.T = T; p.pages = c.pages;
    p.page_stride = c.page_stride; p.token_stride = c.token_stride; p.head_stride = c.head_stride;
    p.B = (int)B; p.Hq = q_heads; p.Hkv = c.heads; p.G = q_heads / c.heads; p.D = c.head_dim;
    p.page_shift = log2_of(c.page_size);
    p.window = (int)window; p.sinks = (int)sinks;
    p.tiles = plan.tiles; p.parts = plan.parts; p.part_len = plan.part_len;
    p.max_new = (int)max_new;
    p.scale_log2 = scale * kLog2e;
    const size_t slots = (size_t)plan.units * plan.parts * 16 * plan.mt;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = workspace ? reinterpret_cast<float2 *>(p.part_o + slots * plan.dp) : nullptr;
    return q_type == W4_BF16 ? attn8_launch_type<true>(p, plan, st) : attn8_launch_type<false>(p, plan, st);
}

}  // namespace w4
