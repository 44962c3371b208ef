// mxfp4.cu -- microscaled 4-bit floating point: the quantizer and its inverse,
// the decode product (M <= 16) and the tcgen05 product of two 4-bit matrices.
//
// Format (OCP Microscaling Formats v1.0): e2m1 codes s|ee|m of the values
// 0, .5, 1, 1.5, 2, 3, 4, 6, one e8m0 scale 2^(s - 127) for 32 of a row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "smem_limit.h"
#include "tcgen05.cuh"
#include "w4.h"

namespace w4 {
namespace {

// ---------------------------------------------------------------- element access

template <int TY>
W4_DEV float load_el(const void *x, int64_t i) {
    if constexpr (TY == W4_F32) return __ldg(static_cast<const float *>(x) + i);
    else if constexpr (TY == W4_BF16) return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(x) + i) << 16);
    else return __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t *>(x) + i)));
}

// 8 consecutive elements, 16-byte aligned.
template <int TY>
W4_DEV void load_el8(const void *x, int64_t i, float (&v)[8]) {
    if constexpr (TY == W4_F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (TY == W4_BF16) {
                v[2 * e] = __uint_as_float(w[e] << 16);
                v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                v[2 * e] = f.x;
                v[2 * e + 1] = f.y;
            }
        }
    }
}

W4_DEV void store_el(void *y, int ty, int64_t i, float v) {
    if (ty == W4_F32) static_cast<float *>(y)[i] = v;
    else if (ty == W4_BF16) static_cast<uint16_t *>(y)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else static_cast<uint16_t *>(y)[i] = __half_as_ushort(__float2half_rn(v));
}

// 2^(s - 127) in f32 (s = 0: a subnormal; 255: NaN).
W4_DEV float e8m0_f32(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// 8 values times f to 8 e2m1 codes (v[0] in bits 0-3), to nearest, ties to the even code, saturated at 6.
W4_DEV uint32_t cvt_e2m1x8(const float (&v)[8], float f) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f), "f"(v[6] * f),
          "f"(v[7] * f));
    return r;
}

// ---------------------------------------------------------------- quantizer

// Four lanes share a block of 32, 8 values each: the maximum takes two
// shuffles, and a lane's 8 codes leave as one word.  floor(log2(max)) is the
// exponent field of the maximum, and x / 2^e a product with an exact power of
// two, so the codes are those of the definition bit for bit.  Bound by memory:
// one read of x, 17 bytes written for 32 values; 13312 x 2048 in f32: 18.5 us, 6.7 TB/s.
// tx = blockDim.x threads walk a row, blockDim.y rows a block.
template <int TY, bool VEC>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const void *__restrict__ x, int64_t R, int64_t K,
                                                             int64_t nb, uint32_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales) {
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = row < R;
    const int64_t groups = nb * 4, steps = (groups + blockDim.x - 1) / blockDim.x;
    for (int64_t i = 0; i < steps; ++i) {
        const int64_t g = i * blockDim.x + threadIdx.x, k = g * 8;
        const bool on = in && g < groups;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on) {
            if (VEC && k + 8 <= K) {
                load_el8<TY>(x, row * K + k, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < K) v[e] = load_el<TY>(x, row * K + k + e);
            }
        }
        // magnitudes order as their bits do, NaN above infinity
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t ef = top >> 23;
        const bool bad = ef == 255;
        const uint32_t s = bad ? 255u : ef > 2 ? ef - 2 : 0u;
        const float inv = __uint_as_float((254u - (bad ? 127u : s)) << 23);  // 2^(127 - s)
        const uint32_t w = bad ? 0u : cvt_e2m1x8(v, inv);
        if (on) {
            codes[row * groups + g] = w;
            if ((threadIdx.x & 3) == 0) scales[row * nb + (g >> 2)] = (uint8_t)s;
        }
    }
}

// 8 codes of a word to the f32 values times s (v[0] from bits 0-3).
W4_DEV void values_e2m1x8(uint32_t w, float s, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
    const uint64_t s2 = f32x2(s, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
        f32x2_split(f32x2_mul(f32x2(f.x, f.y), s2), v[2 * e], v[2 * e + 1]);
    }
}

// One word of codes (8 values) a thread and row, kDeqRows rows at a time: their
// reads are small against what each lets the thread write, so several have to
// be on their way.  13312 x 2048 to bf16: 10.8 us, 6.4 TB/s read and written (one
// row a thread: 12.9 us; that and values put together bit by bit: 15.1 us).  To
// f32: 19.6 us, 6.3 TB/s, with one store of 32 bytes a lane (two of 16 bytes, each
// half of a sector: 29.8 us; one row a thread: 21.2 us).
template <int TY, int kDeqRows>
__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint32_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales, int64_t R,
                                                               int64_t K, int64_t nb, void *__restrict__ y, int vec) {
    const int64_t row0 = (int64_t)blockIdx.x * (blockDim.y * kDeqRows) + threadIdx.y;
    for (int64_t g = threadIdx.x; g * 8 < K; g += blockDim.x) {
        const int64_t k = g * 8;
        uint32_t w[kDeqRows], sc[kDeqRows];
#pragma unroll
        for (int i = 0; i < kDeqRows; ++i) {
            const int64_t row = row0 + i * blockDim.y;
            w[i] = row < R ? __ldcs(codes + row * nb * 4 + g) : 0u;
            sc[i] = row < R ? (uint32_t)__ldg(scales + row * nb + (g >> 2)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kDeqRows; ++i) {
            const int64_t row = row0 + i * blockDim.y;
            if (row >= R) break;
            const float s = e8m0_f32(sc[i]);
            float v[8];
            values_e2m1x8(w[i], s, v);
            if (vec) {
                if constexpr (TY == W4_F32) {
                    float *d = static_cast<float *>(y) + row * K + k;
                    if (vec == 2) {
                        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(v[0]),
                                     "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                                     : "memory");
                    } else {
                        reinterpret_cast<float4 *>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
                        reinterpret_cast<float4 *>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                } else {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (TY == W4_BF16) {
                            __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                            o[e] = *reinterpret_cast<uint32_t *>(&h);
                        } else {
                            __half2 h = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                            o[e] = *reinterpret_cast<uint32_t *>(&h);
                        }
                    }
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(y) + row * K + k) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < K) store_el(y, TY, row * K + k + e, v[e]);
            }
        }
    }
}

// Threads along a row: a power of two between 4 and 256 that covers its groups if it can.
dim3 row_block(int64_t groups) {
    unsigned tx = 4;
    while (tx < 256 && tx < groups) tx *= 2;
    return dim3(tx, 256 / tx);
}

// ---------------------------------------------------------------- decode product (M <= 16)

constexpr int kDecWarps = 8;

struct DecodeParams {
    const uint16_t *x;   // bf16 [M][K], or
    const uint8_t *xq, *sx;  // MXFP4 [M][K]
    const uint8_t *w, *sw;
    void *y;
    int64_t N, K, nb;
    int M, y_type, pdl;
};

// Decoded values are kept as 2^-kDown of what they stand for: bf16 then holds every code
// under every scale exactly (from 2^-128, an eighth of which is a subnormal, to 6 * 2^127,
// which it could not hold itself); the sums are put right when they are stored.
constexpr uint32_t kDown = 3;

// 8 codes of a word -> 4 bf16 pairs (codes i and i + 4) times 2^(s - 127 - kDown).
// s|ee|m as the top bits of a bf16 is the value times 2^-126, so the factor is
// 2^(s - 1 - kDown) = fa * fb, both exact.  One bf16 holds it up to s = kOneFactor (scales
// up to 16): ONE then says that fb is 1 throughout the warp.
constexpr uint32_t kOneFactor = 128 + kDown;
template <bool ONE>
W4_DEV void decode8(uint32_t w, uint32_t fa, uint32_t fb, uint32_t (&o)[4]) {
    const uint32_t e[4] = {w << 6, w << 2, w >> 2, w >> 6}, g[4] = {w << 12, w << 8, w << 4, w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = (e[i] & 0x01C001C0u) | (g[i] & 0x80008000u);
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(v), "r"(fa));
        if constexpr (!ONE) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(fb));
    }
}

// fa and fb of a scale byte, each in both halves; NaN for s = 255.
W4_DEV void scale_pair(uint32_t s, uint32_t &fa, uint32_t &fb) {
    const uint32_t a = min(s, kOneFactor);  // 2^(a - 1 - kDown)
    fa = ((a + 126 - kDown) << 7) * 0x10001u;
    fb = (s == 255 ? 0x7FC0u : (127 + s - a) << 7) * 0x10001u;
}

W4_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes that are read once: not kept in L1.
W4_DEV uint4 ldg_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

W4_DEV uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// 8 bf16 of x at [m][k]; zeros past K.
W4_DEV uint4 load_x8(const DecodeParams &p, int m, int64_t k, bool vec) {
    const uint16_t *at = p.x + m * p.K + k;
    if (vec && k + 8 <= p.K) return __ldg(reinterpret_cast<const uint4 *>(at));
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        e[j] = (k + 2 * j < p.K ? (uint32_t)__ldg(at + 2 * j) : 0u) |
               (k + 2 * j + 1 < p.K ? (uint32_t)__ldg(at + 2 * j + 1) << 16 : 0u);
    return make_uint4(e[0], e[1], e[2], e[3]);
}

// 8 values in order -> the pairs (i, i + 4) of decode8.
W4_DEV uint4 pairs_x8(const uint4 &v) {
    return make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
}

// y = x W^T for up to 16 rows of x.  A block takes RT * 16 rows of W, its warps
// take turns along K in chunks of 128 columns: the four lanes of a row read 64
// contiguous bytes, a whole scale block each, and the weights are the A
// operand of mma.sync with a column order of their own (a sum does not mind).
// A chunk of x belongs to one warp of the block, so its fragments come straight
// from memory, no staging.  Several chunks of weights are requested before the
// first value of x, and before the wait for the kernel in front under PDL; a
// chunk's registers are filled again as soon as it has been multiplied, and the
// next x is fetched before.  Where row tiles are few, the blocks of a cluster
// share K and the first adds their sums in order.
// Bound by the instructions that decode (2.5 for a weight), their fetch and latency.
// With W from memory, for one row of x and for 13: 13312 x 2048 7.7 and 10.2 us, 2048 x
// 13312 10.4 and 14.0, 2048 x 2048 3.5 and 4.6 (a launch and one round of latency).  With
// W in L2: 6.5 and 9.4, 9.1 and 12.7, and 3.0; there one block a tile and batch after batch
// took 13.3 and 23.3 for 2048 x 13312, and x staged in shared memory first 18.6 for 13 rows
// of 13312 x 2048.  Three row tiles by 16 columns spill 11 registers of the 128 that
// two blocks an SM leave.
// RT: row tiles of a warp; XT: column tiles of 8 activation rows.
template <int RT, int XT, bool A4>
__global__ void __launch_bounds__(32 * kDecWarps, 2) mxfp4_decode_kernel(const DecodeParams p) {
    constexpr int kPer = RT == 1 ? 4 : 2;  // chunks of a warp in flight
    constexpr int kCols = 8 * XT, kRowsB = 16 * RT;
    constexpr float kBack = A4 ? (float)(1 << 2 * kDown) : (float)(1 << kDown);
    __shared__ float red[kDecWarps * kCols * kRowsB];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = lane & 3, r = lane >> 2;
    const int64_t n0 = (int64_t)blockIdx.x * kRowsB;
    const int chunks = (int)ceil_div(p.K, 128), nb = (int)p.nb;
    const bool vec = p.K % 8 == 0;
    constexpr bool kAhead = RT == 1 && (XT == 1 || A4);  // x of the next chunk under way: where registers allow
    constexpr bool kRing = RT * XT < 6;          // a chunk of W requested as soon as its registers are free: likewise
    float acc[RT][XT][4] = {};

    // the lane's 32 columns of x in a chunk: as they lie in memory, then 4 words of 8 per row
    struct RawX {
        uint4 v[XT][A4 ? 1 : 4];
        uint32_t s[XT];
    };
    auto fetch_x = [&](int blk, RawX &raw) {
#pragma unroll
        for (int xt = 0; xt < XT; ++xt) {
            const int m = 8 * xt + r;
            if constexpr (A4) {
                const bool on = m < p.M && blk < nb;
                raw.v[xt][0] = on ? __ldg(reinterpret_cast<const uint4 *>(p.xq) + m * p.nb + blk) : make_uint4(0, 0, 0, 0);
                raw.s[xt] = on ? (uint32_t)__ldg(p.sx + m * p.nb + blk) : 127u;
            } else {
#pragma unroll
                for (int word = 0; word < 4; ++word)
                    raw.v[xt][word] = m < p.M ? load_x8(p, m, (int64_t)blk * 32 + 8 * word, vec) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    auto ready_x = [&](const RawX &raw, uint4 (&xv)[XT][4]) {
#pragma unroll
        for (int xt = 0; xt < XT; ++xt) {
            uint32_t fa = 0, fb = 0;
            if constexpr (A4) scale_pair(raw.s[xt], fa, fb);
#pragma unroll
            for (int word = 0; word < 4; ++word) {
                if constexpr (A4) {
                    uint32_t o[4];
                    decode8<false>(word_of(raw.v[xt][0], word), fa, fb, o);
                    xv[xt][word] = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    xv[xt][word] = pairs_x8(raw.v[xt][word]);
                }
            }
        }
    };
    auto product = [&](auto one, const uint4 (&xv)[XT][4], const uint4 (&wv)[RT][2], const uint32_t (&sv)[RT][2]) {
        constexpr bool kOne = decltype(one)::value;
        uint32_t fa[RT][2], fb[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) scale_pair(sv[t][hh], fa[t][hh], fb[t][hh]);
#pragma unroll
        for (int word = 0; word < 4; ++word)
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                uint32_t a[4], b[4];
                decode8<kOne>(word_of(wv[t][0], word), fa[t][0], fb[t][0], a);
                decode8<kOne>(word_of(wv[t][1], word), fa[t][1], fb[t][1], b);
                const uint32_t f0[4] = {a[0], b[0], a[1], b[1]}, f1[4] = {a[2], b[2], a[3], b[3]};
#pragma unroll
                for (int xt = 0; xt < XT; ++xt) {
                    mma_bf16(acc[t][xt], f0, xv[xt][word].x, xv[xt][word].y);
                    mma_bf16(acc[t][xt], f1, xv[xt][word].z, xv[xt][word].w);
                }
            }
    };

    uint4 wv[kPer][RT][2];
    uint32_t sv[kPer][RT][2];
    auto fetch_w = [&](int chunk, uint4 (&w)[RT][2], uint32_t (&sc)[RT][2]) {
        const int blk = chunk * 4 + q;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int64_t n = n0 + 16 * t + 8 * hh + r;
                const bool on = n < p.N && blk < nb;
                w[t][hh] = on ? ldg_stream(reinterpret_cast<const uint4 *>(p.w) + n * p.nb + blk) : make_uint4(0, 0, 0, 0);
                sc[t][hh] = on ? (uint32_t)__ldg(p.sw + n * p.nb + blk) : 127u;
            }
    };
    constexpr bool kParts = RT < 3;  // may share K within a cluster
    const int step = kParts ? kDecWarps * (int)gridDim.y : kDecWarps;
    const int first = kParts ? (int)blockIdx.y * kDecWarps + warp : warp;
    auto fetch_all = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kPer; ++c) fetch_w(c0 + c * step, wv[c], sv[c]);
    };
    bool waited = !p.pdl;
    auto wait_front = [&] {
        if (waited) return;
        griddep_launch_dependents();
        griddep_wait();
        waited = true;
    };
    RawX raw[kAhead ? 2 : 1];
    if constexpr (kRing) {
        fetch_all(first);
        wait_front();
        if (kAhead && first < chunks) fetch_x(first * 4 + q, raw[0]);
    }
    auto chunk_product = [&](auto one, int at, int c) {
        uint4 xv[XT][4];
        if constexpr (kAhead) {
            if (at + step < chunks) fetch_x((at + step) * 4 + q, raw[(c + 1) & 1]);
        } else {
            fetch_x(at * 4 + q, raw[0]);
        }
        ready_x(raw[kAhead ? c & 1 : 0], xv);
        product(one, xv, wv[c], sv[c]);
    };
    for (int c0 = first; c0 < chunks; c0 += kPer * step) {
        if constexpr (kRing) {
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const int at = c0 + c * step;
                if (at >= chunks) break;
                uint32_t most = 0;
#pragma unroll
                for (int t = 0; t < RT; ++t) most = max(most, max(sv[c][t][0], sv[c][t][1]));
                if (__all_sync(0xffffffffu, most <= kOneFactor)) chunk_product(std::true_type{}, at, c);
                else chunk_product(std::false_type{}, at, c);
                if (at + kPer * step < chunks) fetch_w(at + kPer * step, wv[c], sv[c]);
            }
        } else {
            fetch_all(c0);
            wait_front();
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < kPer; ++c)
#pragma unroll
                for (int t = 0; t < RT; ++t) most = max(most, max(sv[c][t][0], sv[c][t][1]));
            auto batch = [&](auto one) {
#pragma unroll
                for (int c = 0; c < kPer; ++c)
                    if (c0 + c * step < chunks) chunk_product(one, c0 + c * step, c);
            };
            if (__all_sync(0xffffffffu, most <= kOneFactor)) batch(std::true_type{});
            else batch(std::false_type{});
        }
    }
    wait_front();
    // the warps' sums in a fixed order: [warp][column][row of W]
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int xt = 0; xt < XT; ++xt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(warp * kCols + 8 * xt + 2 * q + (e & 1)) * kRowsB + 16 * t + r + 8 * (e >> 1)] = acc[t][xt][e];
    __syncthreads();
    if (kParts && gridDim.y > 1) {  // the blocks of a cluster: each its own sum, then the first adds them in their order
        for (int i = tid; i < kCols * kRowsB; i += 32 * kDecWarps) {
            float s = 0.0f;
#pragma unroll
            for (int wq = 0; wq < kDecWarps; ++wq) s += red[wq * kCols * kRowsB + i];
            red[i] = s;  // read by this thread alone
        }
        __syncwarp();
        cluster_sync();
        if (blockIdx.y == 0)
            for (int i = tid; i < p.M * kRowsB; i += 32 * kDecWarps) {
                const int m = i / kRowsB, n = i - m * kRowsB;
                float s = red[i];
                for (uint32_t k = 1; k < gridDim.y; ++k) s += __uint_as_float(dsmem_ld_u32(dsmem_map(&red[i], k)));
                if (n0 + n < p.N) store_el(p.y, p.y_type, m * p.N + n0 + n, s * kBack);
            }
        __syncwarp();
        cluster_sync();  // the others' memory stays until it has been read
        return;
    }
    for (int i = tid; i < p.M * kRowsB; i += 32 * kDecWarps) {
        const int m = i / kRowsB, n = i - m * kRowsB;
        float s = 0.0f;
#pragma unroll
        for (int wq = 0; wq < kDecWarps; ++wq) s += red[(wq * kCols + m) * kRowsB + n];
        if (n0 + n < p.N) store_el(p.y, p.y_type, m * p.N + n0 + n, s * kBack);
    }
}

template <int RT, int XT, bool A4>
cudaError_t decode_launch(const DecodeParams &p, int parts, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div(p.N, 16 * RT), (unsigned)parts);
    cfg.blockDim = dim3(32 * kDecWarps);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (p.pdl) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (parts > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = 1;
        at[n].val.clusterDim.y = (unsigned)parts;
        at[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, mxfp4_decode_kernel<RT, XT, A4>, p);
}

// Clusters of `parts` blocks that run at once on the current device, two blocks an SM: a
// cluster lies within one GPC, so they are fewer than the SMs' places (GB300 with 152 SMs:
// 152 of 2, 74 of 4, 36 of 8).  One more waits for a whole cluster to end: 2400 x 13312 in 75
// clusters of 4 takes 15.8 us for one row, 2368 x 13312 in 74 10.7.  Asked of one kernel for
// all, so that the split does not depend on M.
int64_t cluster_room(int parts) {
    static std::atomic<int> known[64][3];  // [device][parts 2, 4, 8], one more than the number
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::atomic<int> &slot = known[dev][parts == 2 ? 0 : parts == 4 ? 1 : 2];
    int n = slot.load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = (unsigned)parts;
    at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, (unsigned)parts);
    cfg.blockDim = dim3(32 * kDecWarps);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, mxfp4_decode_kernel<2, 2, false>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    slot.store(n + 1, std::memory_order_relaxed);
    return n;
}

// Blocks that share K where those of RT row tiles are few: while all of them run at once and
// each warp keeps two chunks of 128 columns, or one where there is still no more than a block
// an SM (one row, W from memory: 512 x 4096 3.6 us in four parts, 4.0 in two, 4.7 undivided;
// 2048 x 8192, a tile a block, 7.3 in two, 9.1 undivided; W in L2, a chunk a warp: 2048 x 2048
// 3.6 in two, 3.0 undivided).
int parts_of(int RT, int64_t N, int64_t K) {
    const int64_t blocks = ceil_div(N, 16 * RT), sms = 152;
    int parts = 1;
    while (parts < 8 && blocks * parts * 2 <= 2 * sms &&
           K >= (int64_t)128 * kDecWarps * parts * 2 * (blocks * parts * 2 <= sms ? 1 : 2) &&
           blocks <= cluster_room(parts * 2))
        parts *= 2;
    return parts;
}

template <int XT, bool A4>
cudaError_t decode_rows(const DecodeParams &p, cudaStream_t st) {
    // All in us with W from memory.  One tile a block up to a block an SM; with more, two tiles
    // share what a warp fetches of x (M = 13, one tile / two: 2560 x 4096 9.1 / 8.2).  Two as well where one tile in its
    // parts takes more than a block an SM and two tiles get more parts (one / two: 2048 x 8192
    // 7.3 / 6.8 for one row and 10.3 / 9.0 for 13, 1248 x 8192 6.9 / 6.2 and 9.7 / 8.6, 2368 x 13312
    // 10.6 / 10.7 and 15.8 / 14.4; where they do not, 2400 x 8192 7.5 / 8.6 and 10.6 / 11.1, 2048 x
    // 6144 6.1 / 6.9 and 8.5 / 8.8).  Three beyond two blocks an SM of two: 9728 x 2048 7.7 with
    // two, 9.9 with three; 13312 x 2048 13.2 and 10.2.
    const int64_t tiles = ceil_div(p.N, 16), sms = 152;
    if (tiles > 4 * sms) return decode_launch<3, XT, A4>(p, 1, st);
    const int one = parts_of(1, p.N, p.K), two = parts_of(2, p.N, p.K);
    if (tiles > sms || (tiles * one > sms && two > one)) return decode_launch<2, XT, A4>(p, two, st);
    return decode_launch<1, XT, A4>(p, one, st);
}

// ---------------------------------------------------------------- 4-bit product (tcgen05)
//
// Persistent: a CTA an SM walks the 128 (activation rows m) x BN (channels n)
// tiles of y, m fastest.  A stage is 256 columns: 128 bytes of codes a row,
// 128-byte swizzle, and 8 scale bytes a row.
//   warp 0       TMA producer of the code tiles;
//   warp 1       allocates TMEM; per stage copies the scales to TMEM
//                (tcgen05.cp) and issues 4 MMAs of 64 columns (kind::mxf4);
//   warps 2-5    read the scale bytes ahead (row-major in memory) and lay them
//                out in shared memory as tcgen05 wants them;
//   warps 6-13   epilogue: TMEM -> registers -> 128-byte rows in shared memory ->
//                TMA store, each warp for its own 32 rows and half of the columns (all of 64)
//                (y rows that TMA cannot address go out element by element).
// 2048 x 13312 x 2048 to bf16: 33.5 us, 3.3 PFLOP/s (4.25 in the loop over K).  A
// stage takes 0.55 us: the products alone 0.29, the copies alone 0.51; the scale
// reads took 0.58 before one read served two stages.  Rows of y that TMA cannot
// address (not whole 16 bytes) cost far more, a value and a row a lane: N = 13311
// 280 us in bf16 and 179 in f32 (41.7 by TMA).

constexpr int kGM = 128;
constexpr int kSfWarps = 4, kOutWarps = 8;
constexpr int kGThreads = 64 + 32 * (kSfWarps + kOutWarps);
constexpr int kOutBuf = 32 * 128;  // 32 rows of 128 bytes, two for each epilogue warp

template <int BN>
struct GCfg {
    static constexpr int kA = kGM * 128, kB = BN * 128;
    static constexpr int kRowTilesB = (BN + 127) / 128;
    static constexpr int kSfA = 1024, kSfB = 1024 * kRowTilesB;  // two 512-byte atoms (128 rows x 4 scales) a row tile
    static constexpr int kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = BN == 256 ? 3 : BN == 128 ? 4 : 6;
    static constexpr int kOut = 2 * kOutWarps * kOutBuf;
    static constexpr int kSmem = kStages * kStage + kOut + 1024;
    // TMEM: the accumulators, then per stage 8 columns of A's scales and 8 per row tile of B's
    static constexpr int kSfCols = 8 + 8 * kRowTilesB;
    static constexpr int kAccs = BN == 256 ? 1 : 2;
    static_assert(kAccs * BN + kStages * kSfCols <= 512, "TMEM");
    static_assert(kSmem <= 232448, "shared memory");
};

struct MxGemmParams {
    CUtensorMap xmap, wmap;  // codes as bytes [rows][nb * 16], box {128, 128 | BN}
    CUtensorMap ymap;        // y [M][N], box {128 bytes, 32 rows}
    const uint8_t *sw, *sx;
    void *y;
    uint32_t *status;
    int64_t N, M, nb;
    int y_tma, nk, ntm, ntiles;
    int pairs;  // the scales of two stages come as 16 aligned bytes of a row
};

struct GCtl {
    uint64_t full[6], sf_full[6], empty[6];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drained;  // after an abort: all products are through
    uint32_t tmem_base;
    int abort;
    int begun;  // fills of the ring
};

// 8 scale bytes of a row's blocks b0 .. b0 + 7; 127 (a scale of 1, over codes of 0) past its end.
W4_DEV uint2 load_scales8(const uint8_t *s, int64_t row, int64_t rows, int64_t nb, int64_t b0) {
    uint2 v = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (row >= rows) return v;
    const uint8_t *at = s + row * nb + b0;
    if (b0 + 8 <= nb && (reinterpret_cast<uintptr_t>(at) & 7) == 0) return __ldg(reinterpret_cast<const uint2 *>(at));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= (b0 + i < nb ? (uint32_t)__ldg(at + i) : 127u) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

template <int YT>
W4_DEV uint32_t pack_y(float a, float b) {
    if constexpr (YT == W4_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

template <int BN, int YT>
__global__ void __launch_bounds__(kGThreads, 1) mxfp4_gemm_kernel(const __grid_constant__ MxGemmParams p) {
    using C = GCfg<BN>;
    extern __shared__ __align__(1024) uint8_t smem_g[];
    uint8_t *tiles = smem_g;  // [stage] A codes, B codes, A scales, B scales
    uint8_t *outs = smem_g + C::kStages * C::kStage;
    GCtl *ctl = reinterpret_cast<GCtl *>(outs + C::kOut);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mine = blockIdx.x < (unsigned)p.ntiles ? (p.ntiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    auto tile_of = [&](int i, int64_t &m0, int64_t &n0) {
        const int t = (int)blockIdx.x + i * (int)gridDim.x;
        m0 = (int64_t)(t % p.ntm) * kGM;
        n0 = (int64_t)(t / p.ntm) * BN;
    };
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->sf_full[s], kSfWarps);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->acc_full[i], 1);
            mbar_init(&ctl->acc_empty[i], BN == 64 ? kOutWarps / 2 : kOutWarps);
        }
        mbar_init(&ctl->drained, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&ctl->tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    int *abort = &ctl->abort;

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int s = 0, round = 0;  // stage, times around the ring
            for (int i = 0; i < mine && ok; ++i) {
                int64_t m0, n0;
                tile_of(i, m0, n0);
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (round > 0) ok = wait_or_abort(&ctl->empty[s], (round - 1) & 1, abort, p.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&ctl->full[s], C::kA + C::kB);
                    tma_load_2d(tiles + s * C::kStage, &p.xmap, kb * 128, (int)m0, &ctl->full[s]);
                    tma_load_2d(tiles + s * C::kStage + C::kA, &p.wmap, kb * 128, (int)n0, &ctl->full[s]);
                    if (++s == C::kStages) s = 0, ++round;
                }
            }
            ctl->begun = round * C::kStages + s;
        }
        __syncwarp();
    } else if (warp == 1) {
        // the whole warp walks, one lane issues
        const uint32_t lead = elect_lead();
        const uint64_t a_desc = smem_desc_sw128(smem_u32(tiles)), b_desc = smem_desc_sw128(smem_u32(tiles + C::kA)),
                       sf_desc = smem_desc_rows16(smem_u32(tiles + C::kA + C::kB));
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) {
            ok = ok && wait_warp(bar, parity, abort, p.status);
        };
        int s = 0, round = 0;
        for (int i = 0; i < mine && ok; ++i) {
            const int a = i % C::kAccs;
            if (i >= C::kAccs) wait(&ctl->acc_empty[a], ((i / C::kAccs) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + (uint32_t)(BN * a);
            for (int kb = 0; kb < p.nk; ++kb) {
                wait(&ctl->full[s], round & 1);
                wait(&ctl->sf_full[s], round & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t off = (uint32_t)(s * C::kStage);
                const uint32_t ta = tmem + (uint32_t)(C::kAccs * BN + s * C::kSfCols), tb = ta + 8;
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 128 columns: one atom of scales a row tile
                    tmem_cp_sf_lead(ta + 4 * c, desc_at(sf_desc, off + 512 * c), lead);
#pragma unroll
                    for (int rt = 0; rt < C::kRowTilesB; ++rt)
                        tmem_cp_sf_lead(tb + 4 * (c * C::kRowTilesB + rt),
                                        desc_at(sf_desc, off + C::kSfA + 512 * (c * C::kRowTilesB + rt)), lead);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)  // 64 columns (32 bytes) each
                    umma_mxf4_lead(acc, desc_at(a_desc, off + 32 * j), desc_at(b_desc, off + 32 * j),
                                   idesc_mxf4(kGM, BN, 2 * (j & 1)), ta + 4 * (j >> 1), tb + 4 * C::kRowTilesB * (j >> 1),
                                   (kb > 0 || j > 0) ? 1u : 0u, lead);
                umma_commit_lead(&ctl->empty[s], lead);
                if (++s == C::kStages) s = 0, ++round;
            }
            if (ok) umma_commit_lead(&ctl->acc_full[a], lead);
        }
        __syncwarp();
    } else if (warp < 2 + kSfWarps) {
        // thread = row of each 128-row tile; scales of kAhead stages ahead in registers
        const int row = tid - 64;
        constexpr int kAhead = 4;
        uint2 va[kAhead], vb[kAhead][C::kRowTilesB];
        int lt = 0, lk = 0;  // the next stage to read: tile, block of columns
        int64_t m0 = 0, n0 = 0;
        if (mine > 0) tile_of(0, m0, n0);
        // Two stages at a time, in one read of a row where that is aligned (each read of 32 rows
        // is 32 sectors, and their number is what the scales cost).
        auto load1 = [&](uint2 &a, uint2 (&b)[C::kRowTilesB]) {
            if (lt >= mine) return;
            a = load_scales8(p.sx, m0 + row, p.M, p.nb, (int64_t)lk * 8);
#pragma unroll
            for (int rt = 0; rt < C::kRowTilesB; ++rt)
                if (rt * 128 + row < BN) b[rt] = load_scales8(p.sw, n0 + rt * 128 + row, p.N, p.nb, (int64_t)lk * 8);
            if (++lk == p.nk) {
                lk = 0;
                if (++lt < mine) tile_of(lt, m0, n0);
            }
        };
        auto load2 = [&](int i) {
            if (!p.pairs) {
                load1(va[i], vb[i]);
                load1(va[i + 1], vb[i + 1]);
                return;
            }
            if (lt >= mine) return;
            auto read = [&](const uint8_t *base, int64_t r, int64_t rows, uint2 &x, uint2 &y) {
                uint4 v = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                if (r < rows) v = __ldg(reinterpret_cast<const uint4 *>(base + r * p.nb + lk * 8));
                x = make_uint2(v.x, v.y);
                y = make_uint2(v.z, v.w);
            };
            read(p.sx, m0 + row, p.M, va[i], va[i + 1]);
#pragma unroll
            for (int rt = 0; rt < C::kRowTilesB; ++rt)
                if (rt * 128 + row < BN) read(p.sw, n0 + rt * 128 + row, p.N, vb[i][rt], vb[i + 1][rt]);
            if ((lk += 2) == p.nk) {
                lk = 0;
                if (++lt < mine) tile_of(lt, m0, n0);
            }
        };
#pragma unroll
        for (int i = 0; i < kAhead; i += 2) load2(i);
        const int at = (row & 31) * 16 + (row >> 5) * 4;
        const int total = mine * p.nk;
        bool ok = true;
        int s = 0, round = 0;
        for (int g0 = 0; g0 < total && ok; g0 += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (g0 + i >= total || !ok) break;
                if (round > 0) ok = wait_warp(&ctl->empty[s], (round - 1) & 1, abort, p.status);
                if (!ok) break;
                uint8_t *sa = tiles + s * C::kStage + C::kA + C::kB, *sb = sa + C::kSfA;
                *reinterpret_cast<uint32_t *>(sa + at) = va[i].x;
                *reinterpret_cast<uint32_t *>(sa + 512 + at) = va[i].y;
#pragma unroll
                for (int rt = 0; rt < C::kRowTilesB; ++rt)
                    if (rt * 128 + row < BN) {
                        *reinterpret_cast<uint32_t *>(sb + 512 * rt + at) = vb[i][rt].x;
                        *reinterpret_cast<uint32_t *>(sb + 512 * (C::kRowTilesB + rt) + at) = vb[i][rt].y;
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->sf_full[s]);
                if (i & 1) load2(i - 1);
                if (++s == C::kStages) s = 0, ++round;
            }
        }
    } else {
        const int q = warp & 3, half = (warp - 2 - kSfWarps) >> 2;  // TMEM lane quadrant, part of the columns
        constexpr int kParts = BN == 64 ? 1 : 2, kHalf = BN / kParts;  // 64 16-bit columns are one whole row of 128 bytes
        const int tiles_here = half < kParts ? mine : 0;
        constexpr int kYB = YT == W4_F32 ? 4 : 2;
        uint8_t *buf = outs + (warp - 2 - kSfWarps) * (2 * kOutBuf);
        int turn = 0;  // of the two buffers
        for (int i = 0; i < tiles_here; ++i) {
            const int a = i % C::kAccs;
            int64_t m0, n0;
            tile_of(i, m0, n0);
            if (!wait_warp(&ctl->acc_full[a], (i / C::kAccs) & 1, abort, p.status)) break;
            tc_fence_after();
            const int64_t mw = m0 + 32 * q, m = mw + lane;
            // The accumulator into registers first (packed where y has 16 bits), so that the next
            // tile's products wait for the reads alone and not for the stores.
            constexpr int kPack = 4 / kYB, kGroup = 32 * kPack;  // columns to a register, to 32 registers
            constexpr int kRegs = kHalf / kPack < 64 ? kHalf / kPack : 64;
#pragma unroll 1
            for (int c0 = 0; c0 < kHalf; c0 += kRegs * kPack) {
                uint32_t v[kRegs];
#pragma unroll
                for (int c = 0; c < kRegs * kPack; c += 32) {
                    uint32_t f[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(BN * a + kHalf * half + c0 + c), f);
#pragma unroll
                    for (int j = 0; j < 32 / kPack; ++j) {
                        if constexpr (kPack == 1) v[c + j] = f[j];
                        else v[c / 2 + j] = pack_y<YT>(__uint_as_float(f[2 * j]), __uint_as_float(f[2 * j + 1]));
                    }
                }
                if (c0 + kRegs * kPack >= kHalf) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->acc_empty[a]);
                }
#pragma unroll
                for (int gr = 0; gr < kRegs / 32; ++gr) {  // 32 registers: 128 bytes of a row
                    const int64_t n = n0 + kHalf * half + c0 + gr * kGroup;
                    const uint32_t *w = v + 32 * gr;
                    if (p.y_tma) {
                        // the store that read this buffer two turns ago is through with it
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        __syncwarp();
                        uint8_t *at = buf + turn * kOutBuf + lane * 128;
#pragma unroll
                        for (int j = 0; j < 8; ++j)  // 16-byte pieces, swizzled as the tensor map says
                            *reinterpret_cast<uint4 *>(at + ((j ^ (lane & 7)) << 4)) =
                                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            if (mw < p.M && n < p.N) tma_store_2d(&p.ymap, buf + turn * kOutBuf, (int)n, (int)mw);
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                        turn ^= 1;
                    } else if (m < p.M) {
#pragma unroll
                        for (int j = 0; j < kGroup; ++j) {
                            if (n + j >= p.N) break;
                            if constexpr (kPack == 1) static_cast<uint32_t *>(p.y)[m * p.N + n + j] = w[j];
                            else static_cast<uint16_t *>(p.y)[m * p.N + n + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
                        }
                    }
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(*reinterpret_cast<volatile int *>(abort), 0)) {  // of all threads alike
        if (tid == 0) drain_ring(ctl->full, C::kStages, ctl->begun);
        if (warp == 1) drain_products(&ctl->drained);
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int BN, int YT>
cudaError_t mx_gemm_launch(const uint8_t *xq, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, void *y,
                           int64_t M, int64_t N, int64_t K, int sms, uint32_t *status, cudaStream_t st) {
    using C = GCfg<BN>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void *>(mxfp4_gemm_kernel<BN, YT>), C::kSmem);
    if (e != cudaSuccess) return e;
    MxGemmParams p = {};
    p.sw = sw; p.sx = sx; p.y = y; p.status = status;
    p.N = N; p.M = M; p.nb = ceil_div(K, 32);
    p.nk = (int)ceil_div(p.nb, 8);
    p.ntm = (int)ceil_div(M, kGM);
    const int64_t tiles = p.ntm * ceil_div(N, BN);
    if (tiles > 0x7FFFFFFF / (int64_t)p.nk) return cudaErrorInvalidConfiguration;
    p.ntiles = (int)tiles;
    p.pairs = p.nb % 16 == 0 && reinterpret_cast<uintptr_t>(sx) % 16 == 0 && reinterpret_cast<uintptr_t>(sw) % 16 == 0;
    const uint64_t strides[1] = {(uint64_t)p.nb * 16};
    const uint64_t wd[2] = {(uint64_t)p.nb * 16, (uint64_t)N}, xd[2] = {(uint64_t)p.nb * 16, (uint64_t)M};
    const uint32_t wb[2] = {128, BN}, xb[2] = {128, kGM};
    if (!encode_tmap(&p.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w, wd, strides, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap(&p.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, xq, xd, strides, xb, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    constexpr int kYB = YT == W4_F32 ? 4 : 2;
    if (N * kYB % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0) {
        const CUtensorMapDataType ty = YT == W4_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : YT == W4_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const uint64_t yd[2] = {(uint64_t)N, (uint64_t)M}, ys[1] = {(uint64_t)N * kYB};
        const uint32_t yb[2] = {128 / kYB, 32};
        if (!encode_tmap(&p.ymap, ty, 2, y, yd, ys, yb, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
        p.y_tma = 1;
    }
    mxfp4_gemm_kernel<BN, YT><<<std::min(p.ntiles, sms), kGThreads, C::kSmem, st>>>(p);
    return cudaGetLastError();
}

template <int YT>
cudaError_t mx_gemm_tiles(const uint8_t *xq, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, void *y, int64_t M,
                          int64_t N, int64_t K, uint32_t *status, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // The width with the least time: rounds of tiles over the SMs, each round as 7, 9 and
    // 15 for 64, 128 and 256 channels (2048 x 13312 x 2048, many rounds: 57, 37 and 34 us;
    // 1024 x 2048 x 2048, two, one and one: 8.2, 6.6 and 8.2; 2048 x 2048 x 2048, four, two
    // and one: 13.0, 9.3 and 8.4).
    const int64_t ntm = ceil_div(M, kGM);
    auto cost = [&](int bn, int64_t c) { return ceil_div(ntm * ceil_div(N, bn), sms) * c; };
    const int64_t c64 = cost(64, 7), c128 = cost(128, 9), c256 = cost(256, 15);
    if (c256 <= c128 && c256 <= c64) return mx_gemm_launch<256, YT>(xq, sx, w, sw, y, M, N, K, sms, status, st);
    if (c128 <= c64) return mx_gemm_launch<128, YT>(xq, sx, w, sw, y, M, N, K, sms, status, st);
    return mx_gemm_launch<64, YT>(xq, sx, w, sw, y, M, N, K, sms, status, st);
}

}  // namespace

cudaError_t launch_quantize_mxfp4(const void *x, int32_t ty, int64_t R, int64_t K, uint8_t *codes, uint8_t *scales,
                                  cudaStream_t st) {
    const int64_t nb = ceil_div(K, 32);
    const dim3 block = row_block(nb * 4);
    const int64_t blocks = ceil_div(R, block.y);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
    const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, block, 0, st>>>(x, R, K, nb, c, scales);
        return cudaGetLastError();
    };
    switch (ty) {
        case W4_F32: return vec ? go(quantize_mxfp4_kernel<W4_F32, true>) : go(quantize_mxfp4_kernel<W4_F32, false>);
        case W4_BF16: return vec ? go(quantize_mxfp4_kernel<W4_BF16, true>) : go(quantize_mxfp4_kernel<W4_BF16, false>);
        default: return vec ? go(quantize_mxfp4_kernel<W4_F16, true>) : go(quantize_mxfp4_kernel<W4_F16, false>);
    }
}

cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K, void *y,
                                    int32_t ty, cudaStream_t st) {
    const int64_t nb = ceil_div(K, 32);
    const dim3 block = row_block(nb * 4);
    // four rows a thread once that still gives every SM (152) two blocks
    const int rows = R >= (int64_t)block.y * 4 * 2 * 152 ? 4 : 1;
    const int64_t blocks = ceil_div(R, block.y * rows);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const uint32_t *c = reinterpret_cast<const uint32_t *>(codes);
    // 8 values at once (1), in f32 by one store of 32 bytes (2), where K and y allow
    const uintptr_t at = reinterpret_cast<uintptr_t>(y);
    const int vec = K % 8 || at % 16 ? 0 : at % 32 ? 1 : 2;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, block, 0, st>>>(c, scales, R, K, nb, y, vec);
        return cudaGetLastError();
    };
    switch (ty) {
        case W4_F32: return rows == 4 ? go(dequantize_mxfp4_kernel<W4_F32, 4>) : go(dequantize_mxfp4_kernel<W4_F32, 1>);
        case W4_BF16: return rows == 4 ? go(dequantize_mxfp4_kernel<W4_BF16, 4>) : go(dequantize_mxfp4_kernel<W4_BF16, 1>);
        default: return rows == 4 ? go(dequantize_mxfp4_kernel<W4_F16, 4>) : go(dequantize_mxfp4_kernel<W4_F16, 1>);
    }
}

cudaError_t launch_mxfp4_decode(const uint16_t *x, const uint8_t *xq, const uint8_t *sx, const uint8_t *w,
                                const uint8_t *sw, void *y, int32_t y_type, int64_t M, int64_t N, int64_t K,
                                uint32_t flags, cudaStream_t st) {
    const int64_t nb = ceil_div(K, 32);
    const size_t yel = y_type == W4_F32 ? 4 : 2;
    for (int64_t m0 = 0; m0 < M; m0 += 16) {
        DecodeParams p = {};
        p.x = x ? x + m0 * K : nullptr;
        p.xq = xq ? xq + m0 * nb * 16 : nullptr;
        p.sx = sx ? sx + m0 * nb : nullptr;
        p.w = w; p.sw = sw;
        p.y = static_cast<uint8_t *>(y) + (size_t)(m0 * N) * yel;
        p.N = N; p.K = K; p.nb = nb;
        p.M = (int)std::min<int64_t>(16, M - m0);
        p.y_type = y_type;
        p.pdl = (flags & W4_FLAG_PDL) && m0 == 0;
        cudaError_t e;
        if (x) e = p.M > 8 ? decode_rows<2, false>(p, st) : decode_rows<1, false>(p, st);
        else e = p.M > 8 ? decode_rows<2, true>(p, st) : decode_rows<1, true>(p, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_mxfp4_gemm(const uint8_t *xq, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, void *y,
                              int32_t y_type, int64_t M, int64_t N, int64_t K, uint32_t *status, cudaStream_t st) {
    switch (y_type) {
        case W4_F32: return mx_gemm_tiles<W4_F32>(xq, sx, w, sw, y, M, N, K, status, st);
        case W4_BF16: return mx_gemm_tiles<W4_BF16>(xq, sx, w, sw, y, M, N, K, status, st);
        default: return mx_gemm_tiles<W4_F16>(xq, sx, w, sw, y, M, N, K, status, st);
    }
}

}  // namespace w4
