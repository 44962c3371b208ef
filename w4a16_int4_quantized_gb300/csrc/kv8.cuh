// kv8.cuh -- the 8-bit paged cache on the device: scale bytes, and requests in bounds whatever
// the arrays hold.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "w4.h"

namespace w4 {

constexpr int kKvBlock = W4_KV8_BLOCK;  // tokens that share a scale
constexpr int kKvBlockLog = 4;
static_assert(1 << kKvBlockLog == kKvBlock, "");

// Of a page's tokens, a power of two.
inline int log2_of(int32_t n) {
    int s = 0;
    while (1 << s < n) ++s;
    return s;
}

// 2^(s - 127); NaN for 255.
W4_DEV float scale_of(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7FC00000u : s == 0u ? 0x00400000u : s << 23);
}

// Request b: its first new token, their number, the tokens before them (where positions begin, whatever
// the block table has room for), and how many of all the block table has room for.
struct KvRequest {
    int64_t t0;
    int n, ctx, len;
};
W4_DEV KvRequest kv_request(const int32_t *cu_new, const int32_t *ctx_len, int64_t b, int64_t T, int64_t width, int page_shift) {
    KvRequest r;
    const int64_t c0 = max(__ldg(cu_new + b), 0), c1 = min((int64_t)__ldg(cu_new + b + 1), T);
    r.t0 = c0;
    const int64_t top = min(width << page_shift, (int64_t)0x7FFFFF00);
    r.ctx = min(max(__ldg(ctx_len + b), 0), 0x7FFFFF00);
    r.n = (int)max((int64_t)0, min(c1 - c0, (int64_t)0x7FFFFF00 - r.ctx));
    r.len = (int)min((int64_t)r.ctx + r.n, top);
    return r;
}

}  // namespace w4
