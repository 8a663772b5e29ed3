// Addresses inside the paged 4-bit key/value cache, and which pages and slots exist.  Plain
// integer arithmetic shared by the kernels and a host test; offsets into a pool are 64-bit (a
// pool passes 4 GiB at about 2^26 cached tokens of one 128-wide head).
//
// A pool is [layer][page][kv head][page_tokens * d/2 bytes] of codes and the same with d/32
// bytes a token of scales; the block of one (layer, page, kv head) is a slab.  A slab holds
// groups of 16 tokens, each laid out for the matrix-core operands of the attention:
//   key codes    [block of 32 channels][token][16 bytes]: the lanes of one load read 16-byte
//                pieces of consecutive tokens
//   key scales   [token][block]
//   value codes  [h][m < 32][qp][t][d/64 bytes], token 8 qp + 4 h + t, channels (d/32) m + k in
//                half byte k: lane (m, h) of the value operand reads its 8 tokens in one piece
//   value scales [h][block][qp][t]
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// Page id of token slot `pos` of a sequence, or -1: past the table, or a page that is not there.
GDN_HD int kv_page(const int32_t *table, int max_pages, int n_pages, int page_shift, int64_t pos) {
    const int64_t i = pos >> page_shift;
    if (pos < 0 || i >= max_pages) return -1;
    const int32_t id = table[i];
    return id >= 0 && id < n_pages ? id : -1;
}

GDN_HD int64_t kv_slab(int layer, int n_pages, int page, int n_kv_heads, int head) {
    return (int64_t(layer) * n_pages + page) * n_kv_heads + head;
}

// Byte offsets in a slab, for slot t (within the page).
template <int D> struct KvAt {
    static GDN_HD int group_codes(int t) { return (t >> 4) * (8 * D); }
    static GDN_HD int group_scales(int t) { return (t >> 4) * (D / 2); }
    // 4 bytes: channels 8 c .. 8 c + 7 of the key
    static GDN_HD int key(int t, int c) {
        return group_codes(t) + (c >> 2) * 256 + (t & 15) * 16 + (c & 3) * 4;
    }
    static GDN_HD int key_scale(int t, int block) {
        return group_scales(t) + (t & 15) * (D / 32) + block;
    }
    // D/64 bytes: channels (D/32) m .. (D/32) m + D/32 - 1 of the value
    static GDN_HD int value(int t, int m) {
        return group_codes(t) +
               (((((t >> 2) & 1) * 32 + m) * 2 + ((t >> 3) & 1)) * 4 + (t & 3)) * (D / 64);
    }
    static GDN_HD int value_scale(int t, int block) {
        return group_scales(t) + ((((t >> 2) & 1) * (D / 32) + block) * 2 + ((t >> 3) & 1)) * 4 + (t & 3);
    }
};

constexpr int kScaleBias = 127;
constexpr int kScaleMax = 125;     // largest |exponent| of a block scale: 6 * 2^125 is finite
constexpr int kPoison = 255;       // key scale byte of a token that held a NaN or an infinity

// Scale exponent of a block whose largest magnitude has these fp32 bits (finite): two below its
// binary exponent, so it lands in [4, 8) of the 4-bit grid, and one more where it would exceed 7.
// Like every element above 4 it is then off by at most half the grid's step of 2, a fifth of itself at
// 5 (stored as 4), a seventh at 7 (as 6) and beyond (as 8).  Only where e is held at 125 can it be
// clipped further: a magnitude of 2^128 would be a quarter off.
GDN_HD int kv_scale_exp(uint32_t amax_bits) {
    const int e = int(amax_bits >> 23) - 129 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < -kScaleMax ? -kScaleMax : e > kScaleMax ? kScaleMax : e;
}

}  // namespace gdn
