// Attention of new tokens over the 4-bit paged cache, causal or under a tree mask (gfx950).
//
// For a row r = (new token i, query head) of a sequence and its kv head, with the visible slots p:
//   out_r = sum_p P_rp V_p / sum_p P_rp,   P_rp = exp2(c q_r.K_p - m_r),   c = scale log2(e),
// one pass over the cached tokens with the running reference m_r and sum.
//
// A wave owns 32 * RT rows of one kv head and walks its share of the slots 32 at a time, alone: no
// LDS and no barrier in the loop, since a 4-bit tile is small enough (1.0625 d bytes a token) that
// every wave may fetch it from the caches by itself.  Both products run on the matrix cores as
// 32 x 32 x 16 with the tokens as rows and the query rows as columns:
//   S^T = K Q^T   (lane (r, h): query row r, tokens 8 (i/4) + 4 h + i%4 of its 16 values i)
//   O^T += V^T P^T
// so a query row lives in two lanes: its maximum is 16 values and one half-wave swap away, m_r
// and the rescaling factor are per-lane scalars, and the P values a lane forms are exactly its share
// of the second product's right operand when the summation index runs over the tokens in that
// order.  The cache holds keys and values in the order these operands want them (kv_layout.h): a
// lane's keys come in 16-byte pieces of one scale block, its values as the 8 tokens of d/32
// channels.  Codes become bf16 two at a time in the conversion instruction, which applies the
// block's scale too; both are exact.  Values need one permute more, as a register pairs two tokens
// of a channel, while a code byte holds two channels of a token.
//
// m_r is the maximum of the slots up to the last time it moved.  It moves when a lane's sum of a
// tile's weights exceeds 2^12, which also catches the first tile: until then the weights are small
// enough for fp32 and bf16 alike, and neither the tile's maximum nor a rescaling of the accumulators
// is needed.  The sum is, anyway.
//
// bf16 rows: P is rounded to bf16 for the second product, the choice that keeps it at one
// matrix-core pass, and the sum is of the rounded P, so that a row one token dominates does not
// show that token's rounding.  Each term is off by 2^-8 of itself at most; over many terms the error
// (relative 2-norm) comes near the rounding of the bf16 output itself, 0.0016, and the two together
// measure 0.0020 to 0.0022.  Up to 16 rows leave half of the columns free: they take what the
// rounding of P left over, at no further product, and the error is the output's rounding alone.
// fp32 rows: q and P are split into three bf16 terms each (exact), K and V are exact in bf16, so
// every product is exact and sums are fp32: three passes, or two for up to 16 rows, which have their
// first two terms side by side in the 32 columns.
//
// What bounds it: decode reads 1.0625 d bytes a slot and kv head, near the rate of a large copy (32
// sequences of 8000 to 40000 slots, 8 heads of 128, 4 query heads each: 809 MB in 164 us a call, its
// join included, 4.9 TB/s; the kernel takes 155 us at the least and 181 in the median of a trace, and
// 5.2 TB/s is what a copy reaches).  fp32 decode with 256 channels (2 x 131072 slots, 143 MB in 47 us a
// call) is a wave's own chain: 8 tiles, one in flight at a time, whose loads, products, exponentials
// and splits follow one another, with the matrix unit busy 31% and the vector unit 30% of the time.
// With two row tiles the vector unit, which unpacks and takes the exponentials, is as busy as the
// matrix unit: four chunks of prompts, 32 / 8 heads of 128, 435 GFLOP in 424 us, 1.03 PFLOP/s, with
// the two issuing 48% and busy 43% of the time at a clock their power lowers from 2.4 to 2.0 GHz and
// further on some cards (494 us); ordering a wave's own instructions so that they overlap saves cycles
// but no time.  Trees of 22 nodes on 32 caches of 2000 to 16000 slots: 157 GFLOP in 250 us, matrix unit
// busy 30%: 132 rows a kv head walk as blocks of 64 + 64 + 4, the last nearly empty, and 768 units of
// unequal length on 512 slots leave an uneven last round.  256 channels and fp32 rows have one row
// tile and unpack for 32 rows at a time: the same products take 449 us as 16 / 4 heads of 256, 1050 in
// fp32 (three planes a product) and 970 in fp32 with 256 channels, where 3 registers spill.
//
// Waves that share rows join their (m, sum, O) in LDS, workgroups through the workspace and a
// second launch.  A poisoned token has a NaN key scale: its score is NaN where it is visible and
// replaced where it is not; its value is finite, so masked weights of 0 stay 0.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "attention_work.h"
#include "kv_internal.h"
#include "mfma_common.h"

namespace gdn {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnThreads = 256;
constexpr float kNoScore = -3.0e38f;  // m_r before the first visible slot
constexpr float kSlack = 4096.f;      // largest sum of a lane's 16 weights before m_r moves

// Where a unit's fragments are: in this many shares from `first` on; one share: it was not cut.
struct Cut {
    int32_t first, count;
};
static_assert(sizeof(Cut) == kCutBytes, "workspace layout");

struct AttnParams {
    const void *q;
    void *out;
    const uint8_t *kc, *ks, *vc, *vs;
    const int32_t *pages, *length, *seq_off;
    const int32_t *parent;  // tree: global parent ids of the schedule image, else null
    float *part_o;          // [share][2][tile rows][D]: fragments of units cut between shares
    float2 *part_ml;        // [share][2][tile rows]
    Cut *cut;               // [layer][sequence][kv head][row_blocks]
    float c;
    int32_t S, H, G, T, n_pages, max_pages, page_shift, layer_begin, n_layers;
    int32_t row_blocks, shares;
    int32_t parts;  // 0: shares of the line; else a unit is cut into this many equal parts
    SparseShape sparse;       // SP kernels: the slots a selection stands for
    const int32_t *selected;  // [layer][token][kv head][top]: table entries, by a selection's first token
};

// One tile of 32 slots as a lane holds it.
template <int D> struct Keys {
    u32x4 c[D / 64];  // blocks 2 j + h of token lane % 32
    uint32_t e[D == 256 ? 2 : 1];
};
template <int D> struct Values {
    uint32_t c[2][D / 32];  // per 16 tokens: 8 tokens x d/32 channels
    uint32_t e[2][2];
};

struct WaveAt {
    const int32_t *table;
    int64_t slab_base;  // slab of page 0 of this layer and head
    int lane, r, h;
    const int32_t *selected;  // SP: the selection, its entries, and the table entry that follows them
    int chosen, full;
};

// Page ids of 64 consecutive table entries, one a lane (-1: not there).  One vector load serves 64
// pages; ids fetched tile by tile through the scalar cache made every tile wait for them, as
// their counter is shared with the LDS reads'.
struct Pages {
    int first, id;
};

// SP: the slots walked are those of the selected pages, one after the other, then the sequence's from
// the last full page's end on.
template <bool SP>
__device__ __forceinline__ void fetch_pages(Pages &g, const AttnParams &P, const WaveAt &w, int tile) {
    g.first = (tile * 32) >> P.page_shift;
    int i = g.first + w.lane, end = P.max_pages;
    if constexpr (SP) {
        if (i < w.chosen) {
            i = w.selected[i];
            end = w.full;  // of the full pages only: a later one would be seen twice
        } else {
            i += w.full - w.chosen;
        }
    }
    const int id = w.table[min(max(i, 0), P.max_pages - 1)];
    g.id = unsigned(i) < unsigned(end) && unsigned(id) < unsigned(P.n_pages) ? id : -1;
}

// Where a tile's two groups of 16 slots are, in tokens from the pool's start, and which of them have
// a page (the others stand at page 0 and are masked).
struct Place {
    int64_t at[2];
    uint32_t there;  // 0xFFFF for the first group, 0xFFFF0000 for the second
};

template <bool SP>
__device__ __forceinline__ Place place_of(Pages &g, const AttnParams &P, const WaveAt &w, int tile) {
    if (((tile * 32 + 16) >> P.page_shift) - g.first >= 64) fetch_pages<SP>(g, P, w, tile);
    Place x;
    x.there = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int slot = tile * 32 + 16 * s;
        const int page = __builtin_amdgcn_readlane(g.id, (slot >> P.page_shift) - g.first);
        const int64_t slab = w.slab_base + int64_t(max(page, 0)) * P.H;
        x.at[s] = (slab << P.page_shift) + (slot & ((1 << P.page_shift) - 1));
        x.there |= page >= 0 ? 0xFFFFu << (16 * s) : 0u;
    }
    return x;
}

// A group's codes start at (first slot) d/2 and its scales at (first slot) d/32 of its pool: slabs
// and groups are whole multiples of them.
template <int D>
__device__ __forceinline__ void load_keys(Keys<D> &t, const AttnParams &P, const WaveAt &w, const Place &x) {
    constexpr int NB = D / 32;
    const int64_t at = w.r < 16 ? x.at[0] : x.at[1];
    const uint8_t *kp = P.kc + at * (D / 2) + (w.r & 15) * 16 + w.h * 256;
    const uint8_t *sp = P.ks + at * NB + (w.r & 15) * NB;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) t.c[j] = *reinterpret_cast<const u32x4 *>(kp + 512 * j);
    if constexpr (D == 64) {
        t.e[0] = *reinterpret_cast<const uint16_t *>(sp);
    } else if constexpr (D == 128) {
        t.e[0] = *reinterpret_cast<const uint32_t *>(sp);
    } else {
        const uint2 y = *reinterpret_cast<const uint2 *>(sp);
        t.e[0] = y.x;
        t.e[1] = y.y;
    }
}

template <int D>
__device__ __forceinline__ void load_values(Values<D> &t, const AttnParams &P, const WaveAt &w, const Place &x) {
    constexpr int NB = D / 32;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint8_t *vp = P.vc + x.at[s] * (D / 2) + (w.h * 32 + w.r) * (D / 8);
        if constexpr (D == 64) {
            const uint2 y = *reinterpret_cast<const uint2 *>(vp);
            t.c[s][0] = y.x;
            t.c[s][1] = y.y;
        } else {
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                const u32x4 y = reinterpret_cast<const u32x4 *>(vp)[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) t.c[s][4 * i + e] = y[e];
            }
        }
        const uint2 y = *reinterpret_cast<const uint2 *>(P.vs + x.at[s] * NB + (w.h * NB + w.r / (32 / NB)) * 8);
        t.e[s][0] = y.x;
        t.e[s][1] = y.y;
    }
}

template <int SEL> __device__ __forceinline__ uint32_t two_of(uint32_t w, float unit) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, SEL));
}

// Eight codes of one scale block as a matrix-core operand.
__device__ __forceinline__ bf16x8 eight_of(uint32_t w, float unit) {
    const u32x4 v = {two_of<0>(w, unit), two_of<1>(w, unit), two_of<2>(w, unit), two_of<3>(w, unit)};
    return __builtin_bit_cast(bf16x8, v);
}

// 2^e of a scale byte: the byte as an fp32 exponent.  The conversion takes a scale's exponent alone,
// so the neighbouring bytes that come along in the sign and the fraction do not matter.
template <int BYTE> __device__ __forceinline__ float unit_at(uint32_t w) {
    return __uint_as_float(BYTE == 3 ? w >> 1 : w << (23 - 8 * BYTE));
}

__device__ __forceinline__ uint32_t low_pair(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_pair(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Value operands of 16 tokens: o[n] holds channel (D/32) r + n of the lane's 8 tokens.
// unit[i]: scale of token i = 4 qp + t.
template <int D>
__device__ __forceinline__ void value_operands(const uint32_t (&v)[D / 32], const float (&unit)[8],
                                               u32x4 (&o)[D / 32]) {
    if constexpr (D == 64) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t a = two_of<0>(v[q], unit[4 * q]), b = two_of<1>(v[q], unit[4 * q + 1]);
            const uint32_t c = two_of<2>(v[q], unit[4 * q + 2]), d = two_of<3>(v[q], unit[4 * q + 3]);
            o[0][2 * q] = low_pair(a, b);
            o[1][2 * q] = high_pair(a, b);
            o[0][2 * q + 1] = low_pair(c, d);
            o[1][2 * q + 1] = high_pair(c, d);
        }
    } else if constexpr (D == 128) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t a0 = two_of<0>(v[p], unit[2 * p]), a1 = two_of<1>(v[p], unit[2 * p]);
            const uint32_t b0 = two_of<2>(v[p], unit[2 * p + 1]), b1 = two_of<3>(v[p], unit[2 * p + 1]);
            o[0][p] = low_pair(a0, b0);
            o[1][p] = high_pair(a0, b0);
            o[2][p] = low_pair(a1, b1);
            o[3][p] = high_pair(a1, b1);
        }
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float ua = unit[2 * p], ub = unit[2 * p + 1];
            const uint32_t va = v[2 * p], vb = v[2 * p + 1];
            const uint32_t a[4] = {two_of<0>(va, ua), two_of<1>(va, ua), two_of<2>(va, ua), two_of<3>(va, ua)};
            const uint32_t b[4] = {two_of<0>(vb, ub), two_of<1>(vb, ub), two_of<2>(vb, ub), two_of<3>(vb, ub)};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                o[2 * y][p] = low_pair(a[y], b[y]);
                o[2 * y + 1][p] = high_pair(a[y], b[y]);
            }
        }
    }
}

// The other half-wave's value of the same row.
__device__ __forceinline__ float other_half(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    // s[0]: lanes 32-63 hold the low half's values; s[1]: lanes 0-31 hold the high half's
    return __uint_as_float((threadIdx.x & 32) ? s[0] : s[1]);
}

// State of a wave's rows.
template <int D, int RT> struct Rows {
    f32x16 o[RT][D / 32];
    float m[RT], l[RT];
};

template <int NG> struct Probs {
    u32x4 p[NG][2];  // per operand and 16 tokens
};

// Lanes 16-31 of x against lanes 0-15 of y, and 48-63 against 32-47.
__device__ __forceinline__ void swap_columns(uint32_t &x, uint32_t &y) {
    const auto s = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = s[0];
    y = s[1];
}

// The value of the same row in the other half of the columns.
__device__ __forceinline__ float other_columns(float v) {
    uint32_t x = __float_as_uint(v), y = x;
    swap_columns(x, y);
    return __uint_as_float((threadIdx.x & 16) ? x : y);
}

// Operands a product takes: NP, the bf16 terms ("planes") of a value, when a row has a column.  fp32
// rows that fill half of the columns (CW = 16) have their first two planes side by side, row r's in
// columns r and 16 + r, and the third in a second operand: two instead of three.  bf16 rows have q in
// both columns, P's rounding in the first and the rest of P in the second: one.  The scores of the
// two columns are added in an exchange that leaves each with half of the row's tokens, so the
// exponentials and the splitting are halved too.  16 / 2 heads, up to two tokens a sequence (kernel,
// us, three / two operands): 52.4 / 43.1 with 256 channels and 2 x 131072 slots; with 8 x 30000 slots
// and the call's join 44.0 / 39.4 with 128 channels, 31.7 / 30.0 with 64.
template <int NP, int CW> constexpr int operands() { return CW == 16 ? (NP + 1) / 2 : NP; }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// Scores and weights of one tile for the first RA of a wave's RT row tiles; the keys are free after it.
template <int D, int RT, int RA, int NP, int CW>
__device__ __forceinline__ void weigh(Rows<D, RT> &st, Probs<operands<NP, CW>()> (&pr)[RA], const Keys<D> &t, const bf16x8 *q,
                                      const WaveAt &w, float c, bool masked, const uint32_t (&vis)[RT]) {
    constexpr int NB = D / 32, KS = D / 16, NG = operands<NP, CW>();
    f32x16 s[RA];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const float unit = unit_at<0>(t.e[j / 2] >> (16 * (j & 1) + 8 * w.h));
        // a group of q operands is asked for ahead of the products that use it
        bf16x8 qf[RA][NG][4];
#pragma unroll
        for (int rt = 0; rt < RA; ++rt)
#pragma unroll
            for (int p = 0; p < NG; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[rt][p][i] = q[((rt * NG + p) * KS + 4 * j + i) * 64];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x8 a = eight_of(t.c[j][i], unit);
#pragma unroll
            for (int rt = 0; rt < RA; ++rt)
#pragma unroll
                for (int p = NG - 1; p >= 0; --p) {  // smallest terms first
                    const bf16x8 b = qf[rt][p][i];
                    if (j == 0 && i == 0 && p == NG - 1)
                        s[rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, f32x16{}, 0, 0, 0);
                    else
                        s[rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, s[rt], 0, 0, 0);
                }
        }
    }
    // Values of a lane: its 16 tokens, or, of a row in two columns, tokens 0-15 of the tile in the
    // first and 16-31 in the second, as the exchange that adds the planes' scores leaves them.
    constexpr int NV = CW / 2;
#pragma unroll
    for (int rt = 0; rt < RA; ++rt) {
        float x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (CW == 16) {  // bf16: both columns have the row's scores
                uint32_t a = __float_as_uint(s[rt][i]), b = __float_as_uint(s[rt][8 + i]);
                swap_columns(a, b);
                x[i] = NP == 1 ? __uint_as_float(a) : __uint_as_float(a) + __uint_as_float(b);
            } else {
                x[i] = s[rt][i];
            }
        }
        if (__builtin_expect(masked, 0)) {
            const uint32_t mine = vis[rt] >> (4 * w.h + (CW == 16 ? w.r & 16 : 0));
#pragma unroll
            for (int i = 0; i < NV; ++i) x[i] = (mine >> (8 * (i / 4) + i % 4)) & 1u ? x[i] : -__builtin_inff();
        }
        float e[NV], sum;
        auto exponentials = [&] {
#pragma unroll
            for (int i = 0; i < NV; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c, -st.m[rt]));
            if constexpr (NP == 1 && CW == 32) {  // the sum is of the weights as they are rounded
                float y[2] = {0.f, 0.f};
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t two = pack_bf16(e[8 * g + 2 * i], e[8 * g + 2 * i + 1]);
                        pr[rt].p[0][g][i] = two;
                        y[g] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), bf16x2{1.f, 1.f}, y[g], false);
                    }
                sum = y[0] + y[1];
            } else {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = NV == 16 ? e[i] + e[NV - 8 + i] : e[i];
                sum = ((y[0] + y[4]) + (y[1] + y[5])) + ((y[2] + y[6]) + (y[3] + y[7]));
            }
        };
        exponentials();
        // The reference holds while no weight of the wave's rows exceeds it much.  A NaN comes here
        // too, and stays one.
        if (__builtin_expect(__any(!(sum <= kSlack)), 0)) {
            float mx = x[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) mx = fmaxf(mx, x[i]);
            if constexpr (CW == 16) mx = fmaxf(mx, other_columns(mx));
            const float m = fmaxf(st.m[rt], fmaxf(mx, other_half(mx)) * c);
            const float f = __builtin_amdgcn_exp2f(st.m[rt] - m);
            st.m[rt] = m;
            st.l[rt] *= f;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) st.o[rt][n][i] *= f;
            exponentials();
        }
        st.l[rt] += sum;
        if constexpr (NP == 1 && CW == 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi = pack_bf16(e[2 * i], e[2 * i + 1]);
                uint32_t lo = pack_bf16(e[2 * i] - __uint_as_float(hi << 16), e[2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u));
                swap_columns(hi, lo);
                pr[rt].p[0][0][i] = hi;
                pr[rt].p[0][1][i] = lo;
            }
        } else if constexpr (NP == 1) {  // packed with their sum
        } else if constexpr (CW == 16) {
            bf16x8 hi, mid, lo;
            split3(e, hi, mid, lo);
            const u32x4 a = __builtin_bit_cast(u32x4, hi), b = __builtin_bit_cast(u32x4, mid);
            const u32x4 d = __builtin_bit_cast(u32x4, lo);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x0 = a[i], x1 = b[i], y0 = d[i], y1 = 0;
                swap_columns(x0, x1);
                swap_columns(y0, y1);
                pr[rt].p[0][0][i] = x0;
                pr[rt].p[0][1][i] = x1;
                pr[rt].p[1][0][i] = y0;
                pr[rt].p[1][1][i] = y1;
            }
        } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                bf16x8 hi, mid, lo;
                split3(e + 8 * g, hi, mid, lo);
                pr[rt].p[0][g] = __builtin_bit_cast(u32x4, hi);
                pr[rt].p[1][g] = __builtin_bit_cast(u32x4, mid);
                pr[rt].p[2][g] = __builtin_bit_cast(u32x4, lo);
            }
        }
    }
}

// O += P V of one tile; the values are free after it.
template <int D, int RT, int RA, int NG>
__device__ __forceinline__ void gather(Rows<D, RT> &st, const Probs<NG> (&pr)[RA], const Values<D> &t,
                                       const WaveAt &w, bool masked, uint32_t written) {
    constexpr int NB = D / 32;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float unit[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            unit[4 * x] = unit_at<0>(t.e[g][x]);
            unit[4 * x + 1] = unit_at<1>(t.e[g][x]);
            unit[4 * x + 2] = unit_at<2>(t.e[g][x]);
            unit[4 * x + 3] = unit_at<3>(t.e[g][x]);
        }
        if (__builtin_expect(masked, 0)) {  // slots nothing was written to may hold any scale, NaN included
            const uint32_t mine = written >> (16 * g + 4 * w.h);
#pragma unroll
            for (int i = 0; i < 8; ++i) unit[i] = (mine >> (8 * (i / 4) + i % 4)) & 1u ? unit[i] : 1.f;
        }
        u32x4 o[NB];
        value_operands<D>(t.c[g], unit, o);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int rt = 0; rt < RA; ++rt)
#pragma unroll
                for (int p = NG - 1; p >= 0; --p)
                    st.o[rt][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, o[n]), __builtin_bit_cast(bf16x8, pr[rt].p[p][g]),
                        st.o[rt][n], 0, 0, 0);
    }
}

template <typename T> struct Planes {
    static constexpr int n = 1;
};
template <> struct Planes<float> {
    static constexpr int n = 3;
};

// An infinite q makes every score of its row infinite or NaN, and no weight a number, but scores that
// are all -inf would look like a row that sees nothing: it enters as NaN.  (fp32 rows: an infinity's
// second term is NaN.)
__device__ __forceinline__ bf16x8 infinities_to_nan(bf16x8 x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] |= (((w[i] & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u) >> 9;
    return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ uint32_t bits_below(int n) {  // the lowest n bits, n of any sign
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Bytes of LDS: the rows' q as operands; then, up to four channel tiles at a time, the four waves'
// accumulators of a row tile on their way to the waves that join them, and the waves' (m, sum).
template <int D> constexpr int joined_tiles() { return D / 32 < 4 ? D / 32 : 4; }
template <int D> constexpr int joined_bytes() { return joined_tiles<D>() * 16 * 1024; }
template <int D, int RT, int NG> constexpr int attn_lds() {
    constexpr int q = RT * NG * (D / 16) * 1024, j = joined_bytes<D>() + RT * 2048;
    return q > j ? q : j;
}

// N (2 or 4) consecutive channels of a row.
template <int N> __device__ __forceinline__ void store_run(float *p, const float (&x)[N]) {
    if constexpr (N == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}
template <int N> __device__ __forceinline__ void store_run(bf16_t *p, const float (&x)[N]) {
    if constexpr (N == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    else
        *reinterpret_cast<uint32_t *>(p) = pack_bf16(x[0], x[1]);
}

__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(uint64_t(x) >> 32));
    return int64_t(uint64_t(hi) << 32 | lo);
}

// Where a position of the work line lies.
struct UnitAt {
    int li, seq, head, block;
    int64_t x;      // position within the unit
    SeqWork work;   // of the sequence
};

template <bool SP>
__device__ __forceinline__ SeqWork work_of(const AttnParams &P, int seq, int tile_rows) {
    const int64_t capacity = int64_t(P.max_pages) << P.page_shift;
    const int n_new = P.seq_off[seq + 1] - P.seq_off[seq];
    if constexpr (SP)
        return sparse_work(P.sparse, P.length[seq], n_new, P.G, tile_rows, P.parent != nullptr, capacity,
                           P.page_shift);
    else
        return seq_work(P.length[seq], n_new, P.G, tile_rows, P.parent != nullptr, capacity);
}

// x + the value CTRL lanes below, 0 where ROWS leaves the lane out or there is none.
template <int CTRL, int ROWS> __device__ __forceinline__ int64_t plus_below(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(x)), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint64_t(x) >> 32), CTRL, ROWS, 0xF, false);
    return x + int64_t(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ int64_t lane64(int64_t x, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(x), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(uint64_t(x) >> 32), lane);
    return int64_t(uint64_t(hi) << 32 | lo);
}

// Costs of 64 sequences, all heads of a layer, one a lane, and their running sum up to the lane's:
// shifts by 1, 2, 4 and 8 within the rows of 16 lanes, then the rows' last values onwards.
template <bool SP>
__device__ __forceinline__ int64_t costs_of(const AttnParams &P, int first, int lane, int tile_rows, int64_t &run) {
    const int64_t c = first + lane < P.S ? P.H * work_of<SP>(P, first + lane, tile_rows).cost : 0;
    run = plus_below<0x111, 0xF>(c);
    run = plus_below<0x112, 0xF>(run);
    run = plus_below<0x114, 0xF>(run);
    run = plus_below<0x118, 0xF>(run);
    run = plus_below<0x142, 0xA>(run);
    run = plus_below<0x143, 0xC>(run);
    return c;
}

// The start of share `share` of `shares`, its length (0: nothing left for it) and every share's.
template <bool SP>
__device__ __forceinline__ UnitAt share_start(const AttnParams &P, uint32_t share, int lane, int tile_rows,
                                              int64_t &left, int64_t &q) {
    UnitAt u{};
    int64_t run = 0, own = 0, per_layer = 0;
    for (int b = 0; b < P.S; b += 64) {
        own = costs_of<SP>(P, b, lane, tile_rows, run);
        per_layer += lane64(run, 63);
    }
    const int64_t total = per_layer * P.n_layers;
    // all that follows is the same in every lane: scalar registers, which the walk has to spare
    q = uniform64(quotient(total + P.shares - 1, P.shares));
    const int64_t at = share * q;
    left = min(q, total - at);
    if (left <= 0) return u;
    u.li = P.n_layers == 1 ? 0 : __builtin_amdgcn_readfirstlane(int(quotient(at, per_layer)));
    int64_t rem = at - u.li * per_layer;
    for (int b = 0; b < P.S; b += 64) {
        if (P.S > 64) own = costs_of<SP>(P, b, lane, tile_rows, run);
        const uint64_t beyond = __ballot(run > rem);
        if (beyond != 0) {
            const int l = __builtin_ctzll(beyond);
            u.seq = b + l;
            rem -= lane64(run - own, l);
            break;
        }
        rem -= lane64(run, 63);
    }
    u.work = work_of<SP>(P, u.seq, tile_rows);
    u.head = __builtin_amdgcn_readfirstlane(int(quotient(rem, u.work.cost)));
    rem -= u.head * u.work.cost;
    u.block = __builtin_amdgcn_readfirstlane(int(block_at(u.work, rem)));
    u.x = rem - cost_before(u.work, u.block);
    return u;
}

}  // namespace

// SP: sparse attention.  A sequence's blocks are those of its selections, one selection's after the
// other's, and the slots are a selection's (SparseShape); all else is the same.  us: 32 tokens, 35 pages of 64 slots
// each, 24; trees of 22 nodes, 48 heads, 67 pages, 51; four chunks of prompts, 16 tokens a selection, 54 GFLOP in 85.
// The join included: trees in fp32 77, with 256 channels 43, both 71; chunks 162, 91, 163.  fp32 rows with 256 channels
// spill 27 registers, the dense form 3.
template <int D, int RT, typename TIn, int CW, bool SP>
__global__ __launch_bounds__(kAttnThreads, 2) void attention_kernel(AttnParams P) {
    constexpr int NP = Planes<TIn>::n, NG = operands<NP, CW>(), NB = D / 32, KS = D / 16, TR = 32 * RT;
    extern __shared__ __align__(16) char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    WaveAt w;
    w.lane = threadIdx.x & 63;
    w.r = w.lane & 31;
    w.h = w.lane >> 5;
    const bool tree = P.parent != nullptr;
    UnitAt u;
    int64_t left, q = 0;  // of this workgroup's share; length of a share
    uint32_t share = 0;
    bool begins;          // the run at hand is its unit's first
    if (P.parts != 0) {
        // A workgroup a part: heads go to consecutive workgroups, hence XCDs; the last blocks of a
        // sequence, which see the most, start first.  Sequences come one after the other: dealt in
        // turn, those with fewer blocks would leave their turns empty, and as workgroups go round
        // the shader engines in order, with 4 of them one engine had all the work.
        uint32_t i = blockIdx.x;
        share = i;
        const int part = int(i % uint32_t(P.parts));
        i /= uint32_t(P.parts);
        u.head = __builtin_amdgcn_readfirstlane(int(i % uint32_t(P.H)));
        i /= uint32_t(P.H);
        u.block = __builtin_amdgcn_readfirstlane(P.row_blocks - 1 - int(i % uint32_t(P.row_blocks)));
        i /= uint32_t(P.row_blocks);
        u.seq = __builtin_amdgcn_readfirstlane(int(i % uint32_t(P.S)));
        u.li = __builtin_amdgcn_readfirstlane(int(i / uint32_t(P.S)));
        u.work = work_of<SP>(P, u.seq, TR);
        if (u.block >= u.work.blocks) return;
        const Run run = part_of(u.work.a + u.work.b * u.block, part, P.parts);
        u.x = run.x;
        left = run.length;
        begins = run.begins;
    } else {
        // Consecutive shares, which read the same slots, go to one XCD.
        share = xcd_logical(blockIdx.x, uint32_t(P.shares));
        u = share_start<SP>(P, share, w.lane, TR, left, q);
        if (left <= 0) return;
        begins = u.x == 0;  // a share is not empty
    }
    bf16x8 *qs = reinterpret_cast<bf16x8 *>(lds);

    for (bool started = false;; started = true) {
    const int64_t cost = u.work.a + u.work.b * u.block;
    const int64_t x1 = min(cost, u.x + left);
    left -= x1 - u.x;
    const int head = u.head, layer = P.layer_begin + u.li;
    const int off = P.seq_off[u.seq], n_new = P.seq_off[u.seq + 1] - off;
    int64_t capacity = int64_t(P.max_pages) << P.page_shift;
    int past = length_of(P.length[u.seq], capacity);
    // rows of the block, [R0, R)
    int R = n_new * P.G, R0 = u.block * TR;
    if constexpr (SP) {
        const SparseRows rows = sparse_rows(P.sparse, u.block, n_new, P.G, TR);
        const SparseSlots slots = sparse_slots(P.sparse, past, capacity, P.page_shift);
        R0 = rows.first;
        R = rows.end;
        past = slots.past;
        capacity = slots.capacity;
        w.chosen = slots.chosen;
        w.full = slots.full;
        w.selected = P.selected + ((int64_t(layer) * P.T + off + rows.token) * P.H + head) * P.sparse.top;
    }
    w.table = P.pages + int64_t(u.seq) * P.max_pages;
    w.slab_base = kv_slab(layer, P.n_pages, 0, P.H, head);
    if (started) __syncthreads();  // the last unit's states have been read

    // Lane numbers that the compiler takes for new ones in every unit: what it would compute from
    // them ahead of the loop, it would have to keep or spill while the tiles are walked.
    auto fresh = [&] {
        int x = w.lane;
        asm volatile("" : "+v"(x));
        return x;
    };
    // ---- the wave's slots --------------------------------------------------------------
    // The last slot any row of this block sees: its last token's own (tree: the whole tail).
    const int total = slots_upto(past, n_new - 1, capacity);
    const int last_node = __builtin_amdgcn_readfirstlane(min(R0 + TR - 1, R - 1) / P.G);
    const int tiles = ((tree ? total : slots_upto(past, last_node, capacity)) + 31) / 32;
    const int s0 = __builtin_amdgcn_readfirstlane(tile_at(u.x, cost, tiles));
    const int s1 = __builtin_amdgcn_readfirstlane(tile_at(x1, cost, tiles));
    const int t0 = s0 + int(int64_t(s1 - s0) * wave / 4), t1 = s0 + int(int64_t(s1 - s0) * (wave + 1) / 4);
    const int all_see = tree ? past : past + __builtin_amdgcn_readfirstlane(R0 / P.G) + 1;  // slots below this are seen by every row

    // The first page ids, the rows of q and then the first tile are all under way together.
    Pages pages;
    if (t0 < t1) fetch_pages<SP>(pages, P, w, t0);
    // ---- q as operands in LDS, a quarter a wave ---------------------------------------------
    const int ql0 = fresh(), qr = ql0 & 31, qh = ql0 >> 5;
    typedef typename std::conditional<NP == 1, bf16x8, floatx4[2]>::type QLoad;
    QLoad qv[RT][KS / 4];
    int node[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(R0 + 32 * rt + qr % CW, R - 1);  // rows past the end repeat the last one
        node[rt] = row / P.G;
        const int hq = head * P.G + row % P.G;
        const TIn *qp = static_cast<const TIn *>(P.q) +
                        ((int64_t(layer) * P.T + off + node[rt]) * (P.H * P.G) + hq) * D;
#pragma unroll
        for (int k = 0; k < KS / 4; ++k) {  // operand 4 k + wave
            const TIn *src = qp + 32 * (2 * k + qh) + 8 * wave;
            if constexpr (NP == 1) {
                qv[rt][k] = *reinterpret_cast<const bf16x8 *>(src);
            } else {
                qv[rt][k][0] = reinterpret_cast<const floatx4 *>(src)[0];
                qv[rt][k][1] = reinterpret_cast<const floatx4 *>(src)[1];
            }
        }
    }
    Rows<D, RT> st;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        st.m[rt] = kNoScore;
        st.l[rt] = 0.f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) st.o[rt][n][i] = 0.f;
    }
    // Tiles in flight.  A wave with one row tile spends little on each and is bound by how many
    // bytes it has under way; two row tiles leave registers for one tile, whose keys and values are
    // asked for again as soon as they are used up.
    constexpr int NBUF = RT * D * NG <= 128 ? 2 : 1;
    Keys<D> keys[NBUF];
    Values<D> values[NBUF];
    uint32_t there[NBUF];
    if (t0 < t1) {
#pragma unroll
        for (int b = 0; b < NBUF; ++b) {
            const Place x = place_of<SP>(pages, P, w, min(t0 + b, t1 - 1));
            there[b] = x.there;
            load_keys<D>(keys[b], P, w, x);
            load_values<D>(values[b], P, w, x);
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int k = 0; k < KS / 4; ++k) {
            const int ks = 4 * k + wave;
            if constexpr (NP == 1) {
                qs[(rt * KS + ks) * 64 + ql0] = infinities_to_nan(qv[rt][k]);
            } else {
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = qv[rt][k][0][e];
                    x[4 + e] = qv[rt][k][1][e];
                }
                bf16x8 hi, mid, lo;
                split3(x, hi, mid, lo);
                if constexpr (CW == 16) {
                    qs[((rt * NG) * KS + ks) * 64 + ql0] = qr < 16 ? hi : mid;
                    qs[((rt * NG + 1) * KS + ks) * 64 + ql0] = qr < 16 ? lo : bf16x8{};
                } else {
                    qs[((rt * NG) * KS + ks) * 64 + ql0] = hi;
                    qs[((rt * NG + 1) * KS + ks) * 64 + ql0] = mid;
                    qs[((rt * NG + 2) * KS + ks) * 64 + ql0] = lo;
                }
            }
        }
    __syncthreads();
    auto walk = [&](auto active) {
        constexpr int RA = decltype(active)::value;
        for (int tb = t0; tb < t1; tb += NBUF) {
#pragma unroll
            for (int b = 0; b < NBUF; ++b) {
                const int t = tb + b;
                if (t >= t1) break;
                const int base = t * 32;
                const bool masked = base + 32 > all_see || there[b] != ~0u;
                uint32_t vis[RT], written = 0;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) vis[rt] = 0;
                if (__builtin_expect(masked, 0)) {
                    written = there[b] & bits_below(total - base);
#pragma unroll
                    for (int rt = 0; rt < RA; ++rt) {
                        uint32_t bits;
                        if (tree) {
                            bits = bits_below(past - base);
                            const int first = base - past;  // node of the tile's first slot
                            // a row's ancestors have smaller ids: walk up until below this tile
                            for (int a = node[rt]; a >= 0 && a >= first;) {
                                if (a < first + 32) bits |= 1u << (a - first);
                                const int up = P.parent[off + a];
                                a = up < 0 ? -1 : min(up - off, a - 1);
                            }
                        } else {
                            bits = bits_below(past + node[rt] + 1 - base);
                        }
                        vis[rt] = bits & written;
                    }
                }
                // Past the end the last tile is asked for again, so that every step has the same
                // loads under way and waits for no more than the ones it uses.
                const Place x = place_of<SP>(pages, P, w, min(t + NBUF, t1 - 1));
                Probs<NG> pr[RA];
                // q stays in LDS where it and the accumulators would not fit the registers
                // together: the compiler, which sees it does not change, would keep it and spill
                int ql = w.lane;
                if constexpr (RT * D * (2 + NG) > 512) asm volatile("" : "+v"(ql));
                weigh<D, RT, RA, NP, CW>(st, pr, keys[b], qs + ql, w, P.c, masked, vis);
                load_keys<D>(keys[b], P, w, x);
                gather<D, RT, RA, NG>(st, pr, values[b], w, masked, written);
                load_values<D>(values[b], P, w, x);
                there[b] = x.there;
            }
        }
        // The compiler lays the two forms of the walk out one behind the other, and without this its
        // waits in the second would cover loads it takes to be under way from the first.
        if constexpr (RA < RT) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    };
    if (t0 < t1) {
        // a last block whose second row tile is empty does not compute it
        if (RT == 2 && R0 + 32 >= R)
            walk(std::integral_constant<int, 1>{});
        else
            walk(std::integral_constant<int, RT>{});
    }

    // ---- join the waves, and write the rows or their fragment -----------------------------
    // Wave k joins values 4 k .. 4 k + 3 of each accumulator: 8 d/32 consecutive channels of a row.
    constexpr int NJ = joined_tiles<D>();
    const int el = fresh(), er = el & 31, eh = el >> 5;
    floatx4 *box = reinterpret_cast<floatx4 *>(lds);
    float2 *ml = reinterpret_cast<float2 *>(lds + joined_bytes<D>());
    const bool whole = begins && x1 == cost;
    const int64_t fragment = fragment_at(share, begins) * TR;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = 32 * rt + er, row = R0 + r;
        float f[4];
#pragma unroll
        for (int n0 = 0; n0 < NB; n0 += NJ) {
            __syncthreads();  // q, or the last accumulators, have been read
            if (n0 == 0 && rt == 0) {
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    if constexpr (CW == 16) st.l[x] += other_columns(st.l[x]);
                    ml[(x * 4 + wave) * 64 + el] = make_float2(st.m[x], st.l[x] + other_half(st.l[x]));
                }
            }
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    box[((wave * NJ + n) * 4 + k) * 64 + el] =
                        floatx4{st.o[rt][n0 + n][4 * k], st.o[rt][n0 + n][4 * k + 1],
                                st.o[rt][n0 + n][4 * k + 2], st.o[rt][n0 + n][4 * k + 3]};
            __syncthreads();
            if (n0 == 0) {
                float2 y[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) y[x] = ml[(rt * 4 + x) * 64 + el];
                const float m = fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x));
                float l = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    f[x] = __builtin_amdgcn_exp2f(y[x].x - m);
                    l += f[x] * y[x].y;
                }
                if (whole) {  // no visible slot: l = 0 and O = 0, the row is 0
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int x = 0; x < 4; ++x) f[x] *= inv;
                } else if (wave == 0 && eh == 0 && row < R) {
                    P.part_ml[fragment + r] = make_float2(m, l);
                }
            }
            floatx4 sum[NJ] = {};
#pragma unroll 1  // the two columns of a row in turn: unrolled, both would be in registers at once
            for (int at = 0; at < 32; at += CW)
#pragma unroll
                for (int n = 0; n < NJ; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        sum[n] += box[((x * NJ + n) * 4 + wave) * 64 + 32 * eh + er % CW + at] * f[x];
            float o[4][NJ];
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e][n] = sum[n][e];
            if (row < R) {
                // value e of tile n: channel NB (8 k + 4 h + e) + n
                const int64_t at = int64_t(NB) * (8 * wave + 4 * eh) + n0;
                if (!whole) {
                    float *y = P.part_o + (fragment + r) * D + at;
#pragma unroll
                    for (int e = 0; e < 4; ++e) store_run<NJ>(y + e * NB, o[e]);
                } else {
                    TIn *y = static_cast<TIn *>(P.out) +
                             ((int64_t(layer) * P.T + off + row / P.G) * (P.H * P.G) + head * P.G + row % P.G) * D + at;
#pragma unroll
                    for (int e = 0; e < 4; ++e) store_run<NJ>(y + e * NB, o[e]);
                }
            }
        }
    }
    if (begins && P.parts != 1 && threadIdx.x == 0) {
        Cut c;
        c.first = int(share);
        c.count = P.parts != 0 ? P.parts : x1 < cost ? 1 + int(quotient(cost - x1 + q - 1, q)) : 1;
        P.cut[((int64_t(u.li) * P.S + u.seq) * P.H + head) * P.row_blocks + u.block] = c;
    }
    if (left <= 0) return;  // uniform over the workgroup

    // ---- the next unit of the line ------------------------------------------------------
    u.x = 0;
    begins = true;
    if (++u.block == int(u.work.blocks)) {
        u.block = 0;
        if (++u.head == P.H) {
            u.head = 0;
            do {  // a sequence with work: there is one, as some of the share is left
                if (++u.seq == P.S) {
                    u.seq = 0;
                    if (++u.li == P.n_layers) return;  // only if the lengths change under the call
                }
                u.work = work_of<SP>(P, u.seq, TR);
            } while (u.work.blocks == 0);
        }
    }
    }
}

// Joins the fragments of the units that were cut; gridDim.x counts the units.  WIDE: 16 bytes of a row a
// lane, rows dealt to the waves of gridDim.y workgroups; otherwise (many fragments) a workgroup a row, whose
// fragments its eight waves share.  WIDE, fragments of 90 chunk blocks of 64 rows and 8 heads: 11 us; with a row a
// wave, 8 bytes a lane and one fragment at a time, 20.  Dense calls with that join / this one, us: trees of 22 nodes, 48 / 8
// heads of 64, 8 caches 65.4 / 62.2, 20 caches 80.7 / 73.2, of 128 84.8 / 82.7 and 97.1 / 93.3; chunks of 500, 16 / 4 heads of
// 64, 52.7 / 48.0; single tokens and single trees as before (0.98 to 1.02), and all the same bits.
template <int D, typename TIn, bool WIDE, bool SP>
__global__ __launch_bounds__(512) void attention_join_kernel(AttnParams P, int tile_rows) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    uint32_t i = blockIdx.x;
    const Cut cut = P.cut[i];  // not written where the sequence has no such block
    const int block = int(i % uint32_t(P.row_blocks));
    i /= uint32_t(P.row_blocks);
    const int head = int(i % uint32_t(P.H));
    i /= uint32_t(P.H);
    const int seq = int(i % uint32_t(P.S)), layer = P.layer_begin + int(i / uint32_t(P.S));
    const int off = P.seq_off[seq], n_new = P.seq_off[seq + 1] - off;
    int R0 = block * tile_rows, rows = min(tile_rows, n_new * P.G - R0);
    if constexpr (SP) {
        if (n_new == 0) return;
        const SparseRows at = sparse_rows(P.sparse, block, n_new, P.G, tile_rows);
        R0 = at.first;
        rows = at.end - at.first;
    }
    if (rows <= 0 || cut.count == 1) return;
    const int first = cut.first, count = cut.count;
    auto out_of = [&](int row) {
        return static_cast<TIn *>(P.out) +
               ((int64_t(layer) * P.T + off + row / P.G) * (P.H * P.G) + head * P.G + row % P.G) * D;
    };
    auto fragment = [&](int f, int r) { return fragment_at(first + f, f == 0) * tile_rows + r; };
    if constexpr (WIDE) {
        constexpr int LR = D / 4, RW = 64 / LR;  // lanes of a row, rows of a wave
        for (int r0 = (int(blockIdx.y) * 8 + wave) * RW; r0 < rows; r0 += int(gridDim.y) * 8 * RW) {
            const int r = min(r0 + lane / LR, rows - 1), at = lane % LR;
            float2 ml[4];
            floatx4 x[4];
            // four fragments under way together; of fewer the last again, which then counts for nothing
            auto load = [&](int f0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t f = fragment(min(f0 + i, count - 1), r);
                    ml[i] = P.part_ml[f];
                    x[i] = *reinterpret_cast<const floatx4 *>(P.part_o + f * D + 4 * at);
                }
            };
            load(0);
            float m = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
            if (count > 4) {
                for (int f = 4 + at; f < count; f += LR) m = fmaxf(m, P.part_ml[fragment(f, r)].x);
#pragma unroll
                for (int d = LR / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
            }
            float l = 0.f;
            floatx4 o = {};
            for (int f0 = 0;;) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool more = f0 + i < count;
                    const float e = __builtin_amdgcn_exp2f(ml[i].x - m);
                    l = more ? fmaf(ml[i].y, e, l) : l;
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[c] = more ? fmaf(x[i][c], e, o[c]) : o[c];
                }
                f0 += 4;
                if (f0 >= count) break;
                load(f0);
            }
            const float f = l == 0.f ? 0.f : 1.f / l;
            if (r0 + lane / LR >= rows) continue;
            TIn *y = out_of(R0 + r) + 4 * at;
            if constexpr (sizeof(TIn) == 2) {
                ushort4 z;
                z.x = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[0] * f));
                z.y = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[1] * f));
                z.z = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[2] * f));
                z.w = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[3] * f));
                *reinterpret_cast<ushort4 *>(y) = z;
            } else {
                *reinterpret_cast<floatx4 *>(y) = o * f;
            }
        }
    } else {
        constexpr int PL = D / 64;  // channels a lane
        __shared__ float s_l[8], s_o[8][D];
        for (int r = blockIdx.y; r < rows; r += gridDim.y) {
            float m = kNoScore;
            for (int f = lane; f < count; f += 64) m = fmaxf(m, P.part_ml[fragment(f, r)].x);
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
            float l = 0.f, o[PL] = {};
#pragma unroll 8
            for (int f = wave; f < count; f += 8) {
                const float2 ml = P.part_ml[fragment(f, r)];
                const float e = __builtin_amdgcn_exp2f(ml.x - m);
                l += ml.y * e;
                const float *x = P.part_o + fragment(f, r) * D + lane * PL;
#pragma unroll
                for (int i = 0; i < PL; ++i) o[i] += x[i] * e;
            }
            __syncthreads();  // the last row's have been read
            if (lane == 0) s_l[wave] = l;
#pragma unroll
            for (int i = 0; i < PL; ++i) s_o[wave][lane * PL + i] = o[i];
            __syncthreads();
            if (wave != 0) continue;
            l = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) o[i] = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                l += s_l[x];
#pragma unroll
                for (int i = 0; i < PL; ++i) o[i] += s_o[x][lane * PL + i];
            }
            const float f = l == 0.f ? 0.f : 1.f / l;
            TIn *y = out_of(R0 + r) + lane * PL;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                if constexpr (sizeof(TIn) == 2)
                    y[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[i] * f));
                else
                    y[i] = o[i] * f;
            }
        }
    }
}

namespace {

template <int D, int RT, typename TIn, int CW, bool SP>
gdn_status launch_attention(const AttnParams &P, const AttentionPlan &plan, hipStream_t s) {
    constexpr int bytes = attn_lds<D, RT, operands<Planes<TIn>::n, CW>()>();
    static_assert(bytes <= 80 * 1024, "two workgroups a CU");
    hipLaunchKernelGGL((attention_kernel<D, RT, TIn, CW, SP>), dim3(uint32_t(plan.workgroups)), dim3(kAttnThreads),
                       bytes, s, P);
    GDN_LAUNCH_CHECK("attention_kernel");
    if (plan.parts == 1) return GDN_OK;
    // many fragments a unit: a workgroup a row; otherwise a wave, spread over the device where there
    // are few units
    if (plan.workgroups >= 8 * plan.units)
        hipLaunchKernelGGL((attention_join_kernel<D, TIn, false, SP>), dim3(uint32_t(plan.units), plan.max_rows),
                           dim3(512), 0, s, P, plan.tile_rows);
    else {
        constexpr int rows = 8 * 256 / D;  // of a workgroup at a time
        hipLaunchKernelGGL((attention_join_kernel<D, TIn, true, SP>),
                           dim3(uint32_t(plan.units), plan.units < 512 ? (plan.max_rows + rows - 1) / rows : 1),
                           dim3(512), 0, s, P, plan.tile_rows);
    }
    GDN_LAUNCH_CHECK("attention_join_kernel");
    return GDN_OK;
}

template <int D, bool SP>
gdn_status launch_attention(const AttnParams &P, const AttentionPlan &plan, bool bf16, hipStream_t s) {
    if (!bf16) {
        if (plan.max_rows <= 16) return launch_attention<D, 1, float, 16, SP>(P, plan, s);
        return launch_attention<D, 1, float, 32, SP>(P, plan, s);
    }
    if constexpr (D <= 128)
        if (plan.tile_rows == 64) return launch_attention<D, 2, bf16_t, 32, SP>(P, plan, s);
    if (plan.max_rows <= 16) return launch_attention<D, 1, bf16_t, 16, SP>(P, plan, s);
    return launch_attention<D, 1, bf16_t, 32, SP>(P, plan, s);
}

template <bool SP>
gdn_status launch_attention(const AttnParams &P, const AttentionPlan &plan, int32_t head_dim, bool bf16,
                            hipStream_t s) {
    switch (head_dim) {
        case 64: return launch_attention<64, SP>(P, plan, bf16, s);
        case 128: return launch_attention<128, SP>(P, plan, bf16, s);
        default: return launch_attention<256, SP>(P, plan, bf16, s);
    }
}

gdn_status run_attention(const gdn_kv_args *a, const gdn_sparse_args *sparse, const int32_t *host_offs,
                         const int32_t *dev_offs, const int32_t *parent, const char *who, void *stream) {
    gdn_status st = check_attention_sizes(a, host_offs, who);
    if (st != GDN_OK) return st;
    if (sparse != nullptr) {
        st = check_sparse_sizes(a, sparse, host_offs, who);
        if (st != GDN_OK) return st;
        if (sparse->selected == nullptr) return fail(GDN_EINVAL, "%s: null selected", who);
    }
    // the running maximum and the masks are taken of the unscaled products
    const float c = a->scale * 1.44269504088896340736f;
    if (!(a->scale >= FLT_MIN && c <= FLT_MAX))
        return fail(GDN_EINVAL, "%s: scale must be positive, normal and finite", who);
    const void *io[] = {a->q, a->out};
    st = check_aligned16(io, 2, who, "q/out");
    if (st != GDN_OK) return st;
    const AttentionPlan plan = plan_attention(a, host_offs, sparse);
    if (!plan_fits(plan)) return fail(GDN_EINVAL, "%s: too many workgroups", who);
    if (plan.workspace > 0) {
        if (a->workspace == nullptr || a->workspace_bytes < plan.workspace)
            return fail(GDN_ECAPACITY, "%s: workspace holds %lld bytes, the call needs %lld", who,
                        static_cast<long long>(a->workspace ? a->workspace_bytes : 0),
                        static_cast<long long>(plan.workspace));
        const void *ws[] = {a->workspace};
        st = check_aligned16(ws, 1, who, "workspace");
        if (st != GDN_OK) return st;
    }
    AttnParams P{};
    P.q = a->q;
    P.out = a->out;
    P.kc = a->k_codes;
    P.ks = a->k_scales;
    P.vc = a->v_codes;
    P.vs = a->v_scales;
    P.pages = a->pages;
    P.length = a->length;
    P.seq_off = dev_offs;
    P.parent = parent;
    P.S = a->n_seqs;
    P.H = a->n_kv_heads;
    P.G = a->n_heads / a->n_kv_heads;
    P.T = a->n_tokens;
    P.n_pages = a->n_pages;
    P.max_pages = a->max_pages;
    P.page_shift = log2_exact(a->page_tokens);
    P.layer_begin = a->layer_begin;
    P.n_layers = a->n_layers;
    P.row_blocks = plan.row_blocks;
    P.shares = int32_t(plan.workgroups);
    P.parts = plan.parts;
    P.c = c;
    P.part_o = static_cast<float *>(a->workspace);
    P.part_ml = reinterpret_cast<float2 *>(P.part_o + 2 * plan.workgroups * plan.tile_rows * a->head_dim);
    P.cut = reinterpret_cast<Cut *>(P.part_ml + 2 * plan.workgroups * plan.tile_rows);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = a->in_dtype == GDN_BF16;
    if (sparse == nullptr) return launch_attention<false>(P, plan, a->head_dim, bf16, s);
    P.sparse = SparseShape{sparse->top_pages, sparse->share_tokens};
    P.selected = sparse->selected;
    return launch_attention<true>(P, plan, a->head_dim, bf16, s);
}

gdn_status causal_attention(const gdn_kv_args *a, const gdn_sparse_args *sparse, const int32_t *host_seq_offsets,
                            const char *who, void *stream) {
    clear_error();
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, who, true, empty);
    if (st != GDN_OK || empty) return st;
    return run_attention(a, sparse, host_seq_offsets, a->seq_offsets, nullptr, who, stream);
}

gdn_status tree_attention(const gdn_kv_args *a, const gdn_sparse_args *sparse, const int32_t *host_image,
                          const int32_t *dev_image, const char *who, void *stream) {
    clear_error();
    if (!image_ok(host_image) || dev_image == nullptr)
        return fail(GDN_EINVAL, "%s: missing or malformed schedule image", who);
    const ImageView v = view_image(host_image);
    if (a == nullptr) return fail(GDN_EINVAL, "%s: null arguments", who);
    if (v.n_seqs != a->n_seqs || v.n_nodes != a->n_tokens)
        return fail(GDN_EINVAL, "%s: n_seqs/n_tokens differ from the schedule's", who);
    if (sparse != nullptr && sparse->share_tokens != 0)
        return fail(GDN_EINVAL, "%s: share_tokens %d, a tree's nodes share one selection (0)", who,
                    sparse->share_tokens);
    bool empty;
    const int32_t *host_offs = host_image + v.off_seq;
    gdn_status st = check_kv_args(a, host_offs, who, false, empty);
    if (st != GDN_OK || empty) return st;
    return run_attention(a, sparse, host_offs, dev_image + v.off_seq, dev_image + v.off_parent, who, stream);
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                                    void *stream) {
    return causal_attention(a, nullptr, host_seq_offsets, "gdn_attention", stream);
}

extern "C" gdn_status gdn_tree_attention(const gdn_kv_args *a, const int32_t *host_image,
                                         const int32_t *dev_image, void *stream) {
    return tree_attention(a, nullptr, host_image, dev_image, "gdn_tree_attention", stream);
}

extern "C" gdn_status gdn_sparse_attention(const gdn_kv_args *a, const gdn_sparse_args *sparse,
                                           const int32_t *host_seq_offsets, void *stream) {
    if (sparse == nullptr) return fail(GDN_EINVAL, "gdn_sparse_attention: null arguments");
    return causal_attention(a, sparse, host_seq_offsets, "gdn_sparse_attention", stream);
}

extern "C" gdn_status gdn_sparse_tree_attention(const gdn_kv_args *a, const gdn_sparse_args *sparse,
                                                const int32_t *host_image, const int32_t *dev_image, void *stream) {
    if (sparse == nullptr) return fail(GDN_EINVAL, "gdn_sparse_tree_attention: null arguments");
    return tree_attention(a, sparse, host_image, dev_image, "gdn_sparse_tree_attention", stream);
}
