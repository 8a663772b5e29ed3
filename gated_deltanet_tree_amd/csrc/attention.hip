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
// matrix-core pass; the sum is of the unrounded P.  The rounding (2^-9 of each term at most) averages
// out over the terms and stays below the rounding of the bf16 output.
// fp32 rows: q and P are split into three bf16 terms each (exact), K and V are exact in bf16, so
// every product is exact and sums are fp32: three passes.
//
// Waves that share rows join their (m, sum, O) in LDS, workgroups through the workspace and a
// second launch.  A poisoned token has a NaN key scale: its score is NaN where it is visible and
// replaced where it is not; its value is finite, so masked weights of 0 stay 0.
#include <algorithm>
#include <type_traits>

#include "kv_internal.h"
#include "kv_layout.h"
#include "mfma_common.h"

namespace gdn {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnThreads = 256;
constexpr float kNoScore = -3.0e38f;  // m_r before the first visible slot
constexpr float kSlack = 4096.f;      // largest sum of a lane's 16 weights before m_r moves

struct AttnParams {
    const void *q;
    void *out;
    const uint8_t *kc, *ks, *vc, *vs;
    const int32_t *pages, *length, *seq_off;
    const int32_t *parent;  // tree: global parent ids of the schedule image, else null
    float *part_o;          // [splits][n_layers][T][Hq][D]
    float2 *part_ml;        // [splits][n_layers][T][Hq]
    float c;
    int32_t S, H, G, T, n_pages, max_pages, page_shift, layer_begin, n_layers;
    int32_t row_blocks, splits;
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
};

// Where a tile's two groups of 16 slots are, in tokens from the pool's start, and which of them have
// a page (the others stand at page 0 and are masked).
struct Place {
    int64_t at[2];
    uint32_t there;  // 0xFFFF for the first group, 0xFFFF0000 for the second
};

__device__ __forceinline__ Place place_of(const AttnParams &P, const WaveAt &w, int tile) {
    Place x;
    x.there = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int page = __builtin_amdgcn_readfirstlane(
            kv_page(w.table, P.max_pages, P.n_pages, P.page_shift, int64_t(tile) * 32 + 16 * s));
        const int64_t slab = w.slab_base + int64_t(max(page, 0)) * P.H;
        x.at[s] = (slab << P.page_shift) + ((tile * 32 + 16 * s) & ((1 << P.page_shift) - 1));
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

template <int NP> struct Probs {
    u32x4 p[NP][2];  // per plane and 16 tokens
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// Scores and weights of one tile for the first RA of a wave's RT row tiles; the keys are free after it.
template <int D, int RT, int RA, int NP>
__device__ __forceinline__ void weigh(Rows<D, RT> &st, Probs<NP> (&pr)[RA], const Keys<D> &t, const bf16x8 *q,
                                      const WaveAt &w, float c, bool masked, const uint32_t (&vis)[RT]) {
    constexpr int NB = D / 32, KS = D / 16;
    f32x16 s[RA];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const float unit = unit_at<0>(t.e[j / 2] >> (16 * (j & 1) + 8 * w.h));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x8 a = eight_of(t.c[j][i], unit);
#pragma unroll
            for (int rt = 0; rt < RA; ++rt)
#pragma unroll
                for (int p = NP - 1; p >= 0; --p) {  // smallest terms first
                    const bf16x8 b = q[((rt * NP + p) * KS + 4 * j + i) * 64];
                    if (j == 0 && i == 0 && p == NP - 1)
                        s[rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, f32x16{}, 0, 0, 0);
                    else
                        s[rt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, s[rt], 0, 0, 0);
                }
        }
    }
#pragma unroll
    for (int rt = 0; rt < RA; ++rt) {
        if (masked) {
            const uint32_t mine = vis[rt] >> (4 * w.h);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[rt][i] = (mine >> (8 * (i / 4) + i % 4)) & 1u ? s[rt][i] : -__builtin_inff();
        }
        float e[16], sum;
        auto exponentials = [&] {
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(s[rt][i], c, -st.m[rt]));
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = e[i] + e[8 + i];
            sum = ((x[0] + x[4]) + (x[1] + x[5])) + ((x[2] + x[6]) + (x[3] + x[7]));
        };
        exponentials();
        // The reference holds while no weight of the wave's rows exceeds it much.  A NaN comes here
        // too, and stays one.
        if (__any(!(sum <= kSlack))) {
            float mx = s[rt][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[rt][i]);
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
        if constexpr (NP == 1) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    pr[rt].p[0][g][i] = pack_bf16(e[8 * g + 2 * i], e[8 * g + 2 * i + 1]);
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
template <int D, int RT, int RA, int NP>
__device__ __forceinline__ void gather(Rows<D, RT> &st, const Probs<NP> (&pr)[RA], const Values<D> &t,
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
        if (masked) {  // slots nothing was written to may hold any scale, NaN included
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
                for (int p = NP - 1; p >= 0; --p)
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

__device__ __forceinline__ uint32_t bits_below(int n) {  // the lowest n bits, n of any sign
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Bytes of LDS: the rows' q as operands, later the rows' states on their way to one wave.
template <int D, int RT, int NP> constexpr int q_bytes() { return RT * NP * (D / 16) * 1024; }
template <int D, int RT> constexpr int state_bytes() { return RT * (D * 128 + 512); }
template <int D, int RT, int NP, int WR> constexpr int attn_lds() {
    return WR == 1 ? (q_bytes<D, RT, NP>() > 2 * state_bytes<D, RT>() ? q_bytes<D, RT, NP>()
                                                                     : 2 * state_bytes<D, RT>())
                   : WR * q_bytes<D, RT, NP>();
}

template <int D, int RT>
__device__ __forceinline__ void park(const Rows<D, RT> &st, char *mem, int lane) {
    float *ml = reinterpret_cast<float *>(mem);
    floatx4 *o = reinterpret_cast<floatx4 *>(mem + RT * 512);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        ml[(2 * rt) * 64 + lane] = st.m[rt];
        ml[(2 * rt + 1) * 64 + lane] = st.l[rt];
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[((rt * (D / 32) + n) * 4 + i) * 64 + lane] =
                    floatx4{st.o[rt][n][4 * i], st.o[rt][n][4 * i + 1], st.o[rt][n][4 * i + 2], st.o[rt][n][4 * i + 3]};
    }
}

template <int D, int RT>
__device__ __forceinline__ void join(Rows<D, RT> &st, const char *mem, int lane) {
    const float *ml = reinterpret_cast<const float *>(mem);
    const floatx4 *o = reinterpret_cast<const floatx4 *>(mem + RT * 512);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float m2 = ml[(2 * rt) * 64 + lane], l2 = ml[(2 * rt + 1) * 64 + lane];
        const float m = fmaxf(st.m[rt], m2);
        const float f = __builtin_amdgcn_exp2f(st.m[rt] - m), f2 = __builtin_amdgcn_exp2f(m2 - m);
        st.m[rt] = m;
        st.l[rt] = st.l[rt] * f + l2 * f2;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const floatx4 x = o[((rt * (D / 32) + n) * 4 + i) * 64 + lane];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st.o[rt][n][4 * i + e] = st.o[rt][n][4 * i + e] * f + x[e] * f2;
            }
    }
}

}  // namespace

// WR waves of rows a workgroup; the 4 / WR waves of one row group share its slots.
template <int D, int RT, typename TIn, int WR>
__global__ __launch_bounds__(kAttnThreads, 2) void attention_kernel(AttnParams P) {
    constexpr int NP = Planes<TIn>::n, NB = D / 32, KS = D / 16, WK = 4 / WR;
    extern __shared__ __align__(16) char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    WaveAt w;
    w.lane = threadIdx.x & 63;
    w.r = w.lane & 31;
    w.h = w.lane >> 5;
    const int wr = wave % WR, wk = wave / WR;
    // Heads are dealt to consecutive workgroups, hence to the XCDs: workgroups that read the same
    // slots share an L2 when there are 8 kv heads, and few of them when there are less.  The
    // last rows of a sequence, which see the most, start first.
    uint32_t u = blockIdx.x;
    const int head = int(u % uint32_t(P.H));
    u /= uint32_t(P.H);
    const int split = int(u % uint32_t(P.splits));
    u /= uint32_t(P.splits);
    const int seq = int(u % uint32_t(P.S));
    u /= uint32_t(P.S);
    const int li = int(u % uint32_t(P.n_layers));
    const int block = P.row_blocks - 1 - int(u / uint32_t(P.n_layers));
    const int layer = P.layer_begin + li;
    const int off = P.seq_off[seq], n_new = P.seq_off[seq + 1] - off;
    const int R = n_new * P.G;
    if (block * WR * RT * 32 >= R) return;  // uniform over the workgroup
    const int R0 = (block * WR + wr) * RT * 32;
    const int past = max(P.length[seq], 0);
    w.table = P.pages + int64_t(seq) * P.max_pages;
    w.slab_base = kv_slab(layer, P.n_pages, 0, P.H, head);

    // ---- q as operands in LDS -----------------------------------------------------------
    bf16x8 *qs = reinterpret_cast<bf16x8 *>(lds + wr * q_bytes<D, RT, NP>());
    int node[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(R0 + 32 * rt + w.r, R - 1);  // rows past the end repeat the last one
        node[rt] = row / P.G;
        const int hq = head * P.G + row % P.G;
        const TIn *qp = static_cast<const TIn *>(P.q) +
                        ((int64_t(layer) * P.T + off + node[rt]) * (P.H * P.G) + hq) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks % WK != wk) continue;
            const TIn *src = qp + 32 * (2 * (ks / 4) + w.h) + 8 * (ks % 4);
            if constexpr (NP == 1) {
                qs[(rt * KS + ks) * 64 + w.lane] = *reinterpret_cast<const bf16x8 *>(src);
            } else {
                float x[8];
                const floatx4 a = reinterpret_cast<const floatx4 *>(src)[0], b = reinterpret_cast<const floatx4 *>(src)[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = a[e];
                    x[4 + e] = b[e];
                }
                bf16x8 hi, mid, lo;
                split3(x, hi, mid, lo);
                qs[((rt * NP) * KS + ks) * 64 + w.lane] = hi;
                qs[((rt * NP + 1) * KS + ks) * 64 + w.lane] = mid;
                qs[((rt * NP + 2) * KS + ks) * 64 + w.lane] = lo;
            }
        }
    }
    __syncthreads();

    // ---- the wave's slots --------------------------------------------------------------
    // The last slot any row of this wave sees: its last token's own (tree: the whole tail).
    const int total = int(min(int64_t(past) + n_new, int64_t(P.max_pages) << P.page_shift));
    const int last_node = min(R0 + 32 * RT - 1, R - 1) / P.G;
    const bool tree = P.parent != nullptr;
    const int end = R0 >= R ? 0 : tree ? total : min(past + last_node + 1, total);
    const int tiles = (end + 31) / 32;
    const int share = split * WK + wk, shares = P.splits * WK;
    const int t0 = int(int64_t(tiles) * share / shares), t1 = int(int64_t(tiles) * (share + 1) / shares);
    const int all_see = tree ? past : past + R0 / P.G + 1;  // slots below this are seen by every row

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
    auto walk = [&](auto active) {
        constexpr int RA = decltype(active)::value;
        // Tiles in flight.  A wave with one row tile spends little on each and is bound by how
        // many bytes it has under way; two row tiles leave registers for one tile, whose keys and
        // values are asked for again as soon as they are used up.
        constexpr int NBUF = RT * D * NP <= 128 ? 2 : 1;
        Keys<D> keys[NBUF];
        Values<D> values[NBUF];
        uint32_t there[NBUF];
#pragma unroll
        for (int b = 0; b < NBUF; ++b) {
            const Place x = place_of(P, w, min(t0 + b, t1 - 1));
            there[b] = x.there;
            load_keys<D>(keys[b], P, w, x);
            load_values<D>(values[b], P, w, x);
        }
        // Place of the next tile to ask for: its page ids arrive a tile early.  Past the end the last
        // tile is asked for again, so that every step has the same loads under way and waits for
        // no more than the ones it uses.
        Place ahead = place_of(P, w, min(t0 + NBUF, t1 - 1));
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
                if (masked) {
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
                                a = up < 0 ? -1 : up - off;
                            }
                        } else {
                            bits = bits_below(past + node[rt] + 1 - base);
                        }
                        vis[rt] = bits & written;
                    }
                }
                const Place x = ahead;
                ahead = place_of(P, w, min(t + NBUF + 1, t1 - 1));
                Probs<NP> pr[RA];
                // q stays in LDS where it and the accumulators would not fit the registers
                // together: the compiler, which sees it does not change, would keep it and spill
                int ql = w.lane;
                if constexpr (RT * D * (2 + NP) > 512) asm volatile("" : "+v"(ql));
                weigh<D, RT, RA, NP>(st, pr, keys[b], qs + ql, w, P.c, masked, vis);
                load_keys<D>(keys[b], P, w, x);
                gather<D, RT, RA, NP>(st, pr, values[b], w, masked, written);
                load_values<D>(values[b], P, w, x);
                there[b] = x.there;
            }
        }
    };
    if (t0 < t1) {
        // a last block whose second row tile is empty does not compute it
        if (RT == 2 && R0 + 32 >= R)
            walk(std::integral_constant<int, 1>{});
        else
            walk(std::integral_constant<int, RT>{});
    }

    // ---- join the waves of a row group, then the workgroups ---------------------------
    if constexpr (WK == 4) {
        constexpr int kState = state_bytes<D, RT>();
        __syncthreads();  // every wave has read q
        if (wk >= 2) park(st, lds + (wk - 2) * kState, w.lane);
        __syncthreads();
        if (wk < 2) join(st, lds + wk * kState, w.lane);
        __syncthreads();
        if (wk == 1) park(st, lds, w.lane);
        __syncthreads();
        if (wk != 0) return;
        join(st, lds, w.lane);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = R0 + 32 * rt + w.r;
        const float l = st.l[rt] + other_half(st.l[rt]);
        if (row >= R) continue;
        const int hq = head * P.G + row % P.G;
        const int64_t at = (int64_t(off) + row / P.G) * (P.H * P.G) + hq;  // row of one layer
        const int64_t rows = int64_t(P.T) * (P.H * P.G);
        if (P.splits > 1) {
            const int64_t x = (int64_t(split) * P.n_layers + li) * rows + at;
            if (w.h == 0) P.part_ml[x] = make_float2(st.m[rt], l);
            float *o = P.part_o + x * D;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int mm = 8 * (i / 4) + 4 * w.h + i % 4;
#pragma unroll
                for (int n = 0; n < NB; n += 2)
                    *reinterpret_cast<float2 *>(o + mm * NB + n) = make_float2(st.o[rt][n][i], st.o[rt][n + 1][i]);
            }
            continue;
        }
        // no visible slot: l = 0 and O = 0, the row is 0
        const float f = l == 0.f ? 0.f : 1.f / l;
        TIn *o = static_cast<TIn *>(P.out) + (int64_t(layer) * rows + at) * D;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int mm = 8 * (i / 4) + 4 * w.h + i % 4;
#pragma unroll
            for (int n = 0; n < NB; n += 2) {
                const float a = st.o[rt][n][i] * f, b = st.o[rt][n + 1][i] * f;
                if constexpr (NP == 1)
                    *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(o) + mm * NB + n) = pack_bf16(a, b);
                else
                    *reinterpret_cast<float2 *>(o + mm * NB + n) = make_float2(a, b);
            }
        }
    }
}

// One wave a row: joins the splits' (m, sum, O).
template <int D, typename TIn>
__global__ __launch_bounds__(256) void attention_join_kernel(const float *part_o, const float2 *part_ml,
                                                             TIn *out, int64_t rows, int splits) {
    constexpr int PL = D / 64;  // channels a lane
    const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= rows) return;
    const int lane = threadIdx.x & 63;
    float m = kNoScore;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, part_ml[s * rows + row].x);
    float l = 0.f, o[PL] = {};
    for (int s = 0; s < splits; ++s) {
        const float2 ml = part_ml[s * rows + row];
        const float f = __builtin_amdgcn_exp2f(ml.x - m);
        l += ml.y * f;
        const float *x = part_o + (s * rows + row) * D + lane * PL;
#pragma unroll
        for (int i = 0; i < PL; ++i) o[i] += x[i] * f;
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    TIn *y = out + row * D + lane * PL;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        if constexpr (sizeof(TIn) == 2)
            y[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[i] * f));
        else
            y[i] = o[i] * f;
    }
}

namespace {

template <int D, int RT, typename TIn, int WR>
gdn_status launch_kernel(const AttnParams &P, int64_t blocks, hipStream_t s) {
    constexpr int bytes = attn_lds<D, RT, Planes<TIn>::n, WR>();
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    hipLaunchKernelGGL((attention_kernel<D, RT, TIn, WR>), dim3(uint32_t(blocks)), dim3(kAttnThreads),
                       bytes, s, P);
    GDN_LAUNCH_CHECK("attention_kernel");
    return GDN_OK;
}

template <int D, typename TIn>
gdn_status launch_attention(const AttnParams &P, const AttentionPlan &plan, void *out,
                            int n_layers, hipStream_t s) {
    gdn_status st;
    if constexpr (sizeof(TIn) == 2 && D <= 128) {
        if (plan.tile_rows == 64)
            st = plan.row_groups == 4 ? launch_kernel<D, 2, TIn, 4>(P, plan.n_blocks, s)
                                      : launch_kernel<D, 2, TIn, 1>(P, plan.n_blocks, s);
        else
            st = plan.row_groups == 4 ? launch_kernel<D, 1, TIn, 4>(P, plan.n_blocks, s)
                                      : launch_kernel<D, 1, TIn, 1>(P, plan.n_blocks, s);
    } else if constexpr (sizeof(TIn) == 4 && D == 256) {
        st = launch_kernel<D, 1, TIn, 1>(P, plan.n_blocks, s);
    } else {
        st = plan.row_groups == 4 ? launch_kernel<D, 1, TIn, 4>(P, plan.n_blocks, s)
                                  : launch_kernel<D, 1, TIn, 1>(P, plan.n_blocks, s);
    }
    if (st != GDN_OK || P.splits == 1) return st;
    const int64_t per_layer = int64_t(P.T) * P.H * P.G, rows = per_layer * n_layers;
    hipLaunchKernelGGL((attention_join_kernel<D, TIn>), dim3(uint32_t((rows + 3) / 4)), dim3(256), 0, s,
                       P.part_o, P.part_ml, static_cast<TIn *>(out) + P.layer_begin * per_layer * D,
                       rows, P.splits);
    GDN_LAUNCH_CHECK("attention_join_kernel");
    return GDN_OK;
}

gdn_status run_attention(const gdn_kv_args *a, const int32_t *host_offs, const int32_t *dev_offs,
                         const int32_t *parent, const char *who, void *stream) {
    if (a->n_heads < 1 || a->n_heads % a->n_kv_heads != 0)
        return fail(GDN_EINVAL, "%s: n_heads must be a multiple of n_kv_heads", who);
    const void *io[] = {a->q, a->out};
    gdn_status st = check_aligned16(io, 2, who, "q/out");
    if (st != GDN_OK) return st;
    const AttentionPlan plan = plan_attention(a, host_offs);
    if (int64_t(a->n_tokens) * a->n_heads > INT32_MAX)
        return fail(GDN_EINVAL, "%s: more than 2^31 rows", who);
    if (plan.n_blocks > kMaxBlocks ||
        (int64_t(a->n_tokens) * a->n_heads * a->n_layers + 3) / 4 > kMaxBlocks)
        return fail(GDN_EINVAL, "%s: too many workgroups", who);
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
    P.splits = plan.splits;
    P.c = a->scale * 1.44269504088896340736f;
    P.part_o = static_cast<float *>(a->workspace);
    P.part_ml = reinterpret_cast<float2 *>(
        P.part_o + int64_t(plan.splits) * a->n_layers * a->n_tokens * a->n_heads * a->head_dim);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf = a->in_dtype == GDN_BF16;
    switch (a->head_dim) {
        case 64:
            return bf ? launch_attention<64, bf16_t>(P, plan, a->out, a->n_layers, s)
                      : launch_attention<64, float>(P, plan, a->out, a->n_layers, s);
        case 128:
            return bf ? launch_attention<128, bf16_t>(P, plan, a->out, a->n_layers, s)
                      : launch_attention<128, float>(P, plan, a->out, a->n_layers, s);
        default:
            return bf ? launch_attention<256, bf16_t>(P, plan, a->out, a->n_layers, s)
                      : launch_attention<256, float>(P, plan, a->out, a->n_layers, s);
    }
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_attention(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                                    void *stream) {
    clear_error();
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, "gdn_attention", true, empty);
    if (st != GDN_OK || empty) return st;
    return run_attention(a, host_seq_offsets, a->seq_offsets, nullptr, "gdn_attention", stream);
}

extern "C" gdn_status gdn_tree_attention(const gdn_kv_args *a, const int32_t *host_image,
                                         const int32_t *dev_image, void *stream) {
    clear_error();
    if (!image_ok(host_image) || dev_image == nullptr)
        return fail(GDN_EINVAL, "gdn_tree_attention: missing or malformed schedule image");
    const ImageView v = view_image(host_image);
    if (a == nullptr) return fail(GDN_EINVAL, "gdn_tree_attention: null arguments");
    if (v.n_seqs != a->n_seqs || v.n_nodes != a->n_tokens)
        return fail(GDN_EINVAL, "gdn_tree_attention: n_seqs/n_tokens differ from the schedule's");
    bool empty;
    const int32_t *host_offs = host_image + v.off_seq;
    gdn_status st = check_kv_args(a, host_offs, "gdn_tree_attention", false, empty);
    if (st != GDN_OK || empty) return st;
    return run_attention(a, host_offs, dev_image + v.off_seq, dev_image + v.off_parent,
                         "gdn_tree_attention", stream);
}
