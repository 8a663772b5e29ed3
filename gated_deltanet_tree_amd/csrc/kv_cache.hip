// The 4-bit paged key/value cache: append, commit and read (gfx950).
//
// An element is x / 2^e rounded to nearest even on the grid {0, .5, 1, 1.5, 2, 3, 4, 6} with e one
// per 32 channels (see gdn_tree.h).  2^e is a power of two, so the division is exact and every code
// is well defined; the hardware conversion does it for two elements at a time.
//
// All three calls only move data: 2 d s bytes of rows (s = 2 or 4) against 1.0625 d of codes a
// token and kv head.  Four prompts of 1500 to 4096 rows, 8 heads of 128: 12.8 us to append, 11.9 to
// read back, 4.3 TB/s over the two, out of the memory-side cache for the most part; in fp32 17.1 and
// 20.8 us, 5.0 TB/s.  One token a sequence, or one tree's path in 16 layers, is a launch and its chain of
// dependent loads (offsets, page, row index, rows): 3.4 and 4.9 us.  The accepted paths of 32 trees of
// 22 rows in those layers take 11.5 us a call, 5.6 with counts of 0: the grid covers all 22 rows, and
// a quad asks for four rows though the paths' ends hold fewer (7.7 us where the trees have 9 rows).
//
// Work split: a thread takes 8 channels of the 4 tokens of an aligned token quad.  8 channels are one
// 16-byte load of a bf16 row and one dword of codes, a quarter of a scale block (whose largest
// magnitude is two lane exchanges away), and the quad is what a value piece of the cache holds
// contiguously: 4 d/64 bytes for every m, stored at once when the whole quad is written.  Quads at the
// ends of a ragged range store only their own tokens' bytes, so neighbouring calls and neighbouring
// tokens never touch one another's.
#include <algorithm>

#include "gdn_device.h"
#include "kv_internal.h"
#include "kv_layout.h"

namespace gdn {

struct KvParams {
    void *k, *v;
    uint8_t *kc, *ks, *vc, *vs;
    const int32_t *pages, *length, *seq_off;
    const int32_t *begin;         // read: first slot of each sequence (null: its length)
    const int32_t *rows, *counts;  // commit (null: row i, every row)
    int32_t *new_length;           // commit: written by the last workgroup too (null: not here)
    int32_t S, H, T, n_pages, max_pages, page_shift, layer_begin, row_stride;
    int32_t quads, quad_blocks;  // quads a head, workgroups a sequence and layer
};

constexpr int kKvThreads = 256;

template <typename TIn> __device__ __forceinline__ void load8(const TIn *p, float *x);
template <> __device__ __forceinline__ void load8<bf16_t>(const bf16_t *p, float *x) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float *x) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <typename TIn> __device__ __forceinline__ void store8(TIn *p, const float *x);
template <> __device__ __forceinline__ void store8<bf16_t>(bf16_t *p, const float *x) {
    uint32_t w[4];  // a 4-bit float times a power of two has two significant bits: exact
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xFFFF0000u);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float *x) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Largest of the four lanes of an aligned lane quad (a scale block), in every one of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xF, 0xF, true)));
    return x;
}

__device__ __forceinline__ uint32_t magnitude8(const float *x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ uint32_t encode8(const float *x, float unit) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], unit, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], unit, 3);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void decode8(uint32_t w, float unit, float *x) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 3);
    x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1];
    x[4] = c[0]; x[5] = c[1]; x[6] = d[0]; x[7] = d[1];
}

__device__ __forceinline__ float unit_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Codes of 8 value channels of four tokens (one dword each) <-> the pieces of the cache: piece j
// of the 256 / D pieces holds the four tokens' D/64 bytes of one m, token after token.
template <int D> struct ValuePieces;
template <> struct ValuePieces<256> {
    static constexpr int kPieces = 1, kWords = 4;
    static __device__ __forceinline__ void pack(const uint32_t *w, uint32_t (*o)[kWords]) {
        for (int t = 0; t < 4; ++t) o[0][t] = w[t];
    }
    static __device__ __forceinline__ void unpack(const uint32_t (*o)[kWords], uint32_t *w) {
        for (int t = 0; t < 4; ++t) w[t] = o[0][t];
    }
};
template <> struct ValuePieces<128> {
    static constexpr int kPieces = 2, kWords = 2;
    static __device__ __forceinline__ void pack(const uint32_t *w, uint32_t (*o)[kWords]) {
        for (int p = 0; p < 2; ++p) {
            o[0][p] = (w[2 * p] & 0xFFFFu) | (w[2 * p + 1] << 16);
            o[1][p] = (w[2 * p] >> 16) | (w[2 * p + 1] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void unpack(const uint32_t (*o)[kWords], uint32_t *w) {
        for (int p = 0; p < 2; ++p) {
            w[2 * p] = (o[0][p] & 0xFFFFu) | (o[1][p] << 16);
            w[2 * p + 1] = (o[0][p] >> 16) | (o[1][p] & 0xFFFF0000u);
        }
    }
};
template <> struct ValuePieces<64> {
    static constexpr int kPieces = 4, kWords = 1;
    static __device__ __forceinline__ void pack(const uint32_t *w, uint32_t (*o)[kWords]) {
        for (int j = 0; j < 4; ++j) {
            uint32_t x = 0;
            for (int t = 0; t < 4; ++t) x |= ((w[t] >> (8 * j)) & 0xFFu) << (8 * t);
            o[j][0] = x;
        }
    }
    static __device__ __forceinline__ void unpack(const uint32_t (*o)[kWords], uint32_t *w) {
        for (int t = 0; t < 4; ++t) {
            uint32_t x = 0;
            for (int j = 0; j < 4; ++j) x |= ((o[j][0] >> (8 * t)) & 0xFFu) << (8 * j);
            w[t] = x;
        }
    }
};

// Where one thread works: a quad of slots of a sequence and head, and 8 channels of it.
struct QuadAt {
    int seq, head, layer, off, n;  // n: rows this call moves for the sequence
    int64_t slot0, first;          // first slot of the quad, slot of row 0
    int chunk, page;               // page: of the quad (a quad never crosses one), or -1
    int t0;                        // slot within the page
    bool any;
};

template <int D>
__device__ __forceinline__ QuadAt quad_at(const KvParams &P) {
    constexpr int kChunks = D / 8;
    QuadAt q;
    uint32_t u = blockIdx.x;
    const uint32_t i = u % uint32_t(P.quad_blocks) * (kKvThreads / kChunks) + threadIdx.x / kChunks;
    u /= uint32_t(P.quad_blocks);
    q.head = int(i / uint32_t(P.quads));
    q.seq = int(u % uint32_t(P.S));
    q.layer = P.layer_begin + int(u / uint32_t(P.S));
    q.off = P.seq_off[q.seq];
    q.n = max(P.seq_off[q.seq + 1] - q.off, 0);
    if (P.counts != nullptr) q.n = min(min(q.n, P.row_stride), max(P.counts[q.seq], 0));
    q.first = max((P.begin != nullptr ? P.begin : P.length)[q.seq], 0);
    q.chunk = threadIdx.x % kChunks;
    q.slot0 = ((q.first >> 2) + i % uint32_t(P.quads)) * 4;
    q.any = q.head < P.H && q.slot0 < q.first + q.n;
    q.page = q.any ? kv_page(P.pages + int64_t(q.seq) * P.max_pages, P.max_pages, P.n_pages,
                             P.page_shift, q.slot0)
                   : -1;
    q.t0 = int(q.slot0 & ((1 << P.page_shift) - 1));
    return q;
}

// new_length[b] = min(length[b] + rows committed, capacity).
__device__ __forceinline__ void write_length(const KvParams &P, int b) {
    const int n = min(min(max(P.seq_off[b + 1] - P.seq_off[b], 0), P.row_stride), max(P.counts[b], 0));
    P.new_length[b] = int(min(int64_t(max(P.length[b], 0)) + n, int64_t(P.max_pages) << P.page_shift));
}

template <int D, typename TIn>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(KvParams P) {
    constexpr int kChunks = D / 8, kBlocks = D / 32;
    typedef KvAt<D> At;
    if (P.new_length != nullptr && blockIdx.x == gridDim.x - 1)
        for (int b = threadIdx.x; b < P.S; b += kKvThreads) write_length(P, b);
    const QuadAt q = quad_at<D>(P);
    // the lanes of a row leave together (they share the quad), so the exchanges below are whole
    if (!q.any || q.page < 0) return;
    const int lane = threadIdx.x & 63;
    const uint64_t row_lanes = (kChunks == 64 ? ~0ull : (1ull << kChunks) - 1) << (lane & ~(kChunks - 1));
    uint32_t kw[4], vw[4], ke[4], ve[4];
    bool there[4];
    int src[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t i = q.slot0 + t - q.first;
        there[t] = i >= 0 && i < q.n;
        src[t] = there[t] ? int(i) : 0;
        if (P.rows != nullptr && there[t]) {
            src[t] = P.rows[int64_t(q.seq) * P.row_stride + i];
            there[t] = src[t] >= 0 && src[t] < P.seq_off[q.seq + 1] - q.off;
        }
        src[t] = there[t] ? src[t] : 0;  // the sequence has a row 0: it has q.n rows
    }
    // all rows are asked for before the first is looked at
    float kx[4][8], vx[4][8];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t at = ((int64_t(q.layer) * P.T + q.off + src[t]) * P.H + q.head) * D + 8 * q.chunk;
        load8(static_cast<const TIn *>(P.k) + at, kx[t]);
        load8(static_cast<const TIn *>(P.v) + at, vx[t]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        kw[t] = vw[t] = ke[t] = ve[t] = 0;
        if (!there[t]) continue;
        const float *x = kx[t], *y = vx[t];
        const uint32_t mk = magnitude8(x), mv = magnitude8(y);
        if ((__ballot(mk >= 0x7F800000u || mv >= 0x7F800000u) & row_lanes) != 0) {
            ke[t] = kPoison;  // NaN key, zero value
            ve[t] = kScaleBias - kScaleMax;
            continue;
        }
        ke[t] = uint32_t(kv_scale_exp(quad_max(mk)) + kScaleBias);
        ve[t] = uint32_t(kv_scale_exp(quad_max(mv)) + kScaleBias);
        kw[t] = encode8(x, unit_of(ke[t]));
        vw[t] = encode8(y, unit_of(ve[t]));
    }
    const int64_t slab = kv_slab(q.layer, P.n_pages, q.page, P.H, q.head) << P.page_shift;
    uint8_t *kc = P.kc + slab * (D / 2), *vc = P.vc + slab * (D / 2);
    uint8_t *ks = P.ks + slab * kBlocks, *vs = P.vs + slab * kBlocks;
    const bool all = there[0] && there[1] && there[2] && there[3];
    const int block = q.chunk >> 2;
    const bool leader = (q.chunk & 3) == 0;  // one lane of the scale block
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (!there[t]) continue;
        *reinterpret_cast<uint32_t *>(kc + At::key(q.t0 + t, q.chunk)) = kw[t];
        if (leader) ks[At::key_scale(q.t0 + t, block)] = uint8_t(ke[t]);
    }
    typedef ValuePieces<D> VP;
    uint32_t piece[VP::kPieces][VP::kWords];
    VP::pack(vw, piece);
    if (all) {
#pragma unroll
        for (int j = 0; j < VP::kPieces; ++j) {
            uint8_t *p = vc + At::value(q.t0, q.chunk * VP::kPieces + j);
            if constexpr (VP::kWords == 4)
                *reinterpret_cast<uint4 *>(p) = make_uint4(piece[j][0], piece[j][1], piece[j][2], piece[j][3]);
            else if constexpr (VP::kWords == 2)
                *reinterpret_cast<uint2 *>(p) = make_uint2(piece[j][0], piece[j][1]);
            else
                *reinterpret_cast<uint32_t *>(p) = piece[j][0];
        }
        if (leader)
            *reinterpret_cast<uint32_t *>(vs + At::value_scale(q.t0, block)) =
                ve[0] | (ve[1] << 8) | (ve[2] << 16) | (ve[3] << 24);
        return;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (!there[t]) continue;
#pragma unroll
        for (int j = 0; j < VP::kPieces; ++j) {
            uint8_t *p = vc + At::value(q.t0 + t, q.chunk * VP::kPieces + j);
            if constexpr (D == 256)
                *reinterpret_cast<uint32_t *>(p) = vw[t];
            else if constexpr (D == 128)
                *reinterpret_cast<uint16_t *>(p) = uint16_t(vw[t] >> (16 * j));
            else
                *p = uint8_t(vw[t] >> (8 * j));
        }
        if (leader) vs[At::value_scale(q.t0 + t, block)] = uint8_t(ve[t]);
    }
}

template <int D, typename TIn>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvParams P) {
    constexpr int kBlocks = D / 32;
    typedef KvAt<D> At;
    const QuadAt q = quad_at<D>(P);
    if (!q.any) return;
    const int block = q.chunk >> 2;
    float x[4][8] = {}, y[4][8] = {};
    if (q.page >= 0) {
        const int64_t slab = kv_slab(q.layer, P.n_pages, q.page, P.H, q.head) << P.page_shift;
        const uint8_t *kc = P.kc + slab * (D / 2), *vc = P.vc + slab * (D / 2);
        const uint8_t *ks = P.ks + slab * kBlocks, *vs = P.vs + slab * kBlocks;
        typedef ValuePieces<D> VP;
        uint32_t piece[VP::kPieces][VP::kWords], vw[4];
#pragma unroll
        for (int j = 0; j < VP::kPieces; ++j) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(vc + At::value(q.t0, q.chunk * VP::kPieces + j));
#pragma unroll
            for (int i = 0; i < VP::kWords; ++i) piece[j][i] = p[i];
        }
        VP::unpack(piece, vw);
        const uint32_t ve = *reinterpret_cast<const uint32_t *>(vs + At::value_scale(q.t0, block));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t e = ks[At::key_scale(q.t0 + t, block)];
            decode8(*reinterpret_cast<const uint32_t *>(kc + At::key(q.t0 + t, q.chunk)), unit_of(e), x[t]);
            if (e == kPoison)
                for (int i = 0; i < 8; ++i) x[t][i] = __builtin_nanf("");
            decode8(vw[t], unit_of((ve >> (8 * t)) & 0xFFu), y[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t i = q.slot0 + t - q.first;
        if (i < 0 || i >= q.n) continue;
        const int64_t at = ((int64_t(q.layer) * P.T + q.off + i) * P.H + q.head) * D + 8 * q.chunk;
        store8(static_cast<TIn *>(P.k) + at, x[t]);
        store8(static_cast<TIn *>(P.v) + at, y[t]);
    }
}

// The lengths alone: nothing to move, or they take the place of what the append reads.
__global__ void kv_length_kernel(KvParams P) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < P.S) write_length(P, b);
}

static KvParams kv_params(const gdn_kv_args *a) {
    KvParams P{};
    P.k = a->k;
    P.v = a->v;
    P.kc = a->k_codes;
    P.ks = a->k_scales;
    P.vc = a->v_codes;
    P.vs = a->v_scales;
    P.pages = a->pages;
    P.length = a->length;
    P.seq_off = a->seq_offsets;
    P.S = a->n_seqs;
    P.H = a->n_kv_heads;
    P.T = a->n_tokens;
    P.n_pages = a->n_pages;
    P.max_pages = a->max_pages;
    P.page_shift = log2_exact(a->page_tokens);
    P.layer_begin = a->layer_begin;
    return P;
}

template <int D, typename TIn>
static void launch_move(const KvParams &P, bool read, uint32_t blocks, hipStream_t s) {
    if (read)
        hipLaunchKernelGGL((kv_read_kernel<D, TIn>), dim3(blocks), dim3(kKvThreads), 0, s, P);
    else
        hipLaunchKernelGGL((kv_append_kernel<D, TIn>), dim3(blocks), dim3(kKvThreads), 0, s, P);
}

// Moves up to `longest` rows of every sequence between k, v and the pools.
static gdn_status move_rows(const gdn_kv_args *a, KvParams P, int64_t longest, bool read,
                            const char *who, hipStream_t s) {
    const void *rows[] = {a->k, a->v};
    gdn_status st = check_aligned16(rows, 2, who, "k/v");
    if (st != GDN_OK) return st;
    const int64_t per_block = kKvThreads / (a->head_dim / 8);
    // Rows of a sequence may start inside a quad: one quad more than they fill.  The quads of all
    // heads follow one another, so that few rows a head still fill their workgroups.
    const int64_t quads = (longest + 3) / 4 + 1, all = quads * a->n_kv_heads;
    const int64_t blocks = (all + per_block - 1) / per_block * a->n_seqs * a->n_layers;
    P.quads = int32_t(quads);
    P.quad_blocks = int32_t((all + per_block - 1) / per_block);
    if (all > INT32_MAX || blocks > kMaxBlocks) return fail(GDN_EINVAL, "%s: too many workgroups", who);
    const bool bf = a->in_dtype == GDN_BF16;
    const uint32_t nb = uint32_t(blocks);
    switch (a->head_dim) {
        case 64: bf ? launch_move<64, bf16_t>(P, read, nb, s) : launch_move<64, float>(P, read, nb, s); break;
        case 128: bf ? launch_move<128, bf16_t>(P, read, nb, s) : launch_move<128, float>(P, read, nb, s); break;
        default: bf ? launch_move<256, bf16_t>(P, read, nb, s) : launch_move<256, float>(P, read, nb, s); break;
    }
    GDN_LAUNCH_CHECK(who);
    return GDN_OK;
}

static bool disjoint(const int32_t *x, int64_t nx, const int32_t *y, int64_t ny) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return a + size_t(nx) * 4 <= b || b + size_t(ny) * 4 <= a;
}

static int64_t longest_of(const gdn_kv_args *a, const int32_t *offs) {
    int64_t n = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b) n = std::max<int64_t>(n, offs[b + 1] - offs[b]);
    return n;
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_kv_append(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                                    void *stream) {
    clear_error();
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, "gdn_kv_append", true, empty);
    if (st != GDN_OK || empty) return st;
    return move_rows(a, kv_params(a), longest_of(a, host_seq_offsets), false, "gdn_kv_append",
                     static_cast<hipStream_t>(stream));
}

extern "C" gdn_status gdn_kv_read(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                                  const int32_t *begin, void *stream) {
    clear_error();
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, "gdn_kv_read", true, empty);
    if (st != GDN_OK || empty) return st;
    KvParams P = kv_params(a);
    P.begin = begin;
    return move_rows(a, P, longest_of(a, host_seq_offsets), true, "gdn_kv_read",
                     static_cast<hipStream_t>(stream));
}

extern "C" gdn_status gdn_kv_commit(const gdn_kv_args *a, const int32_t *host_seq_offsets,
                                    const int32_t *rows, int32_t row_stride, const int32_t *counts,
                                    int32_t *new_length, void *stream) {
    clear_error();
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, "gdn_kv_commit", true, empty);
    if (st != GDN_OK) return st;
    if (a->n_seqs == 0) return GDN_OK;
    if (counts == nullptr || new_length == nullptr)
        return fail(GDN_EINVAL, "gdn_kv_commit: null counts/new_length");
    if (rows != nullptr && row_stride < 1)
        return fail(GDN_EINVAL, "gdn_kv_commit: row_stride %d", row_stride);
    hipStream_t s = static_cast<hipStream_t>(stream);
    KvParams P = kv_params(a);
    P.rows = rows;
    P.counts = counts;
    P.row_stride = rows != nullptr ? row_stride : a->n_tokens;
    // A sequence's new length may take the place of what only it reads, its length or its count;
    // anywhere else among the inputs it would be another's.
    const int64_t S = a->n_seqs;
    const bool in_place = new_length == a->length || new_length == counts;
    if ((new_length != a->length && !disjoint(new_length, S, a->length, S)) ||
        (new_length != counts && !disjoint(new_length, S, counts, S)) ||
        !disjoint(new_length, S, a->seq_offsets, S + 1) || !disjoint(new_length, S, a->pages, S * a->max_pages) ||
        (rows != nullptr && !disjoint(new_length, S, rows, S * row_stride)))
        return fail(GDN_EINVAL, "gdn_kv_commit: new_length may be length or counts, but not overlap the inputs otherwise");
    // A launch of its own for one integer a sequence takes as long as the append of a tree (22 rows,
    // 8 heads of 128, 16 layers, with the read: 19.1 us in three launches, 15.1 in two), so the
    // append writes the lengths, unless a workgroup may still have to read what they overwrite.
    const bool apart = rows != nullptr && !in_place;
    if (rows != nullptr && !empty) {
        if (apart) P.new_length = new_length;
        st = move_rows(a, P, std::min<int64_t>(longest_of(a, host_seq_offsets), row_stride), false,
                       "gdn_kv_commit", s);
        if (st != GDN_OK || apart) return st;
    }
    P.new_length = new_length;
    hipLaunchKernelGGL(kv_length_kernel, dim3((a->n_seqs + 255) / 256), dim3(256), 0, s, P);
    GDN_LAUNCH_CHECK("kv_length_kernel");
    return GDN_OK;
}
