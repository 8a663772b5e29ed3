// Page selection of the sparse attention (gfx950): bounds of the cached keys a page, scores of pages by
// them, and the best pages of a selection.  The rules are in gdn_tree.h.
//
// Bounds.  A wave takes a page of a head as the cache holds it and keeps the largest and smallest value of 32
// channels a lane, then hands on the half of them at each of four exchanges.  Stored keys are 4-bit floats times
// a power of two, so their limits are bf16 numbers.  Prompts of 110000 tokens, 8 heads of 128: 69 MB in 17.8 us,
// 3.9 TB/s (22.1 with all 32 kept through the exchanges, and a load waiting for the last); about two thirds of the time the
// vector units' for an instruction a value and its two comparisons.
//
// Scores.  With q+ = max(q, 0) and q- = min(q, 0), score = sum_c q+_c largest_c + q-_c smallest_c: a matrix
// product of pages x 2 d by 2 d x rows, in bf16 on the matrix cores (fp32 q as three bf16 terms), 64 terms at
// a time, whose sums are added in fp32.  Such a score is off by at most g |q| |(largest, smallest)|, the
// Euclidean lengths, with g a few more than 64 times 2^-23 (Cauchy-Schwarz on the magnitudes of the terms).
// The choice is made by what that leaves sure: with t the k-th best score and t' the next, the k best
// are known where t - t' > 2 e, e the largest error.  Otherwise the pages from t - 2 e to t' + 2 e are scored
// again in fp64: a limit has two significant bits, so products have 10 bits with bf16 q and 26 with fp32, and 256 of
// them have an exact sum where they lie within 35 (19) binades of one another.  Then the selection is that of exact
// scores.  Beyond, the sums round, in the order of the path that takes them (few pages or many), and pages nearer
// than that may swap with the launch's shape.  With all pages in fp64 trees of 22 nodes, 48 heads, on 8 caches of 16000 to
// 65000 slots in pages of 64 took 125 us, at the fp64 matrix rate (66 TFLOP/s); now 35, the join included.
// Where all scores are equal (a q of zeros, limits alike) every page is in doubt, and a call of selection and attention
// takes 425 us instead of 88 for those trees, 111 instead of 51 for 32 single tokens.
//
// Limits are read as they lie in memory, 64 bytes of a page by four neighbouring lanes, and brought to the
// operands' lanes by 4 x 4 transpositions within them; read 16 bytes here and there, as the operands want
// them, 2000 pages of 256 channels took a workgroup 80 us, now 59.  What a compute unit then gets is 35 GB/s:
// decode of 32 caches, 8 heads, reads 49 MB of limits in 9 us of the kernel's 24, at the rate of a copy; the
// start (lengths, then table and q, then limits, each waiting for the last) takes 3.5, the choice 5.
// With 256 channels a lane's limits take 64 registers beside q's operands; of the 128 that 16 (or twice 8) waves a
// compute unit leave, 20 vector registers spill with bf16 q and 31 with fp32, and no tile is asked for ahead.
//
// Best pages.  Keys are the scores as integers of the same order.  Every wave holds them all in its registers
// and counts those at or above a threshold of its own, so that a pass of 16 waves narrows the range of the
// k-th to a 17th; three or four passes find a threshold with k above it.  Elements stay in the table's
// order, so that equal scores go to the lower entry and the result is ascending without a sort.
#include <algorithm>

#include "attention_work.h"
#include "kv_internal.h"
#include "mfma_common.h"

namespace gdn {

struct SelectParams {
    const void *q;
    const uint16_t *bounds;
    const int32_t *pages, *length, *seq_off;
    int32_t *selected;
    uint32_t *best_key; // [unit][split][room]: scores in order
    int32_t *best_at;   // [unit][split][room]
    int32_t *best_n;    // [unit][split]: how many there are
    float *best_error;  // [unit][split]: how far their scores may be off
    SparseShape shape;
    int32_t S, H, G, T, n_pages, max_pages, page_shift, layer_begin, selections, splits, first, last, spare, batch;
    int32_t room;  // pages a share hands on
};

struct BoundsParams {
    const uint8_t *kc, *ks;
    uint16_t *bounds;
    const int32_t *pages, *length, *seq_off;
    int32_t S, H, n_pages, max_pages, page_shift, layer_begin, pages_each;
    uint32_t units;
};

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int16_t s16x2 __attribute__((ext_vector_type(2)));

// A workgroup has W waves, 16 or 8.
constexpr int kHeld = kMaxTopPages + kSparePages;
template <int W> struct Sizes {
    static constexpr int threads = 64 * W;
    // Elements chosen among at a time, two a thread: the best so far and a chunk of pages.
    static constexpr int elements = 2 * threads, chunk = elements - kHeld;
    static_assert(chunk > 0 && chunk % 16 == 0, "whole tiles of pages");
    static_assert(W <= 16, "a row of lanes has a count of every wave");
};
static_assert(Sizes<16>::elements == kJoinPages, "");
constexpr int kMaxBatch = 16;  // row tiles in LDS at a time

// Keys: scores as integers of the same order, and what is not a score.
constexpr uint32_t kNone = 0, kAbsent = 1, kUnknown = ~0u;  // no element; no page; no number
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 is 0
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
    return __uint_as_float(key == kAbsent ? 0xFF800000u : (key >> 31) != 0 ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t b = uint64_t(__double_as_longlong(x + 0.0));
    return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}

template <int CTRL> __device__ __forceinline__ uint32_t row_take(uint32_t x) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL> __device__ __forceinline__ void row_max(double &x) {
    x = fmax(x, __hiloint2double(int(row_take<CTRL>(uint32_t(__double2hiint(x)))),
                                 int(row_take<CTRL>(uint32_t(__double2loint(x))))));
}
template <int CTRL> __device__ __forceinline__ void row_sum(double &x) {
    x += __hiloint2double(int(row_take<CTRL>(uint32_t(__double2hiint(x)))),
                          int(row_take<CTRL>(uint32_t(__double2loint(x)))));
}
template <int CTRL> __device__ __forceinline__ void row_max(float &x) {
    x = fmaxf(x, __uint_as_float(row_take<CTRL>(__float_as_uint(x))));
}
template <int CTRL> __device__ __forceinline__ void row_max(uint32_t &x) { x = max(x, row_take<CTRL>(x)); }
// Largest of a row of 16 lanes, in all of them.
template <typename X> __device__ __forceinline__ void row_max16(X &x) {
    row_max<0xB1>(x);
    row_max<0x4E>(x);
    row_max<0x141>(x);
    row_max<0x140>(x);
}

// The thread's number, which the compiler takes for a new one: what it would compute from it ahead of the loops
// over chunks and tiles, it would have to keep or spill in them.
__device__ __forceinline__ int fresh_thread() {
    int x = threadIdx.x;
    asm volatile("" : "+v"(x));
    return x;
}

// Largest of the wave, in all lanes: within rows of 16 lanes, then the rows' onwards.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    row_max16(x);
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x142, 0xA, 0xF, false)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x143, 0xC, 0xF, false)));
    return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ uint32_t wave_min(uint32_t x) { return ~wave_max(~x); }

// Sum of a count that is the same in a wave's lanes over the waves before this one, and over all.
template <int W> __device__ __forceinline__ int before(int count, int *sums, int &all) {
    const int tid = fresh_thread(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    __syncthreads();  // the last sums have been read
    if ((tid & 63) == 0) sums[wave] = count;
    __syncthreads();
    int x = sums[tid & (W - 1)], run = x;  // a row of lanes has them all
    run += __builtin_amdgcn_update_dpp(0, run, 0x111, 0xF, 0xF, true);
    run += __builtin_amdgcn_update_dpp(0, run, 0x112, 0xF, 0xF, true);
    run += __builtin_amdgcn_update_dpp(0, run, 0x114, 0xF, 0xF, true);
    run += __builtin_amdgcn_update_dpp(0, run, 0x118, 0xF, 0xF, true);
    all = __builtin_amdgcn_readlane(run, W - 1);
    return __builtin_amdgcn_readlane(run - x, wave);
}

// Where a unit's selection is, and how many pages compete for it.
struct UnitOf {
    int seq, head, layer, off, n_new, first_token, tokens;  // tokens <= 0: no such selection
    int full, mid;                                          // mid: pages to choose, of full - first - last
    int32_t *out;
};
__device__ __forceinline__ UnitOf unit_of(const SelectParams &P, uint32_t i) {
    UnitOf u;
    u.head = int(i % uint32_t(P.H));
    i /= uint32_t(P.H);
    const int selection = int(i % uint32_t(P.selections));
    i /= uint32_t(P.selections);
    u.seq = int(i % uint32_t(P.S));
    u.layer = P.layer_begin + int(i / uint32_t(P.S));
    u.off = P.seq_off[u.seq];
    u.n_new = P.seq_off[u.seq + 1] - u.off;
    const int each = sparse_tokens(P.shape, u.n_new);
    u.first_token = selection * each;
    u.tokens = min(each, u.n_new - u.first_token);
    u.full = length_of(P.length[u.seq], int64_t(P.max_pages) << P.page_shift) >> P.page_shift;
    u.mid = P.shape.top - P.first - P.last;
    u.out = P.selected + ((int64_t(u.layer) * P.T + u.off + u.first_token) * P.H + u.head) * P.shape.top;
    return u;
}

// Entries that need no scores: all of few pages, or the first and last of many.
template <int W> __device__ __forceinline__ void write_kept(const SelectParams &P, const UnitOf &u) {
    const int top = P.shape.top;
    for (int i = threadIdx.x; i < top; i += Sizes<W>::threads) {
        if (u.full <= top)
            u.out[i] = i < u.full ? i : -1;
        else if (i < P.first)
            u.out[i] = i;
        else if (i >= top - P.last)
            u.out[i] = u.full - top + i;
    }
}

// Pages of share `split`: table entries [lo, hi).
__device__ __forceinline__ void share_of(const SelectParams &P, const UnitOf &u, int split, int &lo, int &hi) {
    const int64_t n = u.full - P.first - P.last;
    lo = P.first + int(n * split / P.splits);
    hi = P.first + int(n * (split + 1) / P.splits);
}

// q as bf16 terms ("planes") whose sum it is.
template <typename T> struct QPlanes {
    static constexpr int n = 1;
};
template <> struct QPlanes<float> {
    static constexpr int n = 3;
};
// How far a score is off, relative to the product of the lengths: 64 terms of the first plane in one sum, the
// other planes' 2^-7 of it, an addition for every 32 channels; and what the lengths' own rounding takes.
template <int D> constexpr float score_error() { return 1.05f * (64.f + 4.f + D / 32) * 0x1p-23f; }

template <int D, typename TIn> struct Tiles {
    static constexpr int planes = QPlanes<TIn>::n;
    static constexpr int stride = 2 * planes * D + 8;  // bf16 numbers between rows: q+ and q-, by plane
    static constexpr int bytes = 16 * stride * 2;      // of 16 rows
};

// What a workgroup keeps in LDS of the pages it chooses among; behind it, q of as many row tiles as the
// launch has room for.
template <int W> struct Lds {
    static constexpr int n = Sizes<W>::elements;
    __align__(16) uint32_t key[n];
    int32_t at[n];    // table entry
    int32_t list[n];  // table entries of pages to score in fp64; whether each is taken
    union {
        __align__(16) uint64_t exact[n];
        float size[n];  // squared length of the limits
    };
    uint8_t leave[kMaxBatch * 16];
    uint32_t q_size, page_size;  // bits of the largest |q|^2 of the rows, of the limits'
    int counts[2][W], sums[W];
};
static_assert(sizeof(Lds<16>) % 16 == 0 && sizeof(Lds<8>) % 16 == 0, "q behind it is aligned");

// Where row `row` of the unit's (token, query head of the kv head) is in q.
template <int D, typename TIn>
__device__ __forceinline__ const TIn *row_of(const SelectParams &P, const UnitOf &u, int row) {
    const int token = row / P.G, hq = u.head * P.G + row - token * P.G;
    return static_cast<const TIn *>(P.q) +
           ((int64_t(u.layer) * P.T + u.off + u.first_token + token) * (P.H * P.G) + hq) * D;
}

// fp64 scores of up to kFew pages: 16 lanes a row, whose D / 16 channels each are brought to fp64 once for all
// pages, and the pages' limits in LDS, behind the scores.
constexpr int kFew = 7;
template <int W, int D, typename TIn>
__device__ __forceinline__ void exact_scores_few(const SelectParams &P, const UnitOf &u, int32_t *list, int n,
                                                 uint64_t *exact) {
    constexpr int CH = D / 16, QW = CH * int(sizeof(TIn)) / 4, T = Sizes<W>::threads;
    static_assert(kFew < 8 && 8 * 8 + kFew * 4 * D <= 8 * Sizes<W>::elements, "eight scores and the limits");
    uint16_t *limits = reinterpret_cast<uint16_t *>(exact + 8);
    const int tid = fresh_thread(), part = tid & 15, rows = u.tokens * P.G;
    uint32_t next[QW];
    auto load = [&](int row) {
        const uint2 *q = reinterpret_cast<const uint2 *>(row_of<D, TIn>(P, u, min(row, rows - 1)) + CH * part);
#pragma unroll
        for (int c = 0; c < QW / 2; ++c) {
            next[2 * c] = q[c].x;
            next[2 * c + 1] = q[c].y;
        }
    };
    load(tid >> 4);
    __syncthreads();
    if (tid < n) {  // entries to page ids, -1: not there
        const int id = P.pages[int64_t(u.seq) * P.max_pages + list[tid]];
        list[tid] = unsigned(id) < unsigned(P.n_pages) ? id : -1;
        exact[tid] = 0;
    }
    __syncthreads();
    const uint16_t *bounds = P.bounds + kv_slab(u.layer, P.n_pages, 0, P.H, u.head) * (2 * D);
    for (int i = tid; i < n * (D / 4); i += T) {  // 8 limits each
        const int page = i / (D / 4), at = 8 * (i % (D / 4)), id = list[page];
        if (id < 0) continue;
        const u32x4 x = *reinterpret_cast<const u32x4 *>(bounds + int64_t(id) * P.H * (2 * D) + at);
        *reinterpret_cast<u32x4 *>(limits + page * (2 * D) + at) = x;
        bool unknown = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = x[e];
            unknown |= !(bf16_lo(w) == bf16_lo(w)) || !(bf16_hi(w) == bf16_hi(w));
        }
        if (unknown)
            atomicMax((unsigned long long *)&exact[page], (unsigned long long)order_of(double(__builtin_inff())));
    }
    __syncthreads();
    // the waves have as many turns each, so that all lanes take part in the sums
    for (int from = 0; from < rows; from += T / 16) {
        double x[CH];
        bool bad = false;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float y;
            if constexpr (sizeof(TIn) == 4)
                y = __uint_as_float(next[c]);
            else
                y = (c & 1) != 0 ? bf16_hi(next[c / 2]) : bf16_lo(next[c / 2]);
            const bool finite = fabsf(y) < __builtin_inff();
            bad |= !finite;
            x[c] = double(finite ? y : 0.f);
        }
        load(from + T / 16 + (tid >> 4));
        const bool leave = ((__ballot(bad) >> (tid & 48)) & 0xFFFFu) != 0;
        for (int page = 0; page < n; ++page) {
            if (list[page] < 0) continue;
            const uint16_t *most = limits + page * (2 * D) + CH * part, *least = most + D;
            double sum = 0.0;
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
                const uint2 m = *reinterpret_cast<const uint2 *>(most + c), l = *reinterpret_cast<const uint2 *>(least + c);
                // one term of a channel is 0: not worth its conversion, which the fp64 unit takes longest for
                sum = fma(double(x[c] > 0.0 ? bf16_lo(m.x) : bf16_lo(l.x)), x[c], sum);
                sum = fma(double(x[c + 1] > 0.0 ? bf16_hi(m.x) : bf16_hi(l.x)), x[c + 1], sum);
                sum = fma(double(x[c + 2] > 0.0 ? bf16_lo(m.y) : bf16_lo(l.y)), x[c + 2], sum);
                sum = fma(double(x[c + 3] > 0.0 ? bf16_hi(m.y) : bf16_hi(l.y)), x[c + 3], sum);
            }
            row_sum<0xB1>(sum);
            row_sum<0x4E>(sum);
            row_sum<0x141>(sum);
            row_sum<0x140>(sum);
            sum = !(sum == sum) ? double(__builtin_inff()) : leave ? -double(__builtin_inff()) : sum;
            sum = fmax(sum, __shfl_xor(sum, 16));
            sum = fmax(sum, __shfl_xor(sum, 32));
            if ((tid & 63) == 0)
                atomicMax((unsigned long long *)&exact[page], (unsigned long long)order_of(sum));
        }
    }
    __syncthreads();
}

// fp64 scores of the n pages at table entries list[], as ordered integers into exact[]: a wave takes 16
// pages and 16 rows at a time.  A page that is not there has 0, one whose limits are not numbers +inf.
template <int W, int D, typename TIn>
__device__ __forceinline__ void exact_scores(const SelectParams &P, const UnitOf &u, const int32_t *list, int n,
                                             uint64_t *exact) {
    const int tid = fresh_thread(), lane = tid & 63, wave = tid >> 6, col = lane & 15, kq = lane >> 4;
    const int rows = u.tokens * P.G, row_tiles = (rows + 15) / 16, jobs = (n + 15) / 16 * row_tiles;
    const int32_t *table = P.pages + int64_t(u.seq) * P.max_pages;
    for (int i = tid; i < n; i += Sizes<W>::threads) exact[i] = 0;
    __syncthreads();
    for (int job = wave; job < jobs; job += W) {
        const int tile = job / row_tiles, row = (job - tile * row_tiles) * 16 + col;
        const int id = table[list[min(tile * 16 + col, n - 1)]];
        const bool there = unsigned(id) < unsigned(P.n_pages);
        const uint32_t pages = uint32_t(__ballot(there)) & 0xFFFFu;
        const uint16_t *b = P.bounds + kv_slab(u.layer, P.n_pages, there ? id : 0, P.H, u.head) * (2 * D) + 8 * kq;
        const TIn *q = row_of<D, TIn>(P, u, min(row, rows - 1)) + 8 * kq;
        f64x4 up = {0.0, 0.0, 0.0, 0.0}, down = up;
        bool bad = false;
        // 8 channels at a time, the next ones under way
        u32x4 qw[2], mw, lw;
        auto load = [&](int t) {
            qw[0] = reinterpret_cast<const u32x4 *>(q + t)[0];
            if constexpr (sizeof(TIn) == 4) qw[1] = reinterpret_cast<const u32x4 *>(q + t)[1];
            mw = *reinterpret_cast<const u32x4 *>(b + t);
            lw = *reinterpret_cast<const u32x4 *>(b + D + t);
        };
        load(0);
#pragma unroll 1
        for (int t = 0; t < D; t += 32) {
            const u32x4 y0 = qw[0], y1 = qw[1], m = mw, l = lw;
            load(min(t + 32, D - 32));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x;
                if constexpr (sizeof(TIn) == 4)
                    x = __uint_as_float(e < 4 ? y0[e] : y1[e - 4]);
                else
                    x = (e & 1) != 0 ? bf16_hi(y0[e / 2]) : bf16_lo(y0[e / 2]);
                const bool finite = fabsf(x) < __builtin_inff();
                bad |= !finite;
                x = finite ? x : 0.f;
                const double a = double((e & 1) != 0 ? bf16_hi(m[e / 2]) : bf16_lo(m[e / 2]));
                const double c = double((e & 1) != 0 ? bf16_hi(l[e / 2]) : bf16_lo(l[e / 2]));
                up = __builtin_amdgcn_mfma_f64_16x16x4f64(a, double(fmaxf(x, 0.f)), up, 0, 0, 0);
                down = __builtin_amdgcn_mfma_f64_16x16x4f64(c, double(fminf(x, 0.f)), down, 0, 0, 0);
            }
        }
        const uint64_t any = __ballot(bad);
        const bool leave = row >= rows || (((any | any >> 32) | (any | any >> 32) >> 16) >> col & 1) != 0;
        // Lane (col, kq) has rows 4 v + kq, the pages, of its column.
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            double x = up[v] + down[v];
            x = !(x == x) ? double(__builtin_inff()) : leave ? -double(__builtin_inff()) : x;
            row_max16(x);
            const int page = 4 * v + kq, i = tile * 16 + page;
            if (col == 0 && i < n && ((pages >> page) & 1u))
                atomicMax((unsigned long long *)&exact[i], (unsigned long long)order_of(x));
        }
    }
    __syncthreads();
}

// Calls put(position, element) for every element whose key take() picks, in order; returns their number.
// A thread has two neighbouring elements.
template <int W, typename F, typename G>
__device__ __forceinline__ int place_taken(const uint32_t *keys, int *sums, F take, G put) {
    const int tid = fresh_thread(), lane = tid & 63;
    const uint2 key = *reinterpret_cast<const uint2 *>(keys + 2 * tid);
    const bool a = take(key.x), b = take(key.y);
    const uint64_t in_a = __ballot(a), in_b = __ballot(b), below = (1ull << lane) - 1;
    int all, to = before<W>(__popcll(in_a) + __popcll(in_b), sums, all);
    to += __popcll(in_a & below) + __popcll(in_b & below);
    put(to, to + (a ? 1 : 0), a, b, key, 2 * tid);
    return all;
}

// How far the scores of the pages so far may be off, elements [fresh, have) the newest, with their limits'
// lengths in lds.size.
template <int W, int D> __device__ __forceinline__ float error_of(Lds<W> &lds, int fresh, int have) {
    const int tid = fresh_thread();
    uint32_t size = 0;
    for (int i = fresh + tid; i < have; i += Sizes<W>::threads) {
        // limits that are not numbers, or too large for their length: the score is not known
        const uint32_t z = __float_as_uint(lds.size[i]);
        if (z < 0x7F800000u)
            size = max(size, z);
        else
            lds.key[i] = kUnknown;
    }
    size = wave_max(size);
    if ((tid & 63) == 0) atomicMax(&lds.page_size, size);
    __syncthreads();
    // what is too small to have a square counts as 2^-60
    return score_error<D>() * (sqrtf(__uint_as_float(lds.q_size)) + 0x1p-60f) *
           (sqrtf(__uint_as_float(lds.page_size)) + 0x1p-60f);
}

// Keeps the best of `have` elements at the front, in order: those that are surely or possibly among the k
// best, if that is no more than `cap`, else exactly the k best.  Behind the last the keys are kNone.  `error`:
// how far scores may be off.  Returns how many are kept.
template <int W, int D, typename TIn>
__device__ __forceinline__ int choose(const SelectParams &P, const UnitOf &u, Lds<W> &lds, int have, int k, int cap,
                                      float error) {
    constexpr int SL = Sizes<W>::elements / 256;
    if (have <= k) return have;
    const int tid = fresh_thread(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // ---- the k-th best ----------------------------------------------------------------------
    u32x4 x[SL];  // elements 256 i + 4 lane ..
    uint32_t low = kUnknown, high = kNone;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
        x[i] = u32x4{kNone, kNone, kNone, kNone};
        if (256 * i < have) x[i] = *reinterpret_cast<const u32x4 *>(lds.key + 256 * i + 4 * lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            low = min(low, x[i][e] == kNone ? kUnknown : x[i][e]);
            high = max(high, x[i][e]);
        }
    }
    low = wave_min(low);
    high = wave_max(high);
    auto count = [&](auto f) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            if (256 * i >= have) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) c += __popcll(__ballot(f(x[i][e])));
        }
        return c;
    };
    const bool all_known = high != kUnknown && error < __builtin_inff();
    uint32_t t = low;  // with exactly k keys at or above it, or equal keys to be taken in part
    bool whole = false;
    for (int pass = 0; low < high; ++pass) {
        const uint32_t width = high - low, step = width / (W + 1) + 1;
        auto at = [&](int w) { return low + min(uint32_t(w + 1) * step, width); };
        const uint32_t mine = at(wave);
        const int c = count([&](uint32_t key) { return key >= mine; });
        int *counts = lds.counts[pass & 1];
        if (lane == 0) counts[wave] = c;
        __syncthreads();
        const int of = counts[lane & (W - 1)];
        const uint32_t equal = uint32_t(__ballot(of == k)) & ((1u << W) - 1);
        if (equal != 0) {
            t = at(__builtin_ctz(equal));
            whole = true;
            break;
        }
        const int m = __popc(uint32_t(__ballot(of > k)) & ((1u << W) - 1));  // thresholds with too many keys
        const uint32_t next_low = m > 0 ? at(m - 1) : low;
        if (m < W) high = at(m) - 1;
        low = next_low;
        t = low;
    }
    // ---- what the error leaves sure --------------------------------------------------------
    uint32_t worst = t, best = t;  // keys of the last taken and the first other
    if (whole) {
        worst = kUnknown;
        best = kNone;
#pragma unroll
        for (int i = 0; i < SL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                worst = min(worst, x[i][e] >= t ? x[i][e] : kUnknown);
                best = max(best, x[i][e] < t ? x[i][e] : kNone);
            }
        worst = wave_min(worst);
        best = wave_max(best);
    }
    const float gap = score_of(worst) - score_of(best);
    uint32_t in = kUnknown, out = kAbsent;  // sure above `in`, out below `out`
    if (all_known) {
        in = max(order_of(score_of(best) + 2.f * error), best);
        out = min(order_of(score_of(worst) - 2.f * error), worst);
    }
    const bool sure = all_known && gap > 2.f * error;
    if (sure) out = t;
    if (sure || count([&](uint32_t key) { return key >= out; }) <= cap) {
        // in place: an element moves to the left only, and all have been read before any is written
        return place_taken<W>(lds.key, lds.sums, [&](uint32_t key) { return key >= out; },
                           [&](int p, int q, bool a, bool b, uint2 key, int e) {
                               const int2 at = *reinterpret_cast<const int2 *>(lds.at + e);
                               __syncthreads();
                               if (a) {
                                   lds.key[p] = key.x;
                                   lds.at[p] = at.x;
                               }
                               if (b) {
                                   lds.key[q] = key.y;
                                   lds.at[q] = at.y;
                               }
                               __syncthreads();
                           });
    }
    // ---- the pages in doubt, in fp64 ---------------------------------------------------------
    auto doubtful = [&](uint32_t key) { return key >= out && key <= in; };
    const int wanted = k - count([&](uint32_t key) { return key > in; });
    int first_doubt = 0;  // of this thread's elements, if any
    const int maybe = place_taken<W>(lds.key, lds.sums, doubtful, [&](int p, int q, bool a, bool b, uint2, int e) {
        first_doubt = p;
        if (a) lds.list[p] = lds.at[e];
        if (b) lds.list[q] = lds.at[e + 1];
    });
    __syncthreads();
    // the matrix cores take 16 pages at once, in 1.7 us for 16 rows of 128 channels, the vector units a page
    if (maybe <= kFew)
        exact_scores_few<W, D, TIn>(P, u, lds.list, maybe, lds.exact);
    else
        exact_scores<W, D, TIn>(P, u, lds.list, maybe, lds.exact);
    for (int i = fresh_thread(); i < maybe; i += Sizes<W>::threads) {
        const uint64_t own = lds.exact[i];
        int rank = 0;
        for (int j = 0; j < maybe; ++j) {
            const uint64_t y = lds.exact[j];
            rank += y > own || (y == own && j < i) ? 1 : 0;
        }
        lds.list[i] = rank < wanted ? 1 : 0;
    }
    __syncthreads();
    // pages that are not taken leave
    {
        const int e = 2 * fresh_thread();
        const uint2 key = *reinterpret_cast<const uint2 *>(lds.key + e);
        const bool a = doubtful(key.x), b = doubtful(key.y);
        if (key.x < out || (a && lds.list[first_doubt] == 0)) lds.key[e] = kNone;
        if (key.y < out || (b && lds.list[first_doubt + (a ? 1 : 0)] == 0)) lds.key[e + 1] = kNone;
    }
    __syncthreads();
    return place_taken<W>(lds.key, lds.sums, [&](uint32_t key) { return key != kNone; },
                       [&](int p, int q, bool a, bool b, uint2 key, int e) {
                           const int2 at = *reinterpret_cast<const int2 *>(lds.at + e);
                           __syncthreads();
                           if (a) {
                               lds.key[p] = key.x;
                               lds.at[p] = at.x;
                           }
                           if (b) {
                               lds.key[q] = key.y;
                               lds.at[q] = at.y;
                           }
                           __syncthreads();
                       });
}

// Lane xor 1 or 2's value where `other`, the lane's own elsewhere.
template <int CTRL> __device__ __forceinline__ uint32_t pick(bool other, uint32_t own, uint32_t theirs) {
    const uint32_t x = row_take<CTRL>(theirs);
    return other ? x : own;
}

}  // namespace

template <int W, int D, typename TIn>
__global__ __launch_bounds__(64 * W, 4) void select_kernel(SelectParams P) {
    constexpr int NP = QPlanes<TIn>::n, QS = Tiles<D, TIn>::stride, T = Sizes<W>::threads;
    extern __shared__ __align__(16) char mem[];
    Lds<W> &lds = *reinterpret_cast<Lds<W> *>(mem);
    uint16_t *s_q = reinterpret_cast<uint16_t *>(mem + sizeof(Lds<W>));
    const int TB = P.batch;
    const uint32_t unit = blockIdx.x / uint32_t(P.splits);
    const int split = int(blockIdx.x - unit * uint32_t(P.splits));
    const UnitOf u = unit_of(P, unit);
    if (u.tokens <= 0) return;
    if (split == 0) write_kept<W>(P, u);
    if (u.full <= P.shape.top || u.mid == 0) return;
    int lo, hi;
    share_of(P, u, split, lo, hi);
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int rows = u.tokens * P.G, row_tiles = (rows + 15) / 16;
    const int32_t *table = P.pages + int64_t(u.seq) * P.max_pages;
    const uint16_t *bounds = P.bounds + kv_slab(u.layer, P.n_pages, 0, P.H, u.head) * (2 * D);
    if (threadIdx.x == 0) lds.page_size = 0;
    // where the join holds all pages at once, the choice is its own
    const int others = u.full - P.first - P.last;
    const bool join_all = P.splits > 1 && others <= kJoinPages && others <= P.room * P.splits;
    static_assert(W == 8 || kJoinPages / 2 <= Sizes<W>::chunk, "half of them are a share's at once");
    int held = 0;  // of the best so far, or all
    float error = 0.f;
    for (int c0 = lo; c0 < hi; c0 += Sizes<W>::chunk) {
        const int n = min(Sizes<W>::chunk, hi - c0), tiles = (n + 15) / 16;
        for (int rt0 = 0; rt0 < row_tiles; rt0 += TB) {
            const int batch = min(TB, row_tiles - rt0);
            // Where there are fewer tiles than waves, several share a tile's rows.
            const int parts = min(batch, max(1, W / tiles)), jobs = tiles * parts;
            const int lane = fresh_thread() & 63, col = lane & 15, kq = lane >> 4;
            auto part_of_job = [&](int job) { return parts == 1 ? 0 : job / tiles; };
            // A tile's pages: entries, and limits, one tile ahead where the registers allow it.
            auto id_of = [&](int job) {
                const int id = table[min(c0 + (job - part_of_job(job) * tiles) * 16 + col, hi - 1)];
                return unsigned(id) < unsigned(P.n_pages) ? id : -1;
            };
            // Of a page's 2 D limits, largest then smallest, lane (col, kq) wants numbers 128 s + 32 kq + 8 r ..; four
            // lanes read such 64 bytes of four pages, and exchange them.
            struct Limits {
                u32x4 w[D / 64][4];
            };
            auto load = [&](Limits &x, int id) {
                const int quad[4] = {int(row_take<0x00>(uint32_t(id))), int(row_take<0x55>(uint32_t(id))),
                                     int(row_take<0xAA>(uint32_t(id))), int(row_take<0xFF>(uint32_t(id)))};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint16_t *b = bounds + int64_t(max(quad[j], 0)) * P.H * (2 * D) + 32 * kq + 8 * (lane & 3);
#pragma unroll
                    for (int s = 0; s < D / 64; ++s) x.w[s][j] = *reinterpret_cast<const u32x4 *>(b + 128 * s);
                }
            };
            auto exchange = [&](Limits &x) {
                const bool odd = (lane & 1) != 0, high = (lane & 2) != 0;
#pragma unroll
                for (int s = 0; s < D / 64; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a = x.w[s][0][e], b = x.w[s][1][e], c = x.w[s][2][e], d = x.w[s][3][e];
                        const uint32_t a1 = pick<0xB1>(odd, a, b), b1 = pick<0xB1>(!odd, b, a);
                        const uint32_t c1 = pick<0xB1>(odd, c, d), d1 = pick<0xB1>(!odd, d, c);
                        x.w[s][0][e] = pick<0x4E>(high, a1, c1);
                        x.w[s][2][e] = pick<0x4E>(!high, c1, a1);
                        x.w[s][1][e] = pick<0x4E>(high, b1, d1);
                        x.w[s][3][e] = pick<0x4E>(!high, d1, b1);
                    }
            };
            constexpr bool kAhead = D <= 128;
            int id = id_of(min(wave, jobs - 1)), next_id = id_of(min(wave + W, jobs - 1));
            Limits now, then;
            // the first limits are under way while q is laid out
            if (kAhead && wave < jobs) load(now, id);
            if (row_tiles > TB || c0 == lo) {
                // the rows of q, 16 threads each
                const int tid = fresh_thread();
                __syncthreads();  // the last rows, and their length, have been read
                if (tid == 0 && rt0 == 0) lds.q_size = 0;
                __syncthreads();
                for (int r = tid >> 4; r < batch * 16; r += T / 16) {
                    const int row = rt0 * 16 + r, part = tid & 15;
                    const TIn *src = row_of<D, TIn>(P, u, min(row, rows - 1)) + part * (D / 16);
                    float x[D / 16], size = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 16; i += 4) {
                        if constexpr (sizeof(TIn) == 4) {
                            const floatx4 y = *reinterpret_cast<const floatx4 *>(src + i);
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[i + e] = y[e];
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2 *>(src + i);
                            x[i] = bf16_lo(y.x);
                            x[i + 1] = bf16_hi(y.x);
                            x[i + 2] = bf16_lo(y.y);
                            x[i + 3] = bf16_hi(y.y);
                        }
                    }
                    bool bad = false;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        bad |= !(fabsf(x[i]) < __builtin_inff());
                        size = fmaf(x[i], x[i], size);
                    }
                    const bool leave = row >= rows || ((__ballot(bad) >> (lane & 48)) & 0xFFFFu) != 0;
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) size += __shfl_xor(size, d);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t *to = reinterpret_cast<uint32_t *>(s_q + r * QS + 2 * p * D + part * (D / 16));
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            const uint32_t a = leave ? 0 : __float_as_uint(x[2 * i]) & 0xFFFF0000u;
                            const uint32_t b = leave ? 0 : __float_as_uint(x[2 * i + 1]) & 0xFFFF0000u;
                            const uint32_t neg = (int32_t(a) < 0 ? a >> 16 : 0) | (int32_t(b) < 0 ? b : 0);
                            to[i] = (a >> 16 | b) ^ neg;
                            to[D / 2 + i] = neg;
                            x[2 * i] -= __uint_as_float(a);  // exact, and of the same sign
                            x[2 * i + 1] -= __uint_as_float(b);
                        }
                    }
                    if (part == 0) {
                        lds.leave[r] = leave ? 1 : 0;
                        if (!leave) atomicMax(&lds.q_size, __float_as_uint(size));
                    }
                }
                if (rt0 == 0)
                    for (int i = held + tid; i < Sizes<W>::elements; i += T) lds.key[i] = kNone;
                __syncthreads();
            } else {
                const int tid = fresh_thread();
                for (int i = held + tid; i < Sizes<W>::elements; i += T) lds.key[i] = kNone;
                __syncthreads();
            }
            if (!kAhead && wave < jobs) load(now, id);
            for (int job = wave; job < jobs; job += W) {
                const int after = id_of(min(job + 2 * W, jobs - 1));
                if constexpr (kAhead) load(then, next_id);
                const int part = part_of_job(job), tile = job - part * tiles;
                exchange(now);
                // squared length of the limits; a lane has a quarter of the page's
                float size = 0.f;
#pragma unroll
                for (int s = 0; s < D / 64; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = now.w[s][r][e];
                            const bf16x2 two = __builtin_bit_cast(bf16x2, w);
                            size = __builtin_amdgcn_fdot2_f32_bf16(two, two, size, false);
                        }
                float best[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) best[v] = -__builtin_inff();
#pragma unroll 1
                for (int rt = part; rt < batch; rt += parts) {
                    floatx4 score = {};
                    const uint16_t *q = s_q + (rt * 16 + col) * QS + 32 * kq;
#pragma unroll
                    for (int s = 0; s < D / 64; ++s)
#pragma unroll
                        for (int r = 0; r < 4; r += 2) {  // 64 terms
                            if (NP * D > 256 || (NP * D > 128 && r == 0)) __builtin_amdgcn_sched_barrier(0);
                            floatx4 sum[NP > 1 ? 2 : 1] = {};
#pragma unroll
                            for (int p = 0; p < NP; ++p) {
                                const uint16_t *qp = q + 2 * p * D + 128 * s + 8 * r;
                                floatx4 &y = sum[p > 0 ? 1 : 0];
                                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now.w[s][r]),
                                                                            reinterpret_cast<const bf16x8 *>(qp)[0], y, 0, 0, 0);
                                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now.w[s][r + 1]),
                                                                            reinterpret_cast<const bf16x8 *>(qp)[1], y, 0, 0, 0);
                            }
                            if constexpr (NP > 1) sum[0] += sum[1];
                            score += sum[0];
                        }
                    // Lane (col, kq) has rows 4 kq + v, the pages, of its column.
                    const bool leave = lds.leave[rt * 16 + col] != 0;
#pragma unroll
                    for (int v = 0; v < 4; ++v) best[v] = fmaxf(best[v], leave ? -__builtin_inff() : score[v]);
                }
                const uint32_t pages = uint32_t(__ballot(id >= 0)) & 0xFFFFu;
                size += __shfl_xor(size, 16);
                size += __shfl_xor(size, 32);
                const int first = held + tile * 16;
                if (kq == 0 && tile * 16 + col < n) {
                    lds.size[first + col] = id >= 0 ? size : 0.f;
                    lds.at[first + col] = c0 + tile * 16 + col;
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    row_max16(best[v]);
                    const int page = 4 * kq + v;
                    if (col == 0 && tile * 16 + page < n)
                        atomicMax(&lds.key[first + page], (pages >> page) & 1u ? order_of(best[v]) : kAbsent);
                }
                id = next_id;
                next_id = after;
                if constexpr (kAhead)
                    now = then;
                else if (job + W < jobs)
                    load(now, id);
            }
            __syncthreads();
        }
        error = error_of<W, D>(lds, held, held + n);
        held += n;
        if (join_all) break;  // n is all there is
        const bool ends = c0 + Sizes<W>::chunk >= hi;
        held = choose<W, D, TIn>(P, u, lds, held, u.mid, ends && P.splits == 1 ? u.mid : u.mid + P.spare, error);
    }
    const int tid = fresh_thread();
    if (P.splits == 1) {
        for (int i = tid; i < held; i += T) u.out[P.first + i] = lds.at[i];
    } else {
        const int64_t to = int64_t(blockIdx.x) * P.room;
        for (int i = tid; i < held; i += T) {
            P.best_key[to + i] = lds.key[i];
            P.best_at[to + i] = lds.at[i];
        }
        if (tid == 0) {
            P.best_n[blockIdx.x] = held;
            P.best_error[blockIdx.x] = error;
        }
    }
}

// The best of a unit's shares.  Trees of 22 nodes as above: 16 us for the scores, 19 for the join, 4 or 5 of them the
// fp64 scores of two pages in doubt, of one unit in seven (7 with 16 lanes a page and row, which convert both).
template <int D, typename TIn> __global__ __launch_bounds__(1024) void select_join_kernel(SelectParams P) {
    constexpr int W = 16;
    __shared__ Lds<W> lds;
    const uint32_t unit = blockIdx.x;
    const UnitOf u = unit_of(P, unit);
    if (u.tokens <= 0 || u.full <= P.shape.top || u.mid == 0) return;
    // all shares' counts first, so that their pages are under way together
    const int tid = threadIdx.x;
    if (tid < P.splits) {
        const int64_t share = int64_t(unit) * P.splits + tid;
        lds.list[2 * tid] = P.best_n[share];
        lds.list[2 * tid + 1] = __float_as_int(P.best_error[share]);
    }
    __syncthreads();
    int have = 0;
    float error = 0.f;
    for (int split = 0; split < P.splits; ++split) {
        const int64_t from = (int64_t(unit) * P.splits + split) * P.room;
        const int n = lds.list[2 * split];
        if (tid < n) {  // no more than a share has room for
            lds.key[have + tid] = P.best_key[from + tid];
            lds.at[have + tid] = P.best_at[from + tid];
        }
        have += n;
        error = fmaxf(error, __int_as_float(lds.list[2 * split + 1]));
    }
    for (int i = have + int(threadIdx.x); i < Sizes<W>::elements; i += Sizes<W>::threads) lds.key[i] = kNone;
    __syncthreads();
    have = choose<W, D, TIn>(P, u, lds, have, u.mid, u.mid, error);
    for (int i = threadIdx.x; i < have; i += Sizes<W>::threads) u.out[P.first + i] = lds.at[i];
}

// Two bf16 numbers as 16-bit integers of the same order, and back.
__device__ __forceinline__ uint32_t in_order(uint32_t x) {
    const uint32_t sign = __builtin_bit_cast(uint32_t, __builtin_bit_cast(s16x2, x) >> 15);
    return x ^ (sign & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t ordered_pair(float a, float b) {
    return in_order(__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u));
}
__device__ __forceinline__ uint32_t pair_max(uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, x), __builtin_bit_cast(s16x2, y)));
}
__device__ __forceinline__ uint32_t pair_min(uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(s16x2, x), __builtin_bit_cast(s16x2, y)));
}

// A wave a page and head.  A lane reads 16 bytes of codes, a token's 32 channels of one block, as they lie
// in memory: 64 lanes take 16 tokens of 4 blocks, and 32 values each, whose largest and smallest of a page
// are joined over the 16 lanes of a block at the end.
template <int D> __global__ __launch_bounds__(256, 4) void bounds_kernel(BoundsParams P) {
    constexpr int NB = D / 32;             // blocks of a token
    constexpr int GROUPS = NB < 4 ? 2 : 1;   // groups of 16 tokens a load takes
    constexpr int PASSES = NB > 4 ? 2 : 1;  // loads a group takes
    const uint32_t unit = blockIdx.x * 4u + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (unit >= P.units) return;
    uint32_t i = unit;
    const int head = int(i % uint32_t(P.H));
    i /= uint32_t(P.H);
    const int each = int(i % uint32_t(P.pages_each));
    i /= uint32_t(P.pages_each);
    const int seq = int(i % uint32_t(P.S)), layer = P.layer_begin + int(i / uint32_t(P.S));
    const int length = length_of(P.length[seq], int64_t(P.max_pages) << P.page_shift);
    const int n_new = P.seq_off[seq + 1] - P.seq_off[seq];
    const int entry = (max(length - n_new, 0) >> P.page_shift) + each;
    if (n_new <= 0 || entry >= length >> P.page_shift) return;
    const int id = P.pages[int64_t(seq) * P.max_pages + entry];
    if (unsigned(id) >= unsigned(P.n_pages)) return;
    const int lane = threadIdx.x & 63, token = lane & 15, part = lane >> 4;
    const int block = part & (NB < 4 ? NB - 1 : 3), group = part / (NB < 4 ? NB : 4);  // of the first pass
    const int64_t slab = kv_slab(layer, P.n_pages, id, P.H, head), slots = slab << P.page_shift;
    const uint8_t *codes = P.kc + slots * (D / 2) + KvAt<D>::key(token, 4 * block);
    const uint8_t *scales = P.ks + slots * NB + KvAt<D>::key_scale(token, block);
    const int groups = (1 << P.page_shift) / 16;
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        float most[32], least[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            most[c] = -__builtin_inff();
            least[c] = __builtin_inff();
        }
        bool poison = false;
        for (int g = 0; g < groups; g += 4 * GROUPS) {
            // four loads under way together; past the page's end its last group again
            u32x4 w[4];
            int e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = 16 * min(g + GROUPS * k + group, groups - 1);
                w[k] = *reinterpret_cast<const u32x4 *>(codes + KvAt<D>::group_codes(at) + pass * 1024);
                e[k] = scales[KvAt<D>::group_scales(at) + pass * 4];
            }
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                poison |= e[k] == kPoison || e[k + 1] == kPoison;
                const float unit0 = __uint_as_float(uint32_t(e[k]) << 23), unit1 = __uint_as_float(uint32_t(e[k + 1]) << 23);
                auto two = [&](auto v, auto y, int c) {
                    most[c] = fmaxf(fmaxf(most[c], v[0]), y[0]);
                    least[c] = fminf(fminf(least[c], v[0]), y[0]);
                    most[c + 1] = fmaxf(fmaxf(most[c + 1], v[1]), y[1]);
                    least[c + 1] = fminf(fminf(least[c + 1], v[1]), y[1]);
                };
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t a = w[k][x], b = w[k + 1][x];
                    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a, unit0, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(b, unit1, 0), 8 * x);
                    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a, unit0, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(b, unit1, 1), 8 * x + 2);
                    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a, unit0, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(b, unit1, 2), 8 * x + 4);
                    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a, unit0, 3),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(b, unit1, 3), 8 * x + 6);
                }
            }
        }
        // Over the 16 lanes of the block's tokens (and, with 64 channels, the other group's), two channels a
        // register: as 16-bit integers of the same order.  At each of four exchanges a lane hands the half of its
        // channels that the other keeps, until it has the two of its number.
        uint32_t high[16], low[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            high[c] = ordered_pair(most[2 * c], most[2 * c + 1]);
            low[c] = ordered_pair(least[2 * c], least[2 * c + 1]);
        }
        auto halve = [&](auto take, int n) {
            const bool upper = (lane & n) != 0;
#pragma unroll
            for (int c = 0; c < n; ++c) {
                high[c] = pair_max(upper ? high[c + n] : high[c], take(upper ? high[c] : high[c + n]));
                low[c] = pair_min(upper ? low[c + n] : low[c], take(upper ? low[c] : low[c + n]));
            }
        };
        halve([](uint32_t x) { return row_take<0x140>(x); }, 8);
        halve([](uint32_t x) { return row_take<0x141>(x); }, 4);
        halve([](uint32_t x) { return row_take<0x4E>(x); }, 2);
        halve([](uint32_t x) { return row_take<0xB1>(x); }, 1);
        if constexpr (GROUPS == 2) {
            high[0] = pair_max(high[0], uint32_t(__shfl_xor(high[0], 32)));
            low[0] = pair_min(low[0], uint32_t(__shfl_xor(low[0], 32)));
        }
        uint64_t mine = __ballot(poison);
        mine = GROUPS == 2 ? mine >> (16 * block) | mine >> (16 * block + 32) : mine >> (16 * part);
        const bool nan = (mine & 0xFFFFu) != 0;
        if (group != 0) continue;
        uint32_t *to = reinterpret_cast<uint32_t *>(P.bounds + slab * (2 * D) + 32 * (block + 4 * pass)) + token;
        to[0] = nan ? 0x7FC07FC0u : in_order(high[0]);
        to[D / 2] = nan ? 0x7FC07FC0u : in_order(low[0]);
    }
}

namespace {

template <int W, int D, typename TIn>
gdn_status launch_select(SelectParams P, const SelectPlan &plan, hipStream_t s) {
    // All rows' q at once where it fits: a batch more is a turn more over the pages, and 1.3 us for its q.
    constexpr int each = Tiles<D, TIn>::bytes, most = int((160 * 1024 / (16 / W) - sizeof(Lds<W>)) / each);
    static_assert(most >= 1, "a row tile fits");
    P.batch = int32_t(std::min<int64_t>(plan.row_tiles, std::min(most, kMaxBatch)));
    hipLaunchKernelGGL((select_kernel<W, D, TIn>), dim3(uint32_t(plan.units * plan.splits)), dim3(64 * W),
                       sizeof(Lds<W>) + P.batch * each, s, P);
    GDN_LAUNCH_CHECK("select_kernel");
    if (plan.splits == 1) return GDN_OK;
    hipLaunchKernelGGL((select_join_kernel<D, TIn>), dim3(uint32_t(plan.units)), dim3(1024), 0, s, P);
    GDN_LAUNCH_CHECK("select_join_kernel");
    return GDN_OK;
}

template <int D, typename TIn> gdn_status launch_select(const SelectParams &P, const SelectPlan &plan, hipStream_t s) {
    return plan.narrow ? launch_select<8, D, TIn>(P, plan, s) : launch_select<16, D, TIn>(P, plan, s);
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_kv_bounds(const gdn_kv_args *a, const gdn_sparse_args *x, const int32_t *host_seq_offsets,
                                    void *stream) {
    clear_error();
    const char *who = "gdn_kv_bounds";
    if (x == nullptr) return fail(GDN_EINVAL, "%s: null arguments", who);
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, who, true, empty);
    if (st != GDN_OK || empty) return st;
    const void *bounds[] = {x->bounds};
    st = check_aligned16(bounds, 1, who, "bounds");
    if (st != GDN_OK) return st;
    int64_t longest = 0;
    for (int32_t b = 0; b < a->n_seqs; ++b)
        longest = std::max<int64_t>(longest, host_seq_offsets[b + 1] - host_seq_offsets[b]);
    BoundsParams P{};
    P.kc = a->k_codes;
    P.ks = a->k_scales;
    P.bounds = x->bounds;
    P.pages = a->pages;
    P.length = a->length;
    P.seq_off = a->seq_offsets;
    P.S = a->n_seqs;
    P.H = a->n_kv_heads;
    P.n_pages = a->n_pages;
    P.max_pages = a->max_pages;
    P.page_shift = log2_exact(a->page_tokens);
    P.layer_begin = a->layer_begin;
    // n slots are on n / page_tokens + 1 pages that end with or after them at most
    const int64_t each = std::min<int64_t>(longest / a->page_tokens + 1, a->max_pages);
    P.pages_each = int32_t(each);
    const int64_t heads = int64_t(a->n_kv_heads) * a->n_layers;
    if (heads > kMaxBlocks / a->n_seqs || heads * a->n_seqs > kMaxBlocks / each)
        return fail(GDN_EINVAL, "%s: too many workgroups", who);
    P.units = uint32_t(heads * a->n_seqs * each);
    const dim3 grid((P.units + 3) / 4), block(256);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (a->head_dim) {
        case 64: hipLaunchKernelGGL((bounds_kernel<64>), grid, block, 0, s, P); break;
        case 128: hipLaunchKernelGGL((bounds_kernel<128>), grid, block, 0, s, P); break;
        default: hipLaunchKernelGGL((bounds_kernel<256>), grid, block, 0, s, P);
    }
    GDN_LAUNCH_CHECK("bounds_kernel");
    return GDN_OK;
}

extern "C" gdn_status gdn_kv_select(const gdn_kv_args *a, const gdn_sparse_args *x, const int32_t *host_seq_offsets,
                                    void *stream) {
    clear_error();
    const char *who = "gdn_kv_select";
    if (x == nullptr) return fail(GDN_EINVAL, "%s: null arguments", who);
    bool empty;
    gdn_status st = check_kv_args(a, host_seq_offsets, who, true, empty);
    if (st != GDN_OK || empty) return st;
    st = check_attention_sizes(a, host_seq_offsets, who);
    if (st != GDN_OK) return st;
    st = check_sparse_sizes(a, x, host_seq_offsets, who);
    if (st != GDN_OK) return st;
    if (x->selected == nullptr) return fail(GDN_EINVAL, "%s: null selected", who);
    const void *in[] = {a->q, x->bounds};
    st = check_aligned16(in, 2, who, "q/bounds");
    if (st != GDN_OK) return st;
    const SelectPlan plan = plan_select(a, x, host_seq_offsets);
    if (!select_fits(plan)) return fail(GDN_EINVAL, "%s: too many workgroups", who);
    if (plan.workspace > 0) {
        if (a->workspace == nullptr || a->workspace_bytes < plan.workspace)
            return fail(GDN_ECAPACITY, "%s: workspace holds %lld bytes, the call needs %lld", who,
                        static_cast<long long>(a->workspace ? a->workspace_bytes : 0),
                        static_cast<long long>(plan.workspace));
        const void *ws[] = {a->workspace};
        st = check_aligned16(ws, 1, who, "workspace");
        if (st != GDN_OK) return st;
    }
    SelectParams P{};
    P.q = a->q;
    P.bounds = x->bounds;
    P.pages = a->pages;
    P.length = a->length;
    P.seq_off = a->seq_offsets;
    P.selected = x->selected;
    const int64_t shares = plan.units * plan.splits, best = shares * plan.room;
    P.best_key = static_cast<uint32_t *>(a->workspace);
    P.best_at = reinterpret_cast<int32_t *>(P.best_key + best);
    P.best_n = P.best_at + best;
    P.best_error = reinterpret_cast<float *>(P.best_n + shares);
    P.spare = kSparePages;
    P.room = plan.room;
    P.shape = SparseShape{x->top_pages, x->share_tokens};
    P.S = a->n_seqs;
    P.H = a->n_kv_heads;
    P.G = a->n_heads / a->n_kv_heads;
    P.T = a->n_tokens;
    P.n_pages = a->n_pages;
    P.max_pages = a->max_pages;
    P.page_shift = log2_exact(a->page_tokens);
    P.layer_begin = a->layer_begin;
    P.selections = int32_t(plan.selections);
    P.splits = plan.splits;
    P.first = x->keep_first;
    P.last = x->keep_last;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = a->in_dtype == GDN_BF16;
    switch (a->head_dim) {
        case 64: return bf16 ? launch_select<64, bf16_t>(P, plan, s) : launch_select<64, float>(P, plan, s);
        case 128: return bf16 ? launch_select<128, bf16_t>(P, plan, s) : launch_select<128, float>(P, plan, s);
        default: return bf16 ? launch_select<256, bf16_t>(P, plan, s) : launch_select<256, float>(P, plan, s);
    }
}
