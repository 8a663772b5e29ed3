// Page selection of the sparse attention (gfx950): bounds of the cached keys a page, scores of pages by
// them, and the best pages of a selection.  The rules are in gdn_tree.h.
//
// Bounds.  A wave takes 32 channels of a page and head, 16 tokens at a time as the cache holds them, and
// keeps the largest and smallest value of 8 channels a lane.  Stored keys are 4-bit floats times a power
// of two, so their limits are bf16 numbers.
//
// Scores.  With q+ = max(q, 0) and q- = min(q, 0), score = sum_c q+_c largest_c + q-_c smallest_c: a matrix
// product of pages x 2 d by 2 d x rows, on the fp64 matrix cores, 16 pages x 16 rows x 4 at a time.  fp64 is
// for the choice, not for the numbers: a page's rank among hundreds would otherwise hang on the order of
// a sum (bf16 q and limits have products of 10 bits, whose sums fp64 holds exactly unless they spread
// over more than 40 binades).
//
// Best pages.  Keys are the scores as integers of the same order; the k-th largest is found 8 bits at a
// time from histograms in LDS, over the range the keys span, until a bin is taken whole.  Elements stay in
// the table's order throughout, so that equal scores go to the lower entry and the result is ascending
// without a sort.
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
    uint64_t *best_key;  // [unit][split][top]
    int32_t *best_at;
    SparseShape shape;
    int32_t S, H, G, T, n_pages, max_pages, page_shift, layer_begin, selections, splits, first, last;
};

struct BoundsParams {
    const uint8_t *kc, *ks;
    uint16_t *bounds;
    const int32_t *pages, *length, *seq_off;
    int32_t S, H, n_pages, max_pages, page_shift, layer_begin, pages_each;
};

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kSelectThreads = 256;
constexpr int kChunk = 1024;  // pages scored before the best are kept
constexpr int kChunkEach = (kChunk + kMaxTopPages) / kSelectThreads;
static_assert(kChunkEach * kSelectThreads == kChunk + kMaxTopPages, "");

// Integer of the same order.  Scores that are not numbers come first, see below.
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t b = uint64_t(__double_as_longlong(x + 0.0));  // -0 is 0
    return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}

template <int CTRL> __device__ __forceinline__ double row_max(double x) {
    const int lo = __builtin_amdgcn_mov_dpp(__double2loint(x), CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_mov_dpp(__double2hiint(x), CTRL, 0xF, 0xF, true);
    return fmax(x, __hiloint2double(hi, lo));
}

struct Scratch {
    uint64_t range[2][kSelectThreads / 64];
    uint32_t bins[256];
    int bin, left, count;
    int sums[kSelectThreads / 64];
};

// Sum of x over the threads before this one, and over all.
__device__ __forceinline__ int before(int x, Scratch &s, int &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int run = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(run, d);
        if (lane >= d) run += up;
    }
    __syncthreads();  // the last sums have been read
    if (lane == 63) s.sums[wave] = run;
    __syncthreads();
    int base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kSelectThreads / 64; ++w) {
        base += w < wave ? s.sums[w] : 0;
        all += s.sums[w];
    }
    return base + run - x;
}

// Bits of the k largest of the workgroup's keys, of which a thread holds EACH consecutive ones (bit e of
// `there`: key e exists; more than k exist), equal ones in order.  k > 0.
template <int EACH>
__device__ __forceinline__ uint32_t largest(const uint64_t (&key)[EACH], uint32_t there, int k, Scratch &s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t lo = ~0ull, hi = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        if ((there >> e) & 1u) {
            lo = min(lo, key[e]);
            hi = max(hi, key[e]);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        lo = min(lo, uint64_t(__shfl_xor((unsigned long long)lo, d)));
        hi = max(hi, uint64_t(__shfl_xor((unsigned long long)hi, d)));
    }
    if (lane == 0) {
        s.range[0][wave] = lo;
        s.range[1][wave] = hi;
    }
    s.bins[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelectThreads / 64; ++w) {
        lo = min(lo, s.range[0][w]);
        hi = max(hi, s.range[1][w]);
    }
    const int shift = hi > lo ? __clzll((long long)(hi - lo)) : 0;
    uint64_t prefix = 0, mask = 0;
    int left = k, count = 0;
    for (int at = 56;; at -= 8) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const uint64_t u = (key[e] - lo) << shift;
            if (((there >> e) & 1u) && (u & mask) == prefix) atomicAdd(&s.bins[(u >> at) & 255u], 1u);
        }
        __syncthreads();
        if (wave == 0) {  // from the top: 4 bins a lane
            int c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = int(s.bins[255 - 4 * lane - i]);
                sum += c[i];
            }
            int run = sum;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(run, d);
                if (lane >= d) run += up;
            }
            int above = run - sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (above < left && above + c[i] >= left) {
                    s.bin = 255 - 4 * lane - i;
                    s.left = left - above;
                    s.count = c[i];
                }
                above += c[i];
            }
        }
        __syncthreads();
        prefix |= uint64_t(s.bin) << at;
        mask |= uint64_t(255) << at;
        left = s.left;
        count = s.count;
        if (count == left || at == 0) break;
        s.bins[threadIdx.x] = 0;
        __syncthreads();
    }
    uint32_t more = 0, same = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const uint64_t u = ((key[e] - lo) << shift) & mask;
        if ((there >> e) & 1u) {
            more |= (u > prefix ? 1u : 0u) << e;
            same |= (u == prefix ? 1u : 0u) << e;
        }
    }
    if (count == left) return more | same;
    int all, rank = before(__popc(same), s, all);
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if ((same >> e) & 1u) more |= (rank++ < left ? 1u : 0u) << e;
    return more;
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
__device__ __forceinline__ void write_kept(const SelectParams &P, const UnitOf &u) {
    const int top = P.shape.top;
    for (int i = threadIdx.x; i < top; i += kSelectThreads) {
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

}  // namespace

template <int D, typename TIn>
__global__ __launch_bounds__(kSelectThreads, 4) void select_kernel(SelectParams P) {
    constexpr int QS = D + 4;  // floats between the rows of q in LDS
    __shared__ __align__(16) float s_q[16 * QS];
    __shared__ uint64_t s_key[kChunk + kMaxTopPages];
    __shared__ int32_t s_at[kChunk + kMaxTopPages];
    __shared__ int s_out[16];
    __shared__ Scratch s_scratch;
    const uint32_t unit = blockIdx.x / uint32_t(P.splits);
    const int split = int(blockIdx.x - unit * uint32_t(P.splits));
    const UnitOf u = unit_of(P, unit);
    if (u.tokens <= 0) return;
    if (split == 0) write_kept(P, u);
    if (u.full <= P.shape.top || u.mid == 0) return;
    int lo, hi;
    share_of(P, u, split, lo, hi);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 15, kq = lane >> 4;
    const int rows = u.tokens * P.G, row_tiles = (rows + 15) / 16;
    const int32_t *table = P.pages + int64_t(u.seq) * P.max_pages;
    const uint16_t *bounds = P.bounds + kv_slab(u.layer, P.n_pages, 0, P.H, u.head) * (2 * D);
    int held = 0;  // best pages so far, in s_key and s_at
    for (int c0 = lo; c0 < hi; c0 += kChunk) {
        const int n = min(kChunk, hi - c0), tiles = (n + 15) / 16;
        for (int rt = 0; rt < row_tiles; ++rt) {
            if (rt > 0 || row_tiles > 1 || c0 == lo) {
                // 16 rows of q, 16 threads a row
                __syncthreads();
                const int r = tid >> 4, row = rt * 16 + r, part = tid & 15;
                const int token = u.off + u.first_token + min(row, rows - 1) / P.G;
                const int hq = u.head * P.G + min(row, rows - 1) % P.G;
                const TIn *src = static_cast<const TIn *>(P.q) +
                                 ((int64_t(u.layer) * P.T + token) * (P.H * P.G) + hq) * D + part * (D / 16);
                float x[D / 16];
                bool bad = false;
#pragma unroll
                for (int i = 0; i < D / 16; i += 16 / int(sizeof(TIn)) < D / 16 ? 16 / int(sizeof(TIn)) : D / 16) {
                    if constexpr (sizeof(TIn) == 4) {
                        const floatx4 y = *reinterpret_cast<const floatx4 *>(src + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i + e] = y[e];
                    } else if constexpr (D == 64) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(src + i);
                        x[i] = bf16_lo(y.x); x[i + 1] = bf16_hi(y.x); x[i + 2] = bf16_lo(y.y); x[i + 3] = bf16_hi(y.y);
                    } else {
                        const u32x4 y = *reinterpret_cast<const u32x4 *>(src + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[i + 2 * e] = bf16_lo(y[e]);
                            x[i + 2 * e + 1] = bf16_hi(y[e]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) bad |= !(fabsf(x[i]) < __builtin_inff());
                const bool leave = row >= rows || ((__ballot(bad) >> (lane & 48)) & 0xFFFFu) != 0;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) s_q[r * QS + part * (D / 16) + i] = leave ? 0.f : x[i];
                if (part == 0) s_out[r] = leave ? 1 : 0;
                __syncthreads();
            }
            const bool leave = s_out[col] != 0;
            for (int tile = wave; tile < tiles; tile += kSelectThreads / 64) {
                const int entry = min(c0 + tile * 16 + col, hi - 1);
                int id = table[entry];
                if (unsigned(id) >= unsigned(P.n_pages)) id = -1;
                const uint32_t there = uint32_t(__ballot(id >= 0)) & 0xFFFFu;
                const uint16_t *b = bounds + int64_t(max(id, 0)) * P.H * (2 * D) + 8 * kq;
                u32x4 most[D / 32], least[D / 32];
#pragma unroll
                for (int t = 0; t < D / 32; ++t) {
                    most[t] = *reinterpret_cast<const u32x4 *>(b + 32 * t);
                    least[t] = *reinterpret_cast<const u32x4 *>(b + D + 32 * t);
                }
                f64x4 up = {0.0, 0.0, 0.0, 0.0}, down = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
                for (int t = 0; t < D / 32; ++t) {
                    __builtin_amdgcn_sched_barrier(0);  // all operands widened ahead would not fit
                    const float *q = s_q + col * QS + 32 * t + 8 * kq;
                    const floatx4 q0 = reinterpret_cast<const floatx4 *>(q)[0];
                    const floatx4 q1 = reinterpret_cast<const floatx4 *>(q)[1];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float x = e < 4 ? q0[e] : q1[e - 4];
                        const uint32_t mw = most[t][e / 2], lw = least[t][e / 2];
                        const float m = (e & 1) != 0 ? bf16_hi(mw) : bf16_lo(mw);
                        const float l = (e & 1) != 0 ? bf16_hi(lw) : bf16_lo(lw);
                        up = __builtin_amdgcn_mfma_f64_16x16x4f64(double(m), double(fmaxf(x, 0.f)), up, 0, 0, 0);
                        down = __builtin_amdgcn_mfma_f64_16x16x4f64(double(l), double(fminf(x, 0.f)), down, 0, 0, 0);
                    }
                }
                // Lane (col, kq) has rows 4 v + kq, the pages, of its column.
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    double x = up[v] + down[v];
                    // limits that are not numbers: the page holds a key that is not
                    x = !(x == x) ? double(__builtin_inff()) : leave ? -double(__builtin_inff()) : x;
                    x = row_max<0xB1>(x);
                    x = row_max<0x4E>(x);
                    x = row_max<0x141>(x);
                    x = row_max<0x140>(x);
                    const int page = 4 * v + kq, i = tile * 16 + page;
                    if (col == 0 && i < n) {
                        uint64_t key = (there >> page) & 1u ? order_of(x) : 0;
                        if (rt > 0) key = max(key, s_key[held + i]);
                        s_key[held + i] = key;
                        s_at[held + i] = c0 + i;
                    }
                }
            }
        }
        __syncthreads();
        const int have = held + n;
        if (have > u.mid) {
            uint64_t key[kChunkEach];
            int at[kChunkEach];
            uint32_t exists = 0;
#pragma unroll
            for (int e = 0; e < kChunkEach; ++e) {
                const int i = tid * kChunkEach + e;
                key[e] = s_key[i];
                at[e] = s_at[i];
                exists |= (i < have ? 1u : 0u) << e;
            }
            const uint32_t take = largest<kChunkEach>(key, exists, u.mid, s_scratch);
            int all, to = before(__popc(take), s_scratch, all);
#pragma unroll
            for (int e = 0; e < kChunkEach; ++e) {
                if ((take >> e) & 1u) {
                    s_key[to] = key[e];
                    s_at[to++] = at[e];
                }
            }
            __syncthreads();
            held = u.mid;
        } else {
            held = have;
        }
    }
    if (P.splits == 1) {
        for (int i = tid; i < held; i += kSelectThreads) u.out[P.first + i] = s_at[i];
    } else {
        const int64_t to = int64_t(blockIdx.x) * P.shape.top;
        for (int i = tid; i < held; i += kSelectThreads) {
            P.best_key[to + i] = s_key[i];
            P.best_at[to + i] = s_at[i];
        }
    }
}

// The best of a unit's shares.
template <int EACH> __global__ __launch_bounds__(kSelectThreads) void select_join_kernel(SelectParams P) {
    __shared__ Scratch s_scratch;
    const uint32_t unit = blockIdx.x;
    const UnitOf u = unit_of(P, unit);
    if (u.tokens <= 0 || u.full <= P.shape.top || u.mid == 0) return;
    uint64_t key[EACH];
    int at[EACH];
    uint32_t exists = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int i = int(threadIdx.x) * EACH + e, split = i / u.mid, k = i - split * u.mid;
        key[e] = 0;
        at[e] = 0;
        if (split < P.splits) {
            int lo, hi;
            share_of(P, u, split, lo, hi);
            if (k < hi - lo) {
                const int64_t from = (int64_t(unit) * P.splits + split) * P.shape.top + k;
                key[e] = P.best_key[from];
                at[e] = P.best_at[from];
                exists |= 1u << e;
            }
        }
    }
    const uint32_t take = largest<EACH>(key, exists, u.mid, s_scratch);
    int all, to = before(__popc(take), s_scratch, all);
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if ((take >> e) & 1u) u.out[P.first + to++] = at[e];
}

// A workgroup a page and head, a wave 32 channels: lane = 4 token + piece of 8 channels.
template <int D> __global__ __launch_bounds__(2 * D) void bounds_kernel(BoundsParams P) {
    uint32_t i = blockIdx.x;
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
    const int lane = threadIdx.x & 63, block = threadIdx.x >> 6, token = lane >> 2, piece = lane & 3;
    const int64_t slab = kv_slab(layer, P.n_pages, id, P.H, head), slots = slab << P.page_shift;
    const uint8_t *codes = P.kc + slots * (D / 2) + KvAt<D>::key(token, 4 * block + piece);
    const uint8_t *scales = P.ks + slots * (D / 32) + KvAt<D>::key_scale(token, block);
    float most[8], least[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        most[c] = -__builtin_inff();
        least[c] = __builtin_inff();
    }
    bool poison = false;
#pragma unroll 4
    for (int g = 0; g < (1 << P.page_shift) / 16; ++g) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + KvAt<D>::group_codes(16 * g));
        const int e = scales[KvAt<D>::group_scales(16 * g)];
        poison |= e == kPoison;
        const float unit = __uint_as_float(uint32_t(e) << 23);
        float x[8];
        auto two = [&](auto v, int c) {
            x[c] = v[0];
            x[c + 1] = v[1];
        };
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 0), 0);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 1), 2);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 2), 4);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, unit, 3), 6);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            most[c] = fmaxf(most[c], x[c]);
            least[c] = fminf(least[c], x[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
        for (int d = 4; d < 64; d <<= 1) {
            most[c] = fmaxf(most[c], __shfl_xor(most[c], d));
            least[c] = fminf(least[c], __shfl_xor(least[c], d));
        }
    }
    const bool bad = __ballot(poison) != 0;
    if (token > 1) return;
    u32x4 out;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float a = token == 0 ? most[2 * c] : least[2 * c], b = token == 0 ? most[2 * c + 1] : least[2 * c + 1];
        out[c] = bad ? 0x7FC07FC0u : (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
    }
    *reinterpret_cast<u32x4 *>(P.bounds + slab * (2 * D) + token * D + 32 * block + 8 * piece) = out;
}

namespace {

template <int D>
void launch_select(const SelectParams &P, const SelectPlan &plan, bool bf16, hipStream_t s) {
    const dim3 grid(uint32_t(plan.units * plan.splits)), block(kSelectThreads);
    if (bf16)
        hipLaunchKernelGGL((select_kernel<D, bf16_t>), grid, block, 0, s, P);
    else
        hipLaunchKernelGGL((select_kernel<D, float>), grid, block, 0, s, P);
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
    const int64_t heads = int64_t(a->n_kv_heads) * a->n_layers, most = kMaxBlocks / 2;  // 512 threads
    if (heads > most / a->n_seqs || heads * a->n_seqs > most / each)
        return fail(GDN_EINVAL, "%s: too many workgroups", who);
    const dim3 grid(uint32_t(heads * a->n_seqs * each));
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (a->head_dim) {
        case 64: hipLaunchKernelGGL((bounds_kernel<64>), grid, dim3(128), 0, s, P); break;
        case 128: hipLaunchKernelGGL((bounds_kernel<128>), grid, dim3(256), 0, s, P); break;
        default: hipLaunchKernelGGL((bounds_kernel<256>), grid, dim3(512), 0, s, P);
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
    if (plan.units * plan.splits > kMaxBlocks) return fail(GDN_EINVAL, "%s: too many workgroups", who);
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
    P.best_key = static_cast<uint64_t *>(a->workspace);
    P.best_at = reinterpret_cast<int32_t *>(P.best_key + plan.units * plan.splits * x->top_pages);
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
        case 64: launch_select<64>(P, plan, bf16, s); break;
        case 128: launch_select<128>(P, plan, bf16, s); break;
        default: launch_select<256>(P, plan, bf16, s);
    }
    GDN_LAUNCH_CHECK("select_kernel");
    if (plan.splits == 1) return GDN_OK;
    const int pages = plan.splits * x->top_pages;
    if (pages <= 4 * kSelectThreads)
        hipLaunchKernelGGL((select_join_kernel<4>), dim3(uint32_t(plan.units)), dim3(kSelectThreads), 0, s, P);
    else
        hipLaunchKernelGGL((select_join_kernel<16>), dim3(uint32_t(plan.units)), dim3(kSelectThreads), 0, s, P);
    GDN_LAUNCH_CHECK("select_join_kernel");
    return GDN_OK;
}
