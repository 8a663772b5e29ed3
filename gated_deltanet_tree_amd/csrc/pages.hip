// Page tables and slot maps of the paged cache, built on the device (gfx950).  The rules are in
// gdn_tree.h.
//
// Reserving is a numbering: the r-th table entry without a page, in order of (sequence, entry), takes the
// r-th free page, in order of its id.  Both sides are counted first, then the free pages are listed by
// rank, then every sequence finds its first rank and fills its entries.  No workgroup waits for another, so
// the result does not depend on the order anything runs in: three launches, a workgroup a chunk of pages or a
// sequence, or one launch of one workgroup where pool and tables are small.  What has to be moved is the
// pool's reference counts and the tables, once; below a few thousand pages latencies are all there is to it
// (reserve and release, 32 trees of 22 nodes in 6000 pages: 16.2 us in three launches, 11.1 in one).
#include <algorithm>

#include "kv_internal.h"
#include "kv_layout.h"
#include "gdn_device.h"

namespace gdn {

struct PagesParams {
    int32_t *pages, *refs, *missing;
    const int32_t *length, *seq_off, *depth;
    int64_t *slots;
    int32_t *positions;
    int32_t *free_count;  // [chunks] free pages of a chunk
    int32_t *need;        // [S] entries without a page
    int32_t *need_sum;    // [ceil(S / kSeqBlock)]
    int32_t *list;        // [n_pages] free pages by rank
    int32_t S, n_pages, max_pages, page_shift, chunks;
};

namespace {

constexpr int kPageThreads = 256;
constexpr int kAssignThreads = 512;
constexpr int kEntries = 4;       // table entries, and tokens, that a thread looks at at once
constexpr int kPageChunk = 2048;  // pages a workgroup counts, 8 a thread
constexpr int kSeqBlock = 1024;   // sequences whose needs are summed at once
// One launch up to these sizes, which one compute unit handles in the time of the launches it saves: each of 16 waves
// takes the sequences' slots one after the other, 64 tokens at a time.  The tokens of a sequence are known on the
// device only, so their number is bounded in all and on average.  us, reserve and release, one launch / three, 8192 pages:
//   1 new token a sequence, 16384 entries, 32 sequences 11.9 / 15.6, 64 12.9 / 15.4, 96 14.9 / 15.6, 128 15.6 / 15.7, 256
//   21.4 / 15.9;  64 tokens each, 32 sequences 13.4 / 15.1, 64 14.5 / 15.3, 96 16.4 / 15.6, 128 17.5 / 16.2;
//   one sequence, 256 tokens 11.8 / 14.9, 1024 14.7 / 15.1, 2048 18.4 / 15.6, 8192 42.9 / 18.6;  4 sequences of 256
//   14.6 / 16.2, of 512 16.2 / 16.0, of 1024 18.5 / 16.4;  32 of 128 14.5 / 15.2, of 256 16.2 / 15.9.
constexpr int kSmallThreads = 1024, kSmallPages = 8192, kSmallEntries = 16384, kSmallSeqs = 96;
constexpr int kSmallTokens = 4096, kSmallFew = 1024, kSmallEach = 64;

// Sum of x over the workgroup's WAVES waves; every thread gets it.
template <int WAVES> __device__ __forceinline__ int64_t total(int64_t x, int64_t *sums) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor((long long)x, d);
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) all += sums[w];
    return all;
}

// Sums of x and y, as above.
template <int WAVES> __device__ __forceinline__ void totals(int64_t &x, int64_t &y, int64_t *sums) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        x += __shfl_xor((long long)x, d);
        y += __shfl_xor((long long)y, d);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        sums[threadIdx.x >> 6] = x;
        sums[WAVES + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = y = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        x += sums[w];
        y += sums[WAVES + w];
    }
}

// Sum over the threads before this one, and over all.
template <int WAVES> __device__ __forceinline__ int before_thread(int x, int *sums, int &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int run = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(run, d);
        if (lane >= d) run += up;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    int base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        base += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    return base + run - x;
}

// Table entries that a sequence's committed and new tokens take.
__device__ __forceinline__ int entries_of(const PagesParams &P, int seq) {
    const int64_t length = max(P.length[seq], 0), n = P.seq_off[seq + 1] - P.seq_off[seq];
    const int64_t page = int64_t(1) << P.page_shift;
    return int(min((length + n + page - 1) >> P.page_shift, int64_t(P.max_pages)));
}

__device__ __forceinline__ bool has_page(const PagesParams &P, int id) { return unsigned(id) < unsigned(P.n_pages); }

// Slot of position `at`, page id `id` (-1: none).
__device__ __forceinline__ int64_t slot_of(const PagesParams &P, int id, int64_t at) {
    return id < 0 ? -1 : (int64_t(id) << P.page_shift) + (at & ((int64_t(1) << P.page_shift) - 1));
}
__device__ __forceinline__ int32_t position_of(int64_t length, int64_t depth) {
    return int32_t(min(length + depth, int64_t(INT32_MAX)));
}

// Slots and positions of a sequence's new tokens, by `threads` threads.
__device__ __forceinline__ void write_slots(const PagesParams &P, int seq, int thread, int threads) {
    const int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    const int off = P.seq_off[seq], n_new = P.seq_off[seq + 1] - off;
    const int64_t length = max(P.length[seq], 0);
    for (int i0 = thread; i0 < n_new; i0 += kEntries * threads) {
        int id[kEntries], depth[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int i = min(i0 + e * threads, n_new - 1);
            const int64_t entry = (length + i) >> P.page_shift;
            id[e] = table[min(entry, int64_t(P.max_pages - 1))];
            id[e] = entry < P.max_pages && has_page(P, id[e]) ? id[e] : -1;
            depth[e] = P.depth != nullptr ? P.depth[off + i] : i;
        }
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int i = i0 + e * threads;
            if (i >= n_new) break;
            if (P.slots != nullptr) P.slots[off + i] = slot_of(P, id[e], length + i);
            if (P.positions != nullptr) P.positions[off + i] = position_of(length, depth[e]);
        }
    }
}

}  // namespace

// Workgroups 0 .. chunks - 1 count a chunk's free pages, the others a sequence's entries without one; a thread
// has 8 pages, or kEntries entries, under way together.
__global__ __launch_bounds__(kPageThreads) void pages_count_kernel(PagesParams P) {
    __shared__ int64_t s_sums[kPageThreads / 64];
    const int tid = threadIdx.x;
    int count = 0;
    if (int(blockIdx.x) < P.chunks) {
        constexpr int EACH = kPageChunk / kPageThreads;
        const int64_t first = int64_t(blockIdx.x) * kPageChunk;
        const int n = int(min(int64_t(kPageChunk), P.n_pages - first));
        int refs[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) refs[e] = P.refs[first + min(tid + e * kPageThreads, n - 1)];
#pragma unroll
        for (int e = 0; e < EACH; ++e) count += tid + e * kPageThreads < n && refs[e] == 0 ? 1 : 0;
        const int64_t all = total<kPageThreads / 64>(count, s_sums);
        if (tid == 0) P.free_count[blockIdx.x] = int(all);
        return;
    }
    const int seq = int(blockIdx.x) - P.chunks;
    const int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    const int n = entries_of(P, seq);
    for (int i0 = tid; i0 < n; i0 += kEntries * kPageThreads) {
        int id[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) id[e] = table[min(i0 + e * kPageThreads, n - 1)];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) count += i0 + e * kPageThreads < n && !has_page(P, id[e]) ? 1 : 0;
    }
    const int64_t all = total<kPageThreads / 64>(count, s_sums);
    if (tid == 0) P.need[seq] = int(all);
}

// Lists the free pages by rank, and sums the needs of every kSeqBlock sequences.
__global__ __launch_bounds__(kPageThreads) void pages_list_kernel(PagesParams P) {
    __shared__ int64_t s_sums[kPageThreads / 64];
    __shared__ int s_run[kPageThreads / 64];
    const int tid = threadIdx.x;
    if (int(blockIdx.x) >= P.chunks) {
        const int block = int(blockIdx.x) - P.chunks;
        int64_t sum = 0;
        for (int i = block * kSeqBlock + tid; i < min(P.S, (block + 1) * kSeqBlock); i += kPageThreads) sum += P.need[i];
        sum = total<kPageThreads / 64>(sum, s_sums);
        if (tid == 0) P.need_sum[block] = int(min(sum, int64_t(INT32_MAX)));
        return;
    }
    // 8 consecutive pages a thread, under way beside the counts of the chunks before
    const int64_t first = int64_t(blockIdx.x) * kPageChunk + tid * (kPageChunk / kPageThreads);
    uint32_t free = 0;
#pragma unroll
    for (int i = 0; i < kPageChunk / kPageThreads; ++i)
        free |= (first + i < P.n_pages && P.refs[min(first + i, int64_t(P.n_pages - 1))] == 0 ? 1u : 0u) << i;
    int64_t rank = 0;
    for (int c = tid; c < int(blockIdx.x); c += kPageThreads) rank += P.free_count[c];
    rank = total<kPageThreads / 64>(rank, s_sums);
    int all;
    rank += before_thread<kPageThreads / 64>(__popc(free), s_run, all);
#pragma unroll
    for (int i = 0; i < kPageChunk / kPageThreads; ++i)
        if ((free >> i) & 1u) P.list[rank++] = int32_t(first + i);
}

// A sequence: pages for its entries, then the slots and positions of its new tokens.
__global__ __launch_bounds__(kAssignThreads) void pages_assign_kernel(PagesParams P) {
    constexpr int WAVES = kAssignThreads / 64;
    __shared__ int64_t s_sums[2 * WAVES];
    __shared__ int s_run[WAVES];
    const int tid = threadIdx.x, seq = blockIdx.x;
    int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    const int need = P.need[seq], n = entries_of(P, seq);
    if (need > 0) {
        // a thread's entries, the next ones under way, and the sums
        int id[kEntries];
        auto load = [&](int first) {
#pragma unroll
            for (int e = 0; e < kEntries; ++e) id[e] = table[min(first + e, n - 1)];
        };
        load(tid * kEntries);
        int64_t rank = 0, free = 0;
        for (int b = tid; b < seq / kSeqBlock; b += kAssignThreads) rank += P.need_sum[b];
        for (int b = seq / kSeqBlock * kSeqBlock + tid; b < seq; b += kAssignThreads) rank += P.need[b];
        for (int c = tid; c < P.chunks; c += kAssignThreads) free += P.free_count[c];
        totals<WAVES>(rank, free, s_sums);
        for (int i0 = 0; i0 < n; i0 += kAssignThreads * kEntries) {
            const int first = i0 + tid * kEntries;
            uint32_t want = 0;
#pragma unroll
            for (int e = 0; e < kEntries; ++e)
                want |= (first + e < n && !has_page(P, id[e]) ? 1u : 0u) << e;
            if (i0 + kAssignThreads * kEntries < n) load(first + kAssignThreads * kEntries);
            int found;
            int64_t r = rank + before_thread<WAVES>(__popc(want), s_run, found);
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                if (((want >> e) & 1u) == 0) continue;
                if (r < free) {
                    const int taken = P.list[r];
                    table[first + e] = taken;
                    P.refs[taken] = 1;
                }
                ++r;
            }
            rank += found;
        }
        if (tid == 0 && P.missing != nullptr) {
            const int64_t short_of = rank - free;  // rank: of the first entry after this sequence's
            P.missing[seq] = int(max(int64_t(0), min(short_of, int64_t(need))));
        }
        __syncthreads();
    } else if (tid == 0 && P.missing != nullptr) {
        P.missing[seq] = 0;
    }
    write_slots(P, seq, tid, kAssignThreads);
}

// N (a multiple of 4) consecutive values from `first` on, `rest` behind the last of n; 16 bytes at a time.
template <int N>
__device__ __forceinline__ void load_run(const int32_t *p, int first, int n, int rest, int (&x)[N]) {
#pragma unroll
    for (int q = 0; q < N; q += 4) {
        int4 y = make_int4(rest, rest, rest, rest);
        if (first + q + 4 <= n) {
            y = *reinterpret_cast<const int4 *>(p + first + q);
        } else {
            if (first + q < n) y.x = p[first + q];
            if (first + q + 1 < n) y.y = p[first + q + 1];
            if (first + q + 2 < n) y.z = p[first + q + 2];
        }
        x[q] = y.x;
        x[q + 1] = y.y;
        x[q + 2] = y.z;
        x[q + 3] = y.w;
    }
}

// The whole of a small reservation by one workgroup: the tables' entries are numbered as they lie in memory, and
// kept in LDS for the slots.
__global__ __launch_bounds__(kSmallThreads) void pages_small_kernel(PagesParams P) {
    constexpr int WAVES = kSmallThreads / 64, PAGES = kSmallPages / kSmallThreads, EACH = kSmallEntries / kSmallThreads;
    __shared__ int s_list[kSmallPages], s_table[kSmallEntries + kSmallEntries / EACH];
    __shared__ int s_entries[kSmallSeqs], s_first[kSmallSeqs + 1], s_run[WAVES];
    const int tid = threadIdx.x, total_entries = P.S * P.max_pages;
    // the pages' counts, the tables and the sequences' lengths are under way together
    uint32_t free = 0;
    int refs[PAGES], id[EACH];
    load_run<PAGES>(P.refs, tid * PAGES, P.n_pages, 1, refs);
    load_run<EACH>(P.pages, tid * EACH, total_entries, 0, id);
#pragma unroll
    for (int i = 0; i < PAGES; ++i) free |= (refs[i] == 0 ? 1u : 0u) << i;
    if (tid < P.S) s_entries[tid] = entries_of(P, tid);
    int all, rank = before_thread<WAVES>(__popc(free), s_run, all);
#pragma unroll
    for (int i = 0; i < PAGES; ++i)
        if ((free >> i) & 1u) s_list[rank++] = tid * PAGES + i;
    // entries without a page, by number
    uint32_t want = 0;
    {
        int seq = min(tid * EACH / P.max_pages, P.S - 1), entry = tid * EACH - seq * P.max_pages;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            if (tid * EACH + e < total_entries)
                want |= (entry < s_entries[seq] && !has_page(P, id[e]) ? 1u : 0u) << e;
            if (++entry == P.max_pages && seq + 1 < P.S) {
                entry = 0;
                ++seq;
            }
        }
    }
    int needed, r = before_thread<WAVES>(__popc(want), s_run, needed);
    {
        int seq = min(tid * EACH / P.max_pages, P.S - 1), entry = tid * EACH - seq * P.max_pages;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = tid * EACH + e;
            if (i < total_entries) {
                if (entry == 0) s_first[seq] = r;
                if ((want >> e) & 1u) {
                    if (r < all) {
                        id[e] = s_list[r];
                        P.pages[i] = id[e];
                        P.refs[id[e]] = 1;
                    }
                    ++r;
                }
                s_table[i + tid] = id[e];  // a thread's run a bank further than the last one's
            }
            if (++entry == P.max_pages && seq + 1 < P.S) {
                entry = 0;
                ++seq;
            }
        }
    }
    if (tid == 0) s_first[P.S] = needed;
    __syncthreads();
    if (tid < P.S && P.missing != nullptr) {
        const int from = s_first[tid], to = s_first[tid + 1];
        P.missing[tid] = max(0, min(to - all, to - from));
    }
    for (int seq = tid >> 6; seq < P.S; seq += WAVES) {
        const int off = P.seq_off[seq], n_new = P.seq_off[seq + 1] - off;
        const int64_t length = max(P.length[seq], 0);
        for (int i = tid & 63; i < n_new; i += 64) {
            const int64_t at = length + i, entry = at >> P.page_shift;
            int page = -1;
            if (entry < P.max_pages) {
                const int e = seq * P.max_pages + int(entry);
                page = s_table[e + e / EACH];
            }
            if (P.slots != nullptr) P.slots[off + i] = slot_of(P, has_page(P, page) ? page : -1, at);
            if (P.positions != nullptr)
                P.positions[off + i] = position_of(length, P.depth != nullptr ? P.depth[off + i] : i);
        }
    }
}

__global__ __launch_bounds__(kPageThreads) void pages_release_kernel(PagesParams P, const int32_t *keep) {
    const int seq = blockIdx.x;
    const int64_t page = int64_t(1) << P.page_shift, kept = (max(int64_t(keep[seq]), int64_t(0)) + page - 1) >> P.page_shift;
    int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    for (int64_t i = kept + threadIdx.x; i < P.max_pages; i += kPageThreads) {
        const int id = table[i];
        // the counts' order does not matter: what is left is the count less the entries, not below 0
        if (has_page(P, id)) {
            int old = P.refs[id];
            while (old > 0) {
                const int seen = atomicCAS(P.refs + id, old, old - 1);
                if (seen == old) break;
                old = seen;
            }
        }
        if (id != -1) table[i] = -1;
    }
}

namespace {

int64_t pages_bytes(const gdn_pages_args *a) {
    const int64_t chunks = (int64_t(a->n_pages) + kPageChunk - 1) / kPageChunk;
    const int64_t blocks = (int64_t(a->n_seqs) + kSeqBlock - 1) / kSeqBlock;
    return 4 * (chunks + a->n_seqs + blocks + a->n_pages);
}

gdn_status check_pages(const gdn_pages_args *a, const char *who) {
    if (a == nullptr) return fail(GDN_EINVAL, "%s: null arguments", who);
    if (a->n_seqs < 0 || a->n_seqs > kMaxSeqs || a->n_tokens < 0 || a->n_pages < 1 || a->max_pages < 1)
        return fail(GDN_EINVAL, "%s: bad n_seqs/n_tokens/n_pages/max_pages", who);
    const int32_t pt = a->page_tokens;
    if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256)
        return fail(GDN_EINVAL, "%s: page_tokens %d, must be 16, 32, 64, 128 or 256", who, pt);
    if (int64_t(a->max_pages) * pt > (int64_t(1) << 30))
        return fail(GDN_EINVAL, "%s: more than 2^30 slots a sequence", who);
    if (a->n_seqs > 0 && (!a->pages || !a->refs)) return fail(GDN_EINVAL, "%s: null pages/refs", who);
    return GDN_OK;
}

PagesParams params_of(const gdn_pages_args *a) {
    PagesParams P{};
    P.pages = a->pages;
    P.refs = a->refs;
    P.missing = a->missing;
    P.length = a->length;
    P.seq_off = a->seq_offsets;
    P.depth = a->depth;
    P.slots = a->slots;
    P.positions = a->positions;
    P.S = a->n_seqs;
    P.n_pages = a->n_pages;
    P.max_pages = a->max_pages;
    P.page_shift = log2_exact(a->page_tokens);
    P.chunks = int32_t((int64_t(a->n_pages) + kPageChunk - 1) / kPageChunk);
    P.free_count = static_cast<int32_t *>(a->workspace);
    P.need = P.free_count + P.chunks;
    P.need_sum = P.need + a->n_seqs;
    P.list = P.need_sum + (int64_t(a->n_seqs) + kSeqBlock - 1) / kSeqBlock;
    return P;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_pages_workspace_bytes(const gdn_pages_args *a) {
    clear_error();
    gdn_pages_args sizes{};
    if (a != nullptr) {
        sizes = *a;
        sizes.pages = sizes.refs = reinterpret_cast<int32_t *>(16);  // not asked for yet
    }
    if (check_pages(a != nullptr ? &sizes : nullptr, "gdn_pages_workspace_bytes") != GDN_OK || a->n_seqs == 0) return 0;
    return size_t(pages_bytes(a) + 15) & ~size_t(15);
}

extern "C" gdn_status gdn_kv_reserve(const gdn_pages_args *a, void *stream) {
    clear_error();
    const char *who = "gdn_kv_reserve";
    gdn_status st = check_pages(a, who);
    if (st != GDN_OK || a->n_seqs == 0) return st;
    if (!a->length || !a->seq_offsets) return fail(GDN_EINVAL, "%s: null length/seq_offsets", who);
    const int64_t need = pages_bytes(a);
    if (a->workspace == nullptr || a->workspace_bytes < need)
        return fail(GDN_ECAPACITY, "%s: workspace holds %lld bytes, the call needs %lld", who,
                    static_cast<long long>(a->workspace ? a->workspace_bytes : 0), static_cast<long long>(need));
    if (reinterpret_cast<uintptr_t>(a->workspace) % 16 != 0)
        return fail(GDN_EINVAL, "%s: workspace must be 16-byte aligned", who);
    const PagesParams P = params_of(a);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (P.n_pages <= kSmallPages && P.S <= kSmallSeqs && int64_t(P.S) * P.max_pages <= kSmallEntries &&
        a->n_tokens <= std::min(kSmallTokens, std::max(kSmallFew, kSmallEach * P.S)) &&
        (reinterpret_cast<uintptr_t>(P.pages) | reinterpret_cast<uintptr_t>(P.refs)) % 16 == 0) {
        hipLaunchKernelGGL(pages_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, P);
        GDN_LAUNCH_CHECK("pages_small_kernel");
        return GDN_OK;
    }
    const uint32_t blocks = uint32_t((P.S + kSeqBlock - 1) / kSeqBlock);
    hipLaunchKernelGGL(pages_count_kernel, dim3(uint32_t(P.chunks + P.S)), dim3(kPageThreads), 0, s, P);
    GDN_LAUNCH_CHECK("pages_count_kernel");
    hipLaunchKernelGGL(pages_list_kernel, dim3(uint32_t(P.chunks) + blocks), dim3(kPageThreads), 0, s, P);
    GDN_LAUNCH_CHECK("pages_list_kernel");
    hipLaunchKernelGGL(pages_assign_kernel, dim3(uint32_t(P.S)), dim3(kAssignThreads), 0, s, P);
    GDN_LAUNCH_CHECK("pages_assign_kernel");
    return GDN_OK;
}

extern "C" gdn_status gdn_kv_release(const gdn_pages_args *a, const int32_t *keep, void *stream) {
    clear_error();
    const char *who = "gdn_kv_release";
    gdn_status st = check_pages(a, who);
    if (st != GDN_OK || a->n_seqs == 0) return st;
    if (!keep) return fail(GDN_EINVAL, "%s: null keep", who);
    hipLaunchKernelGGL(pages_release_kernel, dim3(uint32_t(a->n_seqs)), dim3(kPageThreads), 0,
                       static_cast<hipStream_t>(stream), params_of(a), keep);
    GDN_LAUNCH_CHECK("pages_release_kernel");
    return GDN_OK;
}
