// Page tables and slot maps of the paged cache, built on the device (gfx950).  The rules are in
// gdn_tree.h.
//
// Reserving is a numbering: the r-th table entry without a page, in order of (sequence, entry), takes the
// r-th free page, in order of its id.  Both sides are counted first (a workgroup a chunk of pages or a
// sequence), then the free pages are listed by rank, then every sequence finds its first rank and fills
// its entries: three launches, none of which waits for another workgroup, so the result does not
// depend on the order anything runs in.  What has to be moved is the pool's reference counts and the
// tables, once; below a few thousand pages the launches are all there is to it.
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
constexpr int kPageChunk = 2048;  // pages a workgroup counts, 8 a thread
constexpr int kSeqBlock = 1024;   // sequences whose needs are summed at once

// Sum of x over the workgroup; every thread gets it.
__device__ __forceinline__ int64_t total(int64_t x, int64_t *sums) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor((long long)x, d);
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
    __syncthreads();
    return sums[0] + sums[1] + sums[2] + sums[3];
}

// Sum over the threads before this one.
__device__ __forceinline__ int before_thread(int x, int *sums) {
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
#pragma unroll
    for (int w = 0; w < kPageThreads / 64; ++w) base += w < wave ? sums[w] : 0;
    return base + run - x;
}

// Table entries that a sequence's committed and new tokens take.
__device__ __forceinline__ int entries_of(const PagesParams &P, int seq) {
    const int64_t length = max(P.length[seq], 0), n = P.seq_off[seq + 1] - P.seq_off[seq];
    const int64_t page = int64_t(1) << P.page_shift;
    return int(min((length + n + page - 1) >> P.page_shift, int64_t(P.max_pages)));
}

__device__ __forceinline__ bool has_page(const PagesParams &P, int id) { return unsigned(id) < unsigned(P.n_pages); }

}  // namespace

// Workgroups 0 .. chunks - 1 count a chunk's free pages, the others a sequence's entries without one.
__global__ __launch_bounds__(kPageThreads) void pages_count_kernel(PagesParams P) {
    __shared__ int64_t s_sums[kPageThreads / 64];
    const int tid = threadIdx.x;
    int count = 0;
    if (int(blockIdx.x) < P.chunks) {
        const int64_t first = int64_t(blockIdx.x) * kPageChunk;
        const int n = int(min(int64_t(kPageChunk), P.n_pages - first));
        for (int i = tid; i < n; i += kPageThreads) count += P.refs[first + i] == 0 ? 1 : 0;
        const int64_t all = total(count, s_sums);
        if (tid == 0) P.free_count[blockIdx.x] = int(all);
        return;
    }
    const int seq = int(blockIdx.x) - P.chunks;
    const int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    const int n = entries_of(P, seq);
    for (int i = tid; i < n; i += kPageThreads) count += has_page(P, table[i]) ? 0 : 1;
    const int64_t all = total(count, s_sums);
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
        sum = total(sum, s_sums);
        if (tid == 0) P.need_sum[block] = int(min(sum, int64_t(INT32_MAX)));
        return;
    }
    int64_t rank = 0;
    for (int c = tid; c < int(blockIdx.x); c += kPageThreads) rank += P.free_count[c];
    rank = total(rank, s_sums);
    // 8 consecutive pages a thread
    const int64_t first = int64_t(blockIdx.x) * kPageChunk + tid * (kPageChunk / kPageThreads);
    uint32_t free = 0;
#pragma unroll
    for (int i = 0; i < kPageChunk / kPageThreads; ++i)
        free |= (first + i < P.n_pages && P.refs[first + i] == 0 ? 1u : 0u) << i;
    rank += before_thread(__popc(free), s_run);
#pragma unroll
    for (int i = 0; i < kPageChunk / kPageThreads; ++i)
        if ((free >> i) & 1u) P.list[rank++] = int32_t(first + i);
}

// A sequence: pages for its entries, then the slots and positions of its new tokens.
__global__ __launch_bounds__(kPageThreads) void pages_assign_kernel(PagesParams P) {
    __shared__ int64_t s_sums[kPageThreads / 64];
    __shared__ int s_run[kPageThreads / 64];
    const int tid = threadIdx.x, seq = blockIdx.x;
    int32_t *table = P.pages + int64_t(seq) * P.max_pages;
    const int need = P.need[seq];
    if (need > 0) {
        int64_t rank = 0, free = 0;
        for (int b = tid; b < seq / kSeqBlock; b += kPageThreads) rank += P.need_sum[b];
        for (int b = seq / kSeqBlock * kSeqBlock + tid; b < seq; b += kPageThreads) rank += P.need[b];
        for (int c = tid; c < P.chunks; c += kPageThreads) free += P.free_count[c];
        rank = total(rank, s_sums);
        free = total(free, s_sums);
        const int n = entries_of(P, seq);
        for (int i0 = 0; i0 < n; i0 += kPageThreads) {
            const int i = i0 + tid;
            const bool want = i < n && !has_page(P, table[i]);
            const int64_t r = rank + before_thread(want ? 1 : 0, s_run);
            if (want && r < free) {
                const int id = P.list[r];
                table[i] = id;
                P.refs[id] = 1;
            }
            rank += __syncthreads_count(want);
        }
        if (tid == 0 && P.missing != nullptr) {
            const int64_t short_of = rank - free;  // rank: of the first entry after this sequence's
            P.missing[seq] = int(max(int64_t(0), min(short_of, int64_t(need))));
        }
        __syncthreads();
    } else if (tid == 0 && P.missing != nullptr) {
        P.missing[seq] = 0;
    }
    const int off = P.seq_off[seq], n_new = P.seq_off[seq + 1] - off;
    const int64_t length = max(P.length[seq], 0);
    for (int i = tid; i < n_new; i += kPageThreads) {
        const int64_t at = length + i;
        if (P.slots != nullptr) {
            const int id = kv_page(table, P.max_pages, P.n_pages, P.page_shift, at);
            P.slots[off + i] = id < 0 ? -1 : (int64_t(id) << P.page_shift) + (at & ((1 << P.page_shift) - 1));
        }
        if (P.positions != nullptr)
            P.positions[off + i] = int32_t(min(length + (P.depth != nullptr ? P.depth[off + i] : i), int64_t(INT32_MAX)));
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
    const uint32_t blocks = uint32_t((P.S + kSeqBlock - 1) / kSeqBlock);
    hipLaunchKernelGGL(pages_count_kernel, dim3(uint32_t(P.chunks + P.S)), dim3(kPageThreads), 0, s, P);
    GDN_LAUNCH_CHECK("pages_count_kernel");
    hipLaunchKernelGGL(pages_list_kernel, dim3(uint32_t(P.chunks) + blocks), dim3(kPageThreads), 0, s, P);
    GDN_LAUNCH_CHECK("pages_list_kernel");
    hipLaunchKernelGGL(pages_assign_kernel, dim3(uint32_t(P.S)), dim3(kPageThreads), 0, s, P);
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
