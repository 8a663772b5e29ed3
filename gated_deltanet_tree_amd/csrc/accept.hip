// Acceptance of a draft tree's tokens against the target's logits, from given random numbers
// (gfx950).  The rule is in gdn_tree.h: at every node one token is drawn from the target's softmax
// by inverting its running sum, the children's tokens first; the walk follows the child drawn.
//
// What it costs is one read of the logits, T V of them: the first launch takes each node's
// (max, sum of exponentials) in pieces of 2048 logits, one wave a piece, whose 32 values a lane
// stay in registers between the two.  Everything else is small but a chain of dependent steps, so
// it is one more launch: every workgroup of a sequence repeats the walk (the nodes' sums and the
// children's weights in parallel, then the chain from the root over LDS values), which costs no
// time that a launch of its own would not, and then takes its 2048 logits of the node where the
// walk ended.  The workgroup that finishes last joins the pieces and finds the token.
//
// Precision.  A child is accepted where u Z < c: fp32 exponentials with relative errors of some
// 2^-23 decide that wrongly only where u lies that close to a border.  The draw among the whole
// vocabulary has 10^5 borders, and a token's share may be below 2^-23: there the exponentials and
// sums are fp64.
#include "gdn_device.h"

namespace gdn {

struct AcceptParams {
    const void *logits;
    const int32_t *tokens;
    const float *uniform, *temperature;
    int32_t *path, *path_len, *next;
    float4 *stats;    // [T][pieces]: max, sum relative to it, lowest index of the max (bits)
    double *part;     // [S][pieces]: sums at the sequence's last node, without its children
    uint32_t *done;   // [S]: workgroups that have written theirs
    const int32_t *seq_off, *parent;  // schedule image, global ids
    int64_t stride;
    int32_t V, pieces, max_path, max_tree;
};

namespace {

constexpr int kPiece = 2048;   // logits a wave (first launch) or workgroup (second) takes
constexpr int kGroups = kPiece / 8;
constexpr int kAcceptThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_inff();

// Rows may start at any element: groups of eight are counted from the 16-byte boundary at or
// below the row's start.
template <typename T> __device__ __forceinline__ int misaligned(const T *row) {
    return int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

template <typename T> __device__ __forceinline__ float logit(T x) {
    const float f = to_f32<T>(x);
    return f == f ? f : -kInf;  // NaN: never drawn
}

// Logits 8 g - mis .. 8 g - mis + 7 of a row, -inf outside [0, V).
template <typename T>
__device__ __forceinline__ void load_group(const T *row, int mis, int g, int V, float *x) {
    const int first = 8 * g - mis;
    if (first >= 0 && first + 8 <= V) {
        if constexpr (sizeof(T) == 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + first);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
            const float4 a = reinterpret_cast<const float4 *>(row + first)[0];
            const float4 b = reinterpret_cast<const float4 *>(row + first)[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] : -kInf;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = first + i >= 0 && first + i < V ? logit(row[first + i]) : -kInf;
    }
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = min(x, __shfl_xor(x, d));
    return x;
}
template <typename F> __device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// exp((x - m) / T) as exp2 of half the difference times 2 log2(e) / T: the halves of two finite
// logits differ by a finite number.  The factor is finite, so that a difference of 0 gives 1; at
// T = inf it is 0, and -inf logits are the caller's to leave out.
__device__ __forceinline__ float exp2_factor(float T) { return fminf(2.f * kLog2e / T, 3.0e38f); }
__device__ __forceinline__ float weight(float x, float m, float f) {
    return __builtin_amdgcn_exp2f(fmaf(x, 0.5f, -0.5f * m) * f);
}
// The same in fp64, of any logits: next to a +inf one the others have none.
__device__ __forceinline__ double weight64(float x, float m, double inv_t) {
    if (x == -kInf) return 0.0;
    if (x == m) return 1.0;
    return m == kInf ? 0.0 : exp((double(x) - double(m)) * inv_t);
}

__device__ __forceinline__ double lane_value(double x, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), lane),
                            __builtin_amdgcn_readlane(__double2loint(x), lane));
}

// Sum of weights relative to the larger of two maxima, from the sums relative to each.
__device__ __forceinline__ float join_sums(float m1, float z1, float m2, float z2, float f) {
    const float lo = fminf(m1, m2), hi = fmaxf(m1, m2);
    const float zlo = m1 < m2 ? z1 : z2, zhi = m1 < m2 ? z2 : z1;
    if (lo == hi) return z1 + z2;
    // a -inf maximum has no weight, and next to a +inf one nothing else has
    return zlo > 0.f && hi < kInf ? zhi + zlo * weight(lo, hi, f) : zhi;
}

// Joins a lane's (maximum, sum, lowest index of the maximum) with the lane CTRL's.
template <int CTRL>
__device__ __forceinline__ void octet_join(float &m, float &z, int &arg, bool greedy, float f) {
    const float m2 = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), CTRL, 0xF, 0xF, true));
    if (greedy) {
        const int arg2 = __builtin_amdgcn_mov_dpp(arg, CTRL, 0xF, 0xF, true);
        arg = m2 > m ? arg2 : m2 == m ? min(arg, arg2) : arg;
    } else {
        const float z2 = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(z), CTRL, 0xF, 0xF, true));
        z = join_sums(m, z, m2, z2, f);
    }
    m = fmaxf(m, m2);
}

}  // namespace

template <typename TIn>
__global__ __launch_bounds__(kAcceptThreads) void accept_stats_kernel(AcceptParams P) {
    const int seq = blockIdx.z, node = blockIdx.y;
    const int off = P.seq_off[seq];
    if (blockIdx.x == 0 && node == 0 && threadIdx.x == 0) P.done[seq] = 0;
    if (node >= P.seq_off[seq + 1] - off) return;
    const int piece = blockIdx.x * (kAcceptThreads / 64) + (threadIdx.x >> 6);
    if (piece >= P.pieces) return;
    const int lane = threadIdx.x & 63;
    const float T = P.temperature[seq];
    const TIn *row = static_cast<const TIn *>(P.logits) + int64_t(off + node) * P.stride;
    const int mis = misaligned(row);
    float x[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) load_group(row, mis, piece * kGroups + 64 * k + lane, P.V, x[k]);
    float m = -kInf;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, x[k][i]);
    m = wave_max(m);
    float s = 0.f;
    int arg = P.V;
    if (T > 0.f) {
        const float f = exp2_factor(T);
        if (fabsf(m) < kInf && f > 0.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += weight(x[k][i], m, f);
        } else if (m > -kInf) {  // +inf logits share the weight; T = inf: every finite one does
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[k][i] == m || (m < kInf && x[k][i] > -kInf) ? 1.f : 0.f;
        }
        s = wave_sum(s);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (x[k][i] == m && m > -kInf)
                    arg = min(arg, 8 * (piece * kGroups + 64 * k + lane) - mis + i);
        arg = wave_min(arg);
    }
    if (lane == 0)
        P.stats[int64_t(off + node) * P.pieces + piece] = make_float4(m, s, __int_as_float(arg), 0.f);
}

// Per-node tables of the second launch, in LDS.
struct Walk {
    double *z, *w;   // sum of weights; weight of the node's own token under its parent
    float *m, *u;
    int *par, *tok;  // parent (local, -1 for the root)
};

__device__ __forceinline__ Walk walk_tables(char *mem, int n) {
    Walk t;
    t.z = reinterpret_cast<double *>(mem);
    t.w = t.z + n;
    t.m = reinterpret_cast<float *>(t.w + n);
    t.u = t.m + n;
    t.par = reinterpret_cast<int *>(t.u + n);
    t.tok = t.par + n;
    return t;
}
constexpr int kWalkBytes = 32;  // per node

template <typename TIn>
__global__ __launch_bounds__(kAcceptThreads) void accept_walk_kernel(AcceptParams P) {
    extern __shared__ __align__(16) char lds[];
    __shared__ int s_node, s_len, s_path_end, s_pick, s_arg;
    __shared__ double s_children, s_red[kAcceptThreads / 64];
    __shared__ uint32_t s_skip[kPiece / 32];
    __shared__ bool s_last;
    const int seq = blockIdx.y, piece = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int off = P.seq_off[seq], n = P.seq_off[seq + 1] - off;
    const Walk t = walk_tables(lds, P.max_tree);
    const float T = P.temperature[seq];
    const bool greedy = !(T > 0.f);
    const double inv_t = greedy ? 0.0 : 1.0 / double(T);
    const TIn *logits = static_cast<const TIn *>(P.logits);

    // ---- every node's sum, every child's weight ------------------------------------------
    for (int i = tid; i < n; i += kAcceptThreads) {
        const int up = P.parent[off + i];
        t.par[i] = up < 0 ? -1 : up - off;
        t.tok[i] = up < 0 ? -1 : P.tokens[off + i];
        t.u[i] = P.uniform[int64_t(seq) * P.max_path + i];
    }
    // eight lanes a node, so that a tree of 32 nodes waits for its sums' pieces once
    const float f = greedy ? 0.f : exp2_factor(T);
    for (int i0 = 0; i0 < n; i0 += kAcceptThreads / 8) {
        const int i = min(i0 + (tid >> 3), n - 1);
        const float4 *st = P.stats + int64_t(off + i) * P.pieces;
        float m = -kInf, z = 0.f;
        int arg = P.V;
#pragma unroll 8
        for (int c = tid & 7; c < P.pieces; c += 8) {
            const float4 a = st[c];
            if (greedy) {
                arg = a.x > m ? __float_as_int(a.z) : a.x == m ? min(arg, __float_as_int(a.z)) : arg;
            } else {
                z = join_sums(m, z, a.x, a.y, f);
            }
            m = fmaxf(m, a.x);
        }
        octet_join<0xB1>(m, z, arg, greedy, f);
        octet_join<0x4E>(m, z, arg, greedy, f);
        octet_join<0x141>(m, z, arg, greedy, f);
        if ((tid & 7) == 0 && i0 + (tid >> 3) < n) {
            t.m[i] = m;
            // greedy: all the weight is on one token, whose index takes the sum's place
            t.z[i] = greedy ? double(arg) : double(z);
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kAcceptThreads) {
        const int p = t.par[i], tok = t.tok[i];
        double w = 0.0;
        if (p >= 0 && tok >= 0 && tok < P.V) {
            const float m = t.m[p];
            if (greedy) {
                w = m > -kInf && double(tok) == t.z[p] ? 1.0 : 0.0;
            } else {
                const float l = logit(logits[int64_t(off + p) * P.stride + tok]);
                w = weight64(l, m, inv_t);
            }
            // the first sibling with a token has its weight
            bool repeated = false;
#pragma unroll 4
            for (int j = p + 1; j < i; ++j) repeated |= (t.par[j] == p) & (t.tok[j] == tok);
            if (repeated) w = 0.0;
        }
        t.w[i] = w;
    }
    __syncthreads();

    // ---- the walk, by the first wave -----------------------------------------------------
    if (wave == 0) {
        int node = 0, len = 0, pick = -1;
        double children = 0.0;
        bool none = false;
        for (;;) {
            if (piece == 0 && lane == 0) P.path[int64_t(seq) * P.max_path + len] = node;
            const float m = t.m[node];
            const double theta = greedy ? 0.5 : double(t.u[len]) * t.z[node];
            ++len;
            children = 0.0;
            int next = -1, last_child = -1;
            for (int base = node + 1; base < n && next < 0; base += 64) {
                const int mine = min(base + lane, n - 1);
                const bool kid = base + lane < n && t.par[mine] == node;
                const double w = kid ? t.w[mine] : 0.0;
                uint64_t kids = __ballot(kid);
                while (kids != 0 && next < 0) {
                    const int l = __builtin_ctzll(kids);
                    kids &= kids - 1;
                    const double wl = lane_value(w, l);
                    children += wl;
                    if (wl > 0.0) last_child = base + l;
                    if (theta < children) next = base + l;
                }
            }
            if (next >= 0) {
                node = next;
                continue;
            }
            none = m == -kInf;
            pick = last_child >= 0 ? t.tok[last_child] : -1;
            break;
        }
        if (lane == 0) {
            s_node = node;
            s_len = len;
            s_children = children;
            s_pick = pick;  // drawn only where no other token has weight
            s_arg = none ? -1 : greedy ? int(t.z[node]) : -1;
            s_path_end = none ? 1 : 0;
        }
    }
    __syncthreads();
    const int node = s_node, len = s_len;
    const bool none = s_path_end != 0;
    if (piece == 0) {
        for (int i = len + tid; i < P.max_path; i += kAcceptThreads)
            P.path[int64_t(seq) * P.max_path + i] = -1;
        if (tid == 0) {
            P.path_len[seq] = len;
            if (none || greedy) P.next[seq] = s_arg;
        }
    }
    if (none || greedy) return;

    // ---- fp64 weights of this piece of the last node's logits, without its children ---------
    const TIn *row = logits + int64_t(off + node) * P.stride;
    const int mis = misaligned(row);
    const float m = t.m[node];
    auto weights = [&](int pc, double *w) {
        for (int i = tid; i < kPiece / 32; i += kAcceptThreads) s_skip[i] = 0;
        __syncthreads();
        const int first = pc * kPiece - mis;
        for (int i = node + 1 + tid; i < n; i += kAcceptThreads) {
            const int64_t b = int64_t(t.tok[i]) - first;
            if (t.par[i] == node && t.tok[i] >= 0 && b >= 0 && b < kPiece)
                atomicOr(&s_skip[b >> 5], 1u << (b & 31));
        }
        __syncthreads();
        float x[8];
        load_group(row, mis, pc * kGroups + tid, P.V, x);
        const uint32_t skip = s_skip[tid >> 2] >> (8 * (tid & 3));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = (skip >> i) & 1u ? 0.0 : weight64(x[i], m, inv_t);
        }
    };
    double w[8];
    weights(piece, w);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += w[i];
    sum = wave_sum(sum);
    if (lane == 0) s_red[wave] = sum;
    __syncthreads();
    double *part = P.part + int64_t(seq) * P.pieces;
    if (tid == 0) {
        __hip_atomic_store(&part[piece], (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __threadfence();
        const uint32_t before = __hip_atomic_fetch_add(&P.done[seq], 1u, __ATOMIC_ACQ_REL,
                                                       __HIP_MEMORY_SCOPE_AGENT);
        s_last = before + 1 == uint32_t(P.pieces);
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();

    // ---- the last workgroup: which piece, then which token ----------------------------------
    if (wave == 0) {
        // each lane sums a run of consecutive pieces
        const int per = (P.pieces + 63) / 64, c0 = min(lane * per, P.pieces), c1 = min(c0 + per, P.pieces);
        double mine = 0.0;
        for (int c = c0; c < c1; ++c)
            mine += __hip_atomic_load(&part[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        double run = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_up(run, d);
            if (lane >= d) run += up;
        }
        const double rest = __shfl(run, 63);
        const double target = double(t.u[len - 1]) * (s_children + rest) - s_children;
        // first piece whose running sum exceeds the target; behind rounding, the last with weight
        int found = -1, heavy = -1;
        double before = run - mine, at = 0.0;
        for (int c = c0; c < c1; ++c) {
            const double p = __hip_atomic_load(&part[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (p > 0.0) heavy = c;
            if (found < 0 && p > 0.0 && before + p > target) {
                found = c;
                at = before;
            }
            before += p;
        }
        const uint64_t any = __ballot(found >= 0), weighty = __ballot(heavy >= 0);
        if (any != 0) {
            const int l = __ffsll(static_cast<unsigned long long>(any)) - 1;
            found = __shfl(found, l);
            at = __shfl(at, l);
        } else if (weighty != 0) {
            found = __shfl(heavy, 63 - __builtin_clzll(weighty));
            at = -1.0;  // its last token
        }
        if (lane == 0) {
            s_node = found;
            s_red[0] = target;
            s_red[1] = at;
        }
    }
    __syncthreads();
    const int found = s_node;
    const double target = s_red[0], at = s_red[1];
    if (found < 0) {  // all the weight is the children's
        if (tid == 0) P.next[seq] = s_pick;
        return;
    }
    weights(found, w);
    double mine = 0.0;
    int last = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mine += w[i];
        if (w[i] > 0.0) last = i;
    }
    double run = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(run, d);
        if (lane >= d) run += up;
    }
    __syncthreads();  // the target has been read
    if (lane == 63) s_red[wave] = run;
    if (tid == 0) s_arg = P.V, s_pick = -1;
    __syncthreads();
    double before = at + (run - mine);
    for (int i = 0; i < wave; ++i) before += s_red[i];
    const int first = found * kPiece - mis + 8 * tid;
    if (at >= 0.0) {
        int hit = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            before += w[i];
            if (hit < 0 && w[i] > 0.0 && before > target) hit = first + i;
        }
        if (hit >= 0) atomicMin(&s_arg, hit);
    }
    if (last >= 0) atomicMax(&s_pick, first + last);
    __syncthreads();
    if (tid == 0) P.next[seq] = s_arg < P.V ? s_arg : s_pick;
}

namespace {

int32_t pieces_of(int32_t vocab) {
    // up to seven elements of a row's first group may lie before its start
    return int32_t((int64_t(vocab) + 7 + kPiece - 1) / kPiece);
}

int64_t accept_bytes(int64_t S, int64_t T, int32_t vocab) {
    const int64_t pieces = pieces_of(vocab);
    return T * pieces * int64_t(sizeof(float4)) + S * pieces * int64_t(sizeof(double)) + S * 4;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_accept_workspace_bytes(int32_t n_seqs, int32_t n_nodes, int32_t vocab) {
    clear_error();
    if (n_seqs < 0 || n_nodes < 0 || vocab < 1) return 0;
    return size_t(accept_bytes(n_seqs, n_nodes, vocab) + 15) & ~size_t(15);
}

extern "C" gdn_status gdn_tree_accept(const gdn_accept_args *a, const int32_t *host_image,
                                      const int32_t *dev_image, void *stream) {
    clear_error();
    if (a == nullptr) return fail(GDN_EINVAL, "gdn_tree_accept: null arguments");
    if (!image_ok(host_image) || dev_image == nullptr)
        return fail(GDN_EINVAL, "gdn_tree_accept: missing or malformed schedule image");
    const ImageView v = view_image(host_image);
    if (v.n_seqs != a->n_seqs || v.n_nodes != a->n_nodes)
        return fail(GDN_EINVAL, "gdn_tree_accept: n_seqs/n_nodes differ from the schedule's");
    if (a->in_dtype != GDN_F32 && a->in_dtype != GDN_BF16)
        return fail(GDN_EINVAL, "gdn_tree_accept: in_dtype %d", a->in_dtype);
    if (a->vocab < 1 || a->vocab > (1 << 30) || a->logit_stride < a->vocab)
        return fail(GDN_EINVAL, "gdn_tree_accept: vocab %d, logit_stride %lld", a->vocab,
                    static_cast<long long>(a->logit_stride));
    if (a->n_seqs == 0) return GDN_OK;
    if (a->max_path < v.max_tree)
        return fail(GDN_ECAPACITY, "gdn_tree_accept: max_path %d < largest tree %d", a->max_path,
                    v.max_tree);
    if (a->n_seqs > 65535) return fail(GDN_EINVAL, "gdn_tree_accept: n_seqs must be <= 65535");
    const void *ptrs[] = {a->logits, a->tokens, a->uniform, a->temperature, a->path, a->path_len,
                          a->next_token, a->workspace};
    for (const void *p : ptrs)
        if (p == nullptr) return fail(GDN_EINVAL, "gdn_tree_accept: null device pointer");
    const size_t size = a->in_dtype == GDN_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(a->logits) % size != 0 ||
        reinterpret_cast<uintptr_t>(a->workspace) % 16 != 0)
        return fail(GDN_EINVAL, "gdn_tree_accept: misaligned logits or workspace");
    const int64_t need = accept_bytes(a->n_seqs, a->n_nodes, a->vocab);
    if (a->workspace_bytes < need)
        return fail(GDN_ECAPACITY, "gdn_tree_accept: workspace holds %lld bytes, the call needs %lld",
                    static_cast<long long>(a->workspace_bytes), static_cast<long long>(need));
    AcceptParams P{};
    P.logits = a->logits;
    P.tokens = a->tokens;
    P.uniform = a->uniform;
    P.temperature = a->temperature;
    P.path = a->path;
    P.path_len = a->path_len;
    P.next = a->next_token;
    P.pieces = pieces_of(a->vocab);
    P.stats = static_cast<float4 *>(a->workspace);
    P.part = reinterpret_cast<double *>(P.stats + int64_t(a->n_nodes) * P.pieces);
    P.done = reinterpret_cast<uint32_t *>(P.part + int64_t(a->n_seqs) * P.pieces);
    P.seq_off = dev_image + v.off_seq;
    P.parent = dev_image + v.off_parent;
    P.stride = a->logit_stride;
    P.V = a->vocab;
    P.max_path = a->max_path;
    P.max_tree = v.max_tree;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 g1((P.pieces + 3) / 4, v.max_tree, a->n_seqs), g2(P.pieces, a->n_seqs);
    const uint32_t bytes = uint32_t(v.max_tree) * kWalkBytes;
    if (int64_t(g1.x) * g1.y * g1.z > kMaxBlocks || int64_t(g2.x) * g2.y > kMaxBlocks)
        return fail(GDN_EINVAL, "gdn_tree_accept: too many workgroups");
    if (a->in_dtype == GDN_BF16) {
        hipLaunchKernelGGL(accept_stats_kernel<bf16_t>, g1, dim3(kAcceptThreads), 0, s, P);
        GDN_LAUNCH_CHECK("accept_stats_kernel");
        hipLaunchKernelGGL(accept_walk_kernel<bf16_t>, g2, dim3(kAcceptThreads), bytes, s, P);
    } else {
        hipLaunchKernelGGL(accept_stats_kernel<float>, g1, dim3(kAcceptThreads), 0, s, P);
        GDN_LAUNCH_CHECK("accept_stats_kernel");
        hipLaunchKernelGGL(accept_walk_kernel<float>, g2, dim3(kAcceptThreads), bytes, s, P);
    }
    GDN_LAUNCH_CHECK("accept_walk_kernel");
    return GDN_OK;
}
