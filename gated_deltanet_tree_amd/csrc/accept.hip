// Acceptance of a draft tree's tokens against the target's logits, from given random numbers
// (gfx950).  The rule is in gdn_tree.h: at every node one token is drawn from the target's softmax
// by inverting its running sum, the children's tokens first; the walk follows the child drawn.
//
// What it costs is one read of the logits, T V of them: the first launch takes each node's
// (max, sum of exponentials) in pieces of 2048 logits, one wave a piece, whose 32 values a lane
// stay in registers between the two (32 trees of 22 nodes, 131072 bf16 logits: 184 MB in 32.1 us of
// the call's 60.9, 5.7 TB/s from HBM and the memory-side cache).  Everything else is small but a
// chain of dependent steps: the walk (all nodes' sums and all children's weights side by side, then the
// chain from the root over LDS values), the sums of the last node's weights in segments of 512, and the
// draw, which goes over one segment again.  They are launches of their own: a workgroup that waits for
// its sequence's others by a counter has to write its L2 back first, which with 65 workgroups for each
// of 32 trees took 60 us, the three launches take 25.
//
// Precision.  A child is accepted where u Z < c.  Z is summed in fp32, the children's weights in fp64;
// where the two sides lie within the fp32 sum's error of one another (about 3 in 10^5 children, with
// 131072 logits) the workgroup sums Z again in fp64 and the walk decides by that, as the draw does: the
// whole vocabulary has 10^5 borders, and a token's share may be below 2^-23.  Being able to costs 0.5
// to 1.8 us a call (16.9 -> 17.4 for 1 tree, 53.6 -> 54.4 for 32 that all draw).
//
// Error of the fp32 Z, in units of u = 2^-24 of Z.  An exponent x log2(e) / T of size a is off by 5 u a at
// most (the fused difference, the product, the factor), its weight by ln 2 of that; over a node the
// mean of a is at most log2 V, as sum p_j (-log2 w_j) = entropy - log2 Z and Z >= 1: 3.5 log2 V.  exp2 adds 2,
// the sums in a piece 31 + 6, and every join of pieces 4 (its factor's exponents add up to those of
// the weights): ceil(pieces / 16) + 4 joins.  In all 3.5 log2 V + 39 + 4 (pieces / 16 + 5), below 200 + pieces / 2
// up to V = 2^30.
#include "logits.h"

namespace gdn {

// Where a walk ended, for the draw among the vocabulary.
struct Last {
    double children;  // weight of the node's children
    int32_t node;     // -1: there is nothing to draw
    int32_t kids;     // children
    int32_t pick;     // token to take if only children have weight
    float m, u;       // largest logit; random number
    int32_t reserved;
};

struct AcceptParams {
    const void *logits;
    const int32_t *tokens;
    const float *uniform, *temperature;
    int32_t *path, *path_len, *next;
    float2 *stats;    // [T][pieces]: max, and the sum relative to it (greedy: the max's lowest index)
    double *part;     // [S][4 pieces]: sums of 512 logits of the sequence's last node, without its children
    Last *last;       // [S]: where each walk ended
    int32_t *kids;    // [T]: the tokens of that node's children, from the sequence's first node on
    const int32_t *seq_off, *parent;  // schedule image, global ids
    int64_t stride;
    int32_t V, pieces, max_path, max_tree;
};

namespace {

constexpr int kPiece = 2048;    // logits a wave of the first launch takes
constexpr int kGroups = kPiece / 8;
constexpr int kSegment = 512;   // logits a wave of the second launch takes at a time
constexpr int kAcceptThreads = 256, kWalkThreads = 512;
constexpr float kLog2e = 1.44269504088896340736f;

// exp((x - m) / T) as exp2 of half the difference times 2 log2(e) / T: the halves of two finite
// logits differ by a finite number.  The factor is finite, so that a difference of 0 gives 1; at
// T = inf it is 0, and -inf logits are the caller's to leave out.
__device__ __forceinline__ float exp2_factor(float T) { return fminf(2.f * kLog2e / T, 3.0e38f); }
__device__ __forceinline__ float weight(float x, float m, float f) {
    return __builtin_amdgcn_exp2f(fmaf(x, 0.5f, -0.5f * m) * f);
}
// The same in fp64, of any logits: next to a +inf one the others have none (and x = m = -inf has none).
__device__ __forceinline__ double weight64(float x, float m, double inv_t) {
    // selects, not branches: a thread's eight exponentials run side by side
    const double e = exp((double(x) - double(m)) * inv_t);
    return x == -kInf ? 0.0 : x == m ? 1.0 : m == kInf ? 0.0 : e;
}

// This thread's share of a row's weights, summed in fp64; `threads` share it.
template <typename T>
__device__ __forceinline__ double exact_share(const T *row, int V, float m, double inv_t, int threads) {
    const int mis = misaligned(row);
    double s = 0.0;
    for (int g = threadIdx.x; 8 * g - mis < V; g += threads) {
        float x[8];
        load_group(row, mis, g, V, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s += weight64(x[i], m, inv_t);
            __builtin_amdgcn_sched_barrier(0);  // rare: not worth the registers of several side by side
        }
    }
    return s;
}

// LDS accesses of one wave stay in program order across its lanes.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Running sum over the lanes of a wave, own value included.
__device__ __forceinline__ double wave_scan(double x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(x, d);
        if (lane >= d) x += up;
    }
    return x;
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
__device__ __forceinline__ void row_join(float &m, float &z, int &arg, bool greedy, float f) {
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
        P.stats[int64_t(off + node) * P.pieces + piece] = make_float2(m, T > 0.f ? s : __int_as_float(arg));
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

// The walk, by one workgroup: writes the path (if `writes`) and where it ended, its children's tokens
// to `kids`.
template <typename TIn>
__device__ __forceinline__ void walk_tree(const AcceptParams &P, int seq, char *lds, Last &s_last, int *kids,
                                          bool writes) {
    __shared__ int s_len, s_ask;
    __shared__ double s_sum[kWalkThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int off = P.seq_off[seq], n = P.seq_off[seq + 1] - off;
    const Walk t = walk_tables(lds, P.max_tree);
    const float T = P.temperature[seq];
    const bool greedy = !(T > 0.f);
    const double inv_t = greedy ? 0.0 : 1.0 / double(T);
    const TIn *logits = static_cast<const TIn *>(P.logits);

    // ---- every node's sum, every child's weight ------------------------------------------
    // The logit of a child's token is asked for before its parent's sum is known; for the first 512
    // nodes, one a thread.
    float child_logit = -kInf;
    for (int i = tid; i < n; i += kWalkThreads) {
        const int up = P.parent[off + i], p = up < 0 ? -1 : up - off;
        const int tok = up < 0 ? -1 : P.tokens[off + i];
        t.u[i] = P.uniform[int64_t(seq) * P.max_path + i];
        t.par[i] = p;
        t.tok[i] = tok;
        if (i == tid && p >= 0 && tok >= 0 && tok < P.V)
            child_logit = logit(logits[int64_t(off + p) * P.stride + tok]);
    }
    // a row of 16 lanes a node, so that a tree of 32 nodes waits for its sums' pieces once
    const float f = greedy ? 0.f : exp2_factor(T);
    for (int i0 = 0; i0 < n; i0 += kWalkThreads / 16) {
        const int i = min(i0 + (tid >> 4), n - 1);
        const float2 *st = P.stats + int64_t(off + i) * P.pieces;
        float m = -kInf, z = 0.f;
        int arg = P.V;
        for (int c = tid & 15; c < P.pieces; c += 128) {
            float2 a[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                a[k] = c + 16 * k < P.pieces ? st[c + 16 * k] : make_float2(-kInf, greedy ? __int_as_float(P.V) : 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (greedy) {
                    const int x = __float_as_int(a[k].y);
                    arg = a[k].x > m ? x : a[k].x == m ? min(arg, x) : arg;
                } else {
                    z = join_sums(m, z, a[k].x, a[k].y, f);
                }
                m = fmaxf(m, a[k].x);
            }
        }
        row_join<0xB1>(m, z, arg, greedy, f);
        row_join<0x4E>(m, z, arg, greedy, f);
        row_join<0x141>(m, z, arg, greedy, f);
        row_join<0x128>(m, z, arg, greedy, f);
        if ((tid & 15) == 0 && i0 + (tid >> 4) < n) {
            t.m[i] = m;
            // greedy: all the weight is on one token, whose index takes the sum's place
            t.z[i] = greedy ? double(arg) : double(z);
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kWalkThreads) {
        const int p = t.par[i], tok = t.tok[i];
        double w = 0.0;
        if (p >= 0 && tok >= 0 && tok < P.V) {
            const float m = t.m[p];
            if (greedy) {
                w = m > -kInf && double(tok) == t.z[p] ? 1.0 : 0.0;
            } else {
                const float l = i == tid ? child_logit : logit(logits[int64_t(off + p) * P.stride + tok]);
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
    // It stops where a child's border is too near to tell, until all waves have summed the node's
    // weights in fp64, and looks at the node's children anew.
    const double border = (200.0 + 0.5 * P.pieces) * 0x1p-24;  // of Z: the fp32 sum's error
    int node = 0, len = 0, summed = -1;
    double z = 0.0;  // of the node `summed`
    for (;;) {
        if (wave == 0) {
            int pick = -1, ask = -1;
            double children = 0.0;
            bool none = false;
            for (;;) {
                if (writes && lane == 0) P.path[int64_t(seq) * P.max_path + len] = node;
                const float m = t.m[node];
                const bool sure = greedy || summed == node;
                if (summed != node) z = t.z[node];
                const double theta = greedy ? 0.5 : double(t.u[len]) * z, near = sure ? 0.0 : border * z;
                const double low = theta - near, high = theta + near;
                children = 0.0;
                int next = -1, last_child = -1;
                for (int base = node + 1; base < n && next < 0 && ask < 0; base += 64) {
                    const int mine = min(base + lane, n - 1);
                    const bool kid = base + lane < n && t.par[mine] == node;
                    const double w = kid ? t.w[mine] : 0.0;
                    uint64_t kids = __ballot(kid);
                    while (kids != 0 && next < 0 && ask < 0) {
                        const int l = __builtin_ctzll(kids);
                        kids &= kids - 1;
                        const double wl = lane_value(w, l);
                        children += wl;
                        if (wl > 0.0) last_child = base + l;
                        if (children >= low) {
                            if (children > high)
                                next = base + l;
                            else if (!sure && wl > 0.0)
                                ask = node;
                        }
                    }
                }
                if (ask >= 0) break;
                ++len;
                if (next >= 0) {
                    node = next;
                    continue;
                }
                none = m == -kInf;
                pick = last_child >= 0 ? t.tok[last_child] : -1;
                break;
            }
            if (lane == 0) s_ask = ask;
            if (ask < 0) {
                // the children's tokens, in any order
                int count = 0;
                for (int base = node + 1; base < n; base += 64) {
                    const int mine = min(base + lane, n - 1);
                    const bool kid = base + lane < n && t.par[mine] == node;
                    const uint64_t who = __ballot(kid);
                    if (kid) kids[count + __popcll(who & ((1ull << lane) - 1))] = t.tok[mine];
                    count += __popcll(who);
                }
                if (writes)
                    for (int i = lane; i < count; i += 64) P.kids[off + i] = kids[i];
                if (lane == 0) {
                    s_len = len;
                    s_last.children = children;
                    s_last.node = none || greedy ? -1 : node;
                    s_last.kids = count;
                    s_last.pick = pick;  // drawn only where no other token has weight
                    s_last.m = t.m[node];
                    s_last.u = t.u[len - 1];
                    if (writes) {
                        P.last[seq] = s_last;
                        P.path_len[seq] = len;
                        if (none || greedy) P.next[seq] = none ? -1 : int(t.z[node]);
                    }
                }
            }
        }
        __syncthreads();
        const int ask = s_ask;
        if (ask < 0) break;
        const double share =
            wave_sum(exact_share(logits + int64_t(off + ask) * P.stride, P.V, t.m[ask], inv_t, kWalkThreads));
        if (lane == 0) s_sum[wave] = share;
        __syncthreads();
        summed = ask;
        z = 0.0;
        for (int i = 0; i < kWalkThreads / 64; ++i) z += s_sum[i];
    }
    if (writes)
        for (int i = s_len + tid; i < P.max_path; i += kWalkThreads) P.path[int64_t(seq) * P.max_path + i] = -1;
}

// Weights of a segment of the last node's logits, eight a lane, without the node's children, and
// their running sum over the wave.  skip: 16 words of LDS of the wave's own.
template <typename TIn>
__device__ __forceinline__ double segment_weights(const AcceptParams &P, const TIn *row, int segment, const Last &last,
                                                  const int *kids, double inv_t, uint32_t *skip, double (&w)[8],
                                                  int &first) {
    const int lane = threadIdx.x & 63;
    const int mis = misaligned(row);
    if (lane < kSegment / 32) skip[lane] = 0;
    wave_order();
    first = segment * kSegment - mis;
    for (int i = lane; i < last.kids; i += 64) {
        const int64_t b = int64_t(kids[i]) - first;
        if (kids[i] >= 0 && b >= 0 && b < kSegment) atomicOr(&skip[b >> 5], 1u << (b & 31));
    }
    float x[8];
    load_group(row, mis, segment * (kSegment / 8) + lane, P.V, x);
    wave_order();
    const uint32_t mine = skip[lane >> 2] >> (8 * (lane & 3));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = (mine >> i) & 1u ? 0.0 : weight64(x[i], last.m, inv_t);
        sum += w[i];
    }
    return wave_scan(sum);
}

// Sums of the four segments of a piece, a wave each.
template <typename TIn>
__device__ __forceinline__ void piece_sums(const AcceptParams &P, int seq, int piece, const Last &last, const int *kids) {
    __shared__ uint32_t s_skip[kWalkThreads / 64][kSegment / 32];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, segment = 4 * piece + wave % 4;
    const TIn *row = static_cast<const TIn *>(P.logits) + int64_t(P.seq_off[seq] + last.node) * P.stride;
    double w[8];
    int first;
    const double run = segment_weights(P, row, segment, last, kids, 1.0 / double(P.temperature[seq]), s_skip[wave], w, first);
    if (lane == 63) P.part[int64_t(seq) * 4 * P.pieces + segment] = run;
}

// Walk and sums in one launch: every workgroup of a sequence repeats the walk.
template <typename TIn>
__global__ __launch_bounds__(kWalkThreads) void accept_walk_sums_kernel(AcceptParams P) {
    extern __shared__ __align__(16) char lds[];
    __shared__ Last s_last;
    int *kids = reinterpret_cast<int *>(lds + P.max_tree * kWalkBytes);
    const int seq = blockIdx.y, wave = threadIdx.x >> 6;
    walk_tree<TIn>(P, seq, lds, s_last, kids, blockIdx.x == 0);
    if (s_last.node < 0) return;
    const int piece = 2 * blockIdx.x + wave / 4;
    if (piece < P.pieces) piece_sums<TIn>(P, seq, piece, s_last, kids);
}

// The walk alone, one workgroup a sequence.
template <typename TIn>
__global__ __launch_bounds__(kWalkThreads) void accept_walk_kernel(AcceptParams P) {
    extern __shared__ __align__(16) char lds[];
    __shared__ Last s_last;
    walk_tree<TIn>(P, blockIdx.x, lds, s_last, reinterpret_cast<int *>(lds + P.max_tree * kWalkBytes), true);
}

// The sums alone.
template <typename TIn>
__global__ __launch_bounds__(256) void accept_sums_kernel(AcceptParams P) {
    const Last last = P.last[blockIdx.y];
    if (last.node < 0) return;
    piece_sums<TIn>(P, blockIdx.y, blockIdx.x, last, P.kids + P.seq_off[blockIdx.y]);
}

// The draw from the sums: the segment it falls into, then the token; a wave a sequence.
template <typename TIn>
__global__ __launch_bounds__(64) void accept_draw_kernel(AcceptParams P) {
    __shared__ uint32_t s_skip[kSegment / 32];
    const int seq = blockIdx.x, lane = threadIdx.x;
    const Last last = P.last[seq];
    if (last.node < 0) return;
    const int segments = 4 * P.pieces;
    const double *part = P.part + int64_t(seq) * segments;
    // each lane takes a run of consecutive segments
    const int per = (segments + 63) / 64, c0 = min(lane * per, segments), c1 = min(c0 + per, segments);
    double own = 0.0;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) own += part[c];
    const double incl = wave_scan(own), rest = lane_value(incl, 63);
    double target = double(last.u) * (last.children + rest) - last.children;
    // first segment whose sum passes the target; behind rounding, the last with weight
    int segment = -1, heavy = -1;
    double before = incl - own, at = 0.0;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        const double p = part[c];
        if (p > 0.0) {
            heavy = c;
            if (segment < 0 && before + p > target) {
                segment = c;
                at = before;
            }
        }
        before += p;
    }
    const uint64_t any = __ballot(segment >= 0), some = __ballot(heavy >= 0);
    if (some != 0) heavy = __builtin_amdgcn_readlane(heavy, 63 - __builtin_clzll(some));
    if (any != 0) {
        const int l = __builtin_ctzll(any);
        segment = __builtin_amdgcn_readlane(segment, l);
        at = lane_value(at, l);
    } else {
        segment = -1;
    }
    if (some == 0) {  // all the weight is the children's
        if (lane == 0) P.next[seq] = last.pick;
        return;
    }
    if (segment < 0) {
        segment = heavy;
        target = __builtin_inf();
    }
    const TIn *row = static_cast<const TIn *>(P.logits) + int64_t(P.seq_off[seq] + last.node) * P.stride;
    double w[8];
    int first;
    const double run = segment_weights(P, row, segment, last, P.kids + P.seq_off[seq],
                                       1.0 / double(P.temperature[seq]), s_skip, w, first);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += w[i];
    // the first token whose running sum passes the target; behind rounding, the segment's last
    int hit = P.V, end = -1;
    double upto = at + (run - sum);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        upto += w[i];
        if (w[i] > 0.0) {
            end = first + 8 * lane + i;
            if (hit == P.V && upto > target) hit = end;
        }
    }
    hit = wave_min(hit);
    end = -wave_min(-end);
    if (lane == 0) P.next[seq] = hit < P.V ? hit : end;
}

namespace {

int32_t pieces_of(int32_t vocab) {
    // up to seven elements of a row's first group may lie before its start
    return int32_t((int64_t(vocab) + 7 + kPiece - 1) / kPiece);
}

// Up to this many pieces in all, walk and sums are one launch, whose workgroups, of two pieces, each
// repeat the walk; they must all run at once, and the device holds three a CU, 1536 pieces.  us a call
// in one launch / in two, trees of 22 nodes over 131072 bf16 logits (65 pieces a tree): 19.3 / 20.8 for 1
// tree, 29.0 / 29.7 for 8, 36.6 / 37.8 for 16, 43.2 / 43.5 for 22, 50.6 / 45.3 for 24, 56.8 / 52.6 for 32; over
// 65536, 42.5 / 43.1 for 44, 49.8 / 45.1 for 48; over 32000, 32.6 / 33.4 for 48.  With larger trees two are
// ahead somewhat earlier, by less: 64 nodes 64.1 / 65.4 for 16, 88.8 / 89.0 for 22, 104.6 / 95.2 for 24; 250
// nodes 128.4 / 128.6 for 8, 221.5 / 214.7 for 16; 1000 nodes 292.6 / 299.7 for 4, 492.7 / 471.3 for 8.
constexpr int64_t kOneLaunch = 1500;

int64_t accept_bytes(int64_t S, int64_t T, int32_t vocab) {
    const int64_t pieces = pieces_of(vocab);
    return S * int64_t(sizeof(Last)) + S * pieces * 4 * int64_t(sizeof(double)) +
           T * pieces * int64_t(sizeof(float2)) + T * 4;
}

template <typename TIn>
gdn_status launch_accept(const AcceptParams &P, int S, dim3 g1, dim3 g2, hipStream_t s) {
    const uint32_t bytes = uint32_t(P.max_tree) * (kWalkBytes + 4);
    const dim3 threads(kAcceptThreads);
    hipLaunchKernelGGL(accept_stats_kernel<TIn>, g1, threads, 0, s, P);
    GDN_LAUNCH_CHECK("accept_stats_kernel");
    if (int64_t(g2.x) * g2.y <= kOneLaunch) {
        hipLaunchKernelGGL(accept_walk_sums_kernel<TIn>, dim3((g2.x + 1) / 2, S), dim3(kWalkThreads), bytes, s, P);
        GDN_LAUNCH_CHECK("accept_walk_sums_kernel");
    } else {
        hipLaunchKernelGGL(accept_walk_kernel<TIn>, dim3(S), dim3(kWalkThreads), bytes, s, P);
        GDN_LAUNCH_CHECK("accept_walk_kernel");
        hipLaunchKernelGGL(accept_sums_kernel<TIn>, g2, threads, 0, s, P);
        GDN_LAUNCH_CHECK("accept_sums_kernel");
    }
    hipLaunchKernelGGL(accept_draw_kernel<TIn>, dim3(S), dim3(64), 0, s, P);
    GDN_LAUNCH_CHECK("accept_draw_kernel");
    return GDN_OK;
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
    P.last = static_cast<Last *>(a->workspace);
    P.part = reinterpret_cast<double *>(P.last + a->n_seqs);
    P.stats = reinterpret_cast<float2 *>(P.part + int64_t(a->n_seqs) * P.pieces * 4);
    P.kids = reinterpret_cast<int32_t *>(P.stats + int64_t(a->n_nodes) * P.pieces);
    P.seq_off = dev_image + v.off_seq;
    P.parent = dev_image + v.off_parent;
    P.stride = a->logit_stride;
    P.V = a->vocab;
    P.max_path = a->max_path;
    P.max_tree = v.max_tree;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 g1((P.pieces + 3) / 4, v.max_tree, a->n_seqs), g2(P.pieces, a->n_seqs);
    if (int64_t(g1.x) * g1.y * g1.z > kMaxBlocks || int64_t(g2.x) * g2.y > kMaxBlocks)
        return fail(GDN_EINVAL, "gdn_tree_accept: too many workgroups");
    return a->in_dtype == GDN_BF16 ? launch_accept<bf16_t>(P, a->n_seqs, g1, g2, s)
                                   : launch_accept<float>(P, a->n_seqs, g1, g2, s);
}
