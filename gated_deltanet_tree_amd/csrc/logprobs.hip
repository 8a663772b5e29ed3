// Log probabilities of rows of logits: given tokens, entropy and the top alternatives (gfx950).
//
// With m = max l and w_j = exp(l_j - m):  Z = sum w,  logp_j = (l_j - m) - log Z,
//   H = log Z + sum w_j (m - l_j) / Z,
// both sums of terms that are not negative.
//
// What it costs is one read of the logits.  The first launch takes them in pieces of 2048, a wave a
// piece, whose 32 values a lane stay in registers between maximum and sums; it leaves the piece's
// (m, Z, T = sum w (m - l)) and the maximum of every 64 consecutive logits.  The second, a workgroup a row,
// joins the pieces in fp64 and finds the K best logits: they lie in the K groups of 64 with the best
// maxima (every other group's best comes after those K), so of V logits only 64 K are read again.
// Sums within a piece are fp32 (a weight is off by about 2^-24 of its exponent, sums of 32 terms and 6 joins),
// all else is fp64, rounded once.
//
// 384 rows of 131072 bf16 logits, 4 alternatives: 19.6 us, 5.1 TB/s, and 6.8 for the rows; 2047 rows of 32001 fp32
// logits, 20 alternatives: 46 us, 5.7 TB/s, and 13.5; 12 rows of 32000: 3.9 and 6.4, all latency.
#include "logits.h"
#include "mfma_common.h"

namespace gdn {

struct LogprobsParams {
    const void *logits;
    const int32_t *given;
    float *given_logp, *top_logp, *entropy;
    int32_t *top_token;
    float4 *stats;  // [row][pieces]: m, Z, T
    float *group;   // [row][pieces][32]: maximum of 64 logits
    int64_t stride;
    int32_t rows, V, pieces, K, n_given;
};

namespace {

constexpr int kLogPiece = 2048, kLogThreads = 256;
constexpr int kMaxTop = 64;
constexpr int32_t kMaxTopVocab = 1 << 20;
// Keys listed at once: the K best of the threads' groups have one best each turn; the logits of K groups.
__host__ __device__ inline int list_size(int32_t pieces, int32_t K) {
    const int turns = (pieces * 32 + kLogThreads - 1) / kLogThreads;
    return K * (turns > 64 ? turns : 64);
}
// Logits ranked as they are listed; of more, those that reach a threshold.  us, 12 rows, 16 alternatives of 140 (190, 250)
// fp32 logits: 15.0 (16.2, 17.2) ranked, 14.2 (14.5, 14.3) by a threshold; from 64 on, 64 of 32000: 15.6 / 17.4.  All of
// them ranked: 64 of 1714 309, now 18; 64 of 4000 1178, now 21; 64 of 32000 equal ones 94, now 17.
constexpr int kListed = 128;
constexpr int kHeldTurns = 9;  // kept in registers between two looks: vocabularies up to 147456
constexpr float kLog2e = 1.44269504088896340736f;

__host__ __device__ inline int32_t pieces_of_row(int32_t vocab) {
    return (vocab + 7 + kLogPiece - 1) / kLogPiece;  // a row starts up to 7 logits into its first
}

template <int CTRL> __device__ __forceinline__ float lane_take(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// Largest of the wave, in all lanes; a lane's NaN is left out.
__device__ __forceinline__ float wave_largest(float x) {
    x = fmaxf(x, -kInf);
    x = fmaxf(x, lane_take<0xB1>(x));
    x = fmaxf(x, lane_take<0x4E>(x));
    x = fmaxf(x, lane_take<0x141>(x));
    x = fmaxf(x, lane_take<0x140>(x));
    const int low = __float_as_int(-kInf);
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(low, __float_as_int(x), 0x142, 0xA, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(low, __float_as_int(x), 0x143, 0xC, 0xF, false)));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

__device__ __forceinline__ uint32_t wave_largest(uint32_t x) {
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0xB1, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x4E, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x141, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), 0x140, 0xF, 0xF, true)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x142, 0xA, 0xF, false)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x143, 0xC, 0xF, false)));
    return __builtin_amdgcn_readlane(x, 63);
}

// Sums of a piece with a finite maximum.  A NaN logit has the clamped difference, and no weight.
__device__ __forceinline__ void piece_sums(const float (&x)[4][8], float m, float &z, float &t) {
    float zs[4] = {}, ts[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = fmaxf(x[k][i] - m, -1000.f);  // exp(-1000) is 0, and so is its term
            const float w = __builtin_amdgcn_exp2f(d * kLog2e);
            zs[k] += w;
            ts[k] = fmaf(w, -d, ts[k]);
        }
    z = (zs[0] + zs[1]) + (zs[2] + zs[3]);
    t = (ts[0] + ts[1]) + (ts[2] + ts[3]);
}

// Eight logits as they lie in memory.
template <typename T> struct Eight {
    uint32_t w[2 * sizeof(T)];
};
template <typename T> __device__ __forceinline__ Eight<T> load_eight(const T *p) {
    Eight<T> y;
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        y.w[4 * i] = v.x;
        y.w[4 * i + 1] = v.y;
        y.w[4 * i + 2] = v.z;
        y.w[4 * i + 3] = v.w;
    }
    return y;
}
template <typename T> __device__ __forceinline__ void widen(const Eight<T> &y, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4)
            x[i] = __uint_as_float(y.w[i]);
        else
            x[i] = (i & 1) != 0 ? bf16_hi(y.w[i / 2]) : bf16_lo(y.w[i / 2]);
    }
}

// A lane's four groups of a piece, -inf outside the row.  All loads are under way before the first is used.
template <typename T>
__device__ __forceinline__ void load_piece(const T *row, int mis, int piece, int lane, int V, float (&x)[4][8]) {
    const int start = piece * kLogPiece - mis, first = start + 8 * lane;
    Eight<T> y[4];
    if (start >= 0 && start + kLogPiece <= V) {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = load_eight(row + first + 512 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) widen(y[k], x[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = first + 512 * k;
        if (at >= 0 && at + 8 <= V) y[k] = load_eight(row + at);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = first + 512 * k;
        if (at >= 0 && at + 8 <= V) {
            widen(y[k], x[k]);
        } else {  // the row's two ends
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = at + i >= 0 && at + i < V ? to_f32<T>(row[at + i]) : -kInf;
        }
    }
}

// Order of a logit and its index, the larger logit and the smaller index first; 0: no probability.
__device__ __forceinline__ uint64_t key_of(float x, int index) {
    if (!(x > -kInf)) return 0;
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 is 0
    return uint64_t((b >> 31) != 0 ? ~b : b | 0x80000000u) << 32 | uint32_t(~index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t b = uint32_t(key >> 32);
    return __uint_as_float((b >> 31) != 0 ? b & 0x7FFFFFFFu : ~b);
}

struct Top {
    __align__(16) uint64_t first[kLogThreads];  // every thread's best
    __align__(16) uint64_t groups[kMaxTop];     // the K best, in order
    float m[kLogThreads / 64];
    double z[kLogThreads / 64], t[kLogThreads / 64];
    uint64_t threshold;
    int count[2];
};
static_assert(sizeof(Top) % 16 == 0, "the list behind it is aligned");

// How many of the first n keys of the list are larger than key; an odd one more is 0 behind them.
__device__ __forceinline__ int rank_of(uint64_t key, const uint64_t *keys, int n) {
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; i += 2) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(keys + i);
        rank += (y.x > key ? 1 : 0) + (i + 1 < n && y.y > key ? 1 : 0);
    }
    return rank;
}

// The largest threshold > 0 that at least K of the workgroup's bests reach, or 1 where fewer than K are more
// than 0.  A wave looks at all of them: the range is halved until just K lie above, 80 ns a time.  bf16
// values differ in the upper half of their keys' only.
template <typename T> __device__ __forceinline__ uint64_t kth_of(const uint64_t *first, int K) {
    constexpr int N = kLogThreads / 64, SHIFT = sizeof(T) == 2 ? 16 : 0;
    const int lane = threadIdx.x & 63;
    uint64_t key[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(first + 2 * lane + 64 * i);
        key[i] = y.x;
        key[i + 1] = y.y;
    }
    auto search = [&](const uint32_t (&x)[N], uint32_t &lo, uint32_t hi) {  // whether just K reach lo
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int c = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) c += __popcll(__ballot(x[i] >= mid));
            if (c >= K) lo = mid;
            if (c == K) return true;
            if (c < K) hi = mid - 1;
        }
        return false;
    };
    // by value first, between the smallest and the largest
    uint32_t x[N], lo = ~0u, hi = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = uint32_t(key[i] >> 32) >> SHIFT;
        lo = min(lo, x[i]);
        hi = max(hi, x[i]);
    }
    lo = ~wave_largest(~lo);
    hi = wave_largest(hi);
    if (search(x, lo, hi)) return uint64_t(lo) << (32 + SHIFT);
    if (lo == 0) return 1;
    // equal ones go by their index
    uint32_t from = ~0u, to = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t index = uint32_t(key[i]);
        if (x[i] == lo) {
            from = min(from, index);
            to = max(to, index);
        }
        x[i] = x[i] > lo ? ~0u : x[i] == lo ? index : 0;
    }
    from = ~wave_largest(~from);
    search(x, from, wave_largest(to));
    const uint32_t below = SHIFT != 0 && lo < 0x8000u ? 0xFFFFu : 0;  // of a negative value's key
    return uint64_t(lo << SHIFT | below) << 32 | from;
}

// Adds a key to the list in any order: it is ranked there.
__device__ __forceinline__ void add(uint64_t *list, int &count, uint64_t key) { list[atomicAdd(&count, 1)] = key; }

}  // namespace

template <typename T>
__global__ __launch_bounds__(kLogThreads) void logprobs_pieces_kernel(LogprobsParams P) {
    const uint32_t per_row = uint32_t(P.pieces + 3) / 4;
    const int row = int(blockIdx.x / per_row);
    const int piece = int(blockIdx.x - uint32_t(row) * per_row) * 4 + int(threadIdx.x >> 6);
    if (piece >= P.pieces) return;
    const int lane = threadIdx.x & 63;
    const T *logits = static_cast<const T *>(P.logits) + int64_t(row) * P.stride;
    const int mis = misaligned(logits);
    float x[4][8];
    load_piece(logits, mis, piece, lane, P.V, x);
    float part[4], m = -kInf;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        part[k] = x[k][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) part[k] = fmaxf(part[k], x[k][i]);
        m = fmaxf(m, part[k]);
    }
    m = wave_largest(m);
    float z = 0.f, t = 0.f;
    if (fabsf(m) < kInf) {
        piece_sums(x, m, z, t);
    } else if (m > 0.f) {  // +inf logits share the weight
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) z += x[k][i] == m ? 1.f : 0.f;
    }
    z = wave_total(z);
    t = wave_total(t);
    const int64_t at = int64_t(row) * P.pieces + piece;
    if (lane == 0) P.stats[at] = make_float4(m, z, t, 0.f);
    if (P.K > 0) {
        // 8 lanes hold 64 consecutive logits of each of the four runs
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            part[k] = fmaxf(part[k], lane_take<0xB1>(part[k]));
            part[k] = fmaxf(part[k], lane_take<0x4E>(part[k]));
            part[k] = fmaxf(part[k], lane_take<0x141>(part[k]));
        }
        const int k = lane & 7;
        if (k < 4) P.group[at * 32 + 8 * k + (lane >> 3)] = k == 0 ? part[0] : k == 1 ? part[1] : k == 2 ? part[2] : part[3];
    }
}

template <typename T>
__global__ __launch_bounds__(kLogThreads, 8) void logprobs_rows_kernel(LogprobsParams P) {
    extern __shared__ __align__(16) char mem[];
    Top &s = *reinterpret_cast<Top *>(mem);
    uint64_t *list = reinterpret_cast<uint64_t *>(mem + sizeof(Top));
    constexpr int WAVES = kLogThreads / 64;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const T *logits = static_cast<const T *>(P.logits) + int64_t(row) * P.stride;
    const int mis = misaligned(logits);
    // The pieces' sums, the groups' maxima and the first given token are under way together.
    const float4 *st = P.stats + int64_t(row) * P.pieces;
    const float4 own = tid < P.pieces ? st[tid] : make_float4(-kInf, 0.f, 0.f, 0.f);
    const float *group = P.group + int64_t(row) * P.pieces * 32;
    const int groups = P.pieces * 32;
    float held[kHeldTurns];
    uint64_t best = 0;
    if (P.K > 0) {
#pragma unroll
        for (int k = 0; k < kHeldTurns; ++k) {
            const int i = tid + k * kLogThreads;
            held[k] = i < groups ? group[i] : -kInf;
        }
    }
    float given = -kInf;
    if (tid < P.n_given) {
        const int token = P.given[int64_t(row) * P.n_given + tid];
        if (token >= 0 && token < P.V) given = logit(logits[token]);
    }
    float m = own.x;
    for (int p = tid + kLogThreads; p < P.pieces; p += kLogThreads) m = fmaxf(m, st[p].x);
    m = wave_largest(m);
    if (lane == 0) s.m[wave] = m;
    if (P.K > 0) {
#pragma unroll
        for (int k = 0; k < kHeldTurns; ++k) best = max(best, key_of(held[k], tid + k * kLogThreads));
        for (int i = tid + kHeldTurns * kLogThreads; i < groups; i += kLogThreads) best = max(best, key_of(group[i], i));
        s.first[tid] = best;
        if (tid < 2) s.count[tid] = 0;
    }
    __syncthreads();
    m = s.m[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) m = fmaxf(m, s.m[w]);
    double z = 0.0, t = 0.0;
    auto join = [&](const float4 &y) {
        if (y.x == m) {
            z += double(y.y);
            t += double(y.z);
        } else if (y.x > -kInf && m < kInf) {
            const double away = double(m) - double(y.x), f = exp(-away);
            z += f * double(y.y);
            t += f * (double(y.z) + away * double(y.y));
        }
    };
    if (wave * 64 < P.pieces) {
        join(own);
        for (int p = tid + kLogThreads; p < P.pieces; p += kLogThreads) join(st[p]);
        z = wave_sum(z);
        t = wave_sum(t);
    }
    if (lane == 0) {
        s.z[wave] = z;
        s.t[wave] = t;
    }
    if (P.K > 0) {
        // the last wave, which has fewest pieces to join; on all four it took as much of the vector unit as the rest
        if (wave == WAVES - 1) {
            const uint64_t kth = kth_of<T>(s.first, P.K);
            if (lane == 0) s.threshold = kth;
        }
        __syncthreads();
        const uint64_t threshold = s.threshold;
        if (best >= threshold) {
#pragma unroll
            for (int k = 0; k < kHeldTurns; ++k) {
                const uint64_t key = key_of(held[k], tid + k * kLogThreads);
                if (key >= threshold) add(list, s.count[0], key);
            }
            for (int i = tid + kHeldTurns * kLogThreads; i < groups; i += kLogThreads) {
                const uint64_t key = key_of(group[i], i);
                if (key >= threshold) add(list, s.count[0], key);
            }
        }
    }
    __syncthreads();
    z = s.z[0];
    t = s.t[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        z += s.z[w];
        t += s.t[w];
    }
    const double logz = m > -kInf ? log(z) : 0.0;
    auto logp = [&](float x) {
        if (!(x > -kInf)) return -kInf;
        return x == m ? float(-logz) : float((double(x) - double(m)) - logz);
    };
    if (tid == 0 && P.entropy != nullptr) P.entropy[row] = m > -kInf ? float(logz + t / z) : 0.f;
    for (int i = tid; i < P.n_given; i += kLogThreads) {
        const int64_t at = int64_t(row) * P.n_given + i;
        if (i >= kLogThreads) {
            const int token = P.given[at];
            given = token >= 0 && token < P.V ? logit(logits[token]) : -kInf;
        }
        P.given_logp[at] = logp(given);
    }
    if (P.K == 0) return;
    // ---- the K best groups in order ----------------------------------------------------------
    int n = s.count[0];
    for (int i = tid; i < n; i += kLogThreads) {
        const int rank = rank_of(list[i], list, n);
        if (rank < P.K) s.groups[rank] = list[i];
    }
    const int found = min(n, P.K);
    __syncthreads();
    // ---- their logits; no better one is below the last group's best ----------------------------
    const uint64_t least = found == P.K ? s.groups[P.K - 1] >> 32 << 32 : 1;
    constexpr int AHEAD = 6;  // loads under way together
    for (int i0 = wave; i0 < found; i0 += AHEAD * WAVES) {
        float x[AHEAD];
        int at[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k * WAVES;
            at[k] = i < found ? 64 * int(~uint32_t(s.groups[i])) + lane - mis : -1;
            x[k] = at[k] >= 0 && at[k] < P.V ? to_f32<T>(logits[at[k]]) : -kInf;
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const uint64_t key = key_of(x[k], at[k]);
            if (key >= least) add(list, s.count[1], key);
        }
    }
    __syncthreads();
    n = s.count[1];
    // Fewer groups than alternatives, or many equal logits, list thousands: those that reach the K-th of the threads' bests
    // move to the front.  They are K threads' keys, 1024 of 4096 at most the first time and 256 the second.
    for (int limit = kListed, c = 0; n > limit; limit = kLogThreads, c ^= 1) {
        best = 0;
        for (int i = tid; i < n; i += kLogThreads) best = max(best, list[i]);
        s.first[tid] = best;
        if (tid == 0) s.count[c] = 0;
        __syncthreads();
        const uint64_t threshold = kth_of<T>(s.first, P.K);  // by every wave: a case too rare for a barrier more
        for (int i0 = 0; i0 < n; i0 += kLogThreads) {
            const uint64_t key = i0 + tid < n ? list[i0 + tid] : 0;
            __syncthreads();  // these 256 have been read; no more than that many are written so far
            if (key >= threshold) add(list, s.count[c], key);
        }
        __syncthreads();
        n = s.count[c];
    }
    for (int i = tid; i < n; i += kLogThreads) {
        const uint64_t key = list[i];
        const int rank = rank_of(key, list, n);
        if (rank < P.K) {
            const float x = logp(value_of(key));  // -inf next to +inf logits, which have all the weight
            P.top_token[int64_t(row) * P.K + rank] = x > -kInf ? int(~uint32_t(key)) : -1;
            P.top_logp[int64_t(row) * P.K + rank] = x;
        }
    }
    for (int i = n + tid; i < P.K; i += kLogThreads) {  // fewer tokens with a probability than K
        P.top_token[int64_t(row) * P.K + i] = -1;
        P.top_logp[int64_t(row) * P.K + i] = -kInf;
    }
}

namespace {

int64_t logprobs_bytes(int64_t rows, int32_t vocab, int32_t top_k) {
    const int64_t pieces = pieces_of_row(vocab);
    return rows * pieces * (int64_t(sizeof(float4)) + (top_k > 0 ? 32 * int64_t(sizeof(float)) : 0));
}

// Workgroups of the first launch, a wave a piece.
int64_t logprobs_blocks(int64_t rows, int32_t vocab) { return rows * ((pieces_of_row(vocab) + 3) / 4); }

gdn_status check_logprobs_sizes(int32_t n_rows, int32_t vocab, int32_t top_k, const char *who) {
    if (n_rows < 0) return fail(GDN_EINVAL, "%s: n_rows %d", who, n_rows);
    if (vocab < 1 || vocab > (1 << 30)) return fail(GDN_EINVAL, "%s: vocab %d", who, vocab);
    if (top_k < 0 || top_k > kMaxTop || (top_k > 0 && vocab > kMaxTopVocab))
        return fail(GDN_EINVAL, "%s: top_k %d of vocab %d, at most %d of %d", who, top_k, vocab, kMaxTop, kMaxTopVocab);
    if (logprobs_blocks(n_rows, vocab) > kMaxBlocks) return fail(GDN_EINVAL, "%s: too many workgroups", who);
    return GDN_OK;
}

template <typename T> gdn_status launch_logprobs(const LogprobsParams &P, uint32_t blocks, hipStream_t s) {
    hipLaunchKernelGGL((logprobs_pieces_kernel<T>), dim3(blocks), dim3(kLogThreads), 0, s, P);
    GDN_LAUNCH_CHECK("logprobs_pieces_kernel");
    const size_t lds = sizeof(Top) + size_t(list_size(P.pieces, P.K)) * sizeof(uint64_t);
    hipLaunchKernelGGL((logprobs_rows_kernel<T>), dim3(uint32_t(P.rows)), dim3(kLogThreads), lds, s, P);
    GDN_LAUNCH_CHECK("logprobs_rows_kernel");
    return GDN_OK;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_logprobs_workspace_bytes(int32_t n_rows, int32_t vocab, int32_t top_k) {
    clear_error();
    if (check_logprobs_sizes(n_rows, vocab, top_k, "gdn_logprobs_workspace_bytes") != GDN_OK) return 0;
    return size_t(logprobs_bytes(n_rows, vocab, top_k));
}

extern "C" gdn_status gdn_token_logprobs(const gdn_logprobs_args *a, void *stream) {
    clear_error();
    const char *who = "gdn_token_logprobs";
    if (a == nullptr) return fail(GDN_EINVAL, "%s: null arguments", who);
    if (a->in_dtype != GDN_F32 && a->in_dtype != GDN_BF16) return fail(GDN_EINVAL, "%s: in_dtype %d", who, a->in_dtype);
    const gdn_status st = check_logprobs_sizes(a->n_rows, a->vocab, a->top_k, who);
    if (st != GDN_OK) return st;
    if (a->n_given < 0) return fail(GDN_EINVAL, "%s: n_given %d", who, a->n_given);
    if (a->logit_stride < a->vocab)
        return fail(GDN_EINVAL, "%s: logit_stride %lld of vocab %d", who, static_cast<long long>(a->logit_stride),
                    a->vocab);
    if (a->n_rows == 0) return GDN_OK;
    const bool top = a->top_k > 0, given = a->n_given > 0;
    if (!a->logits || !a->workspace || (top && (!a->top_token || !a->top_logp)) ||
        (given && (!a->given || !a->given_logp)))
        return fail(GDN_EINVAL, "%s: null device pointer", who);
    if (reinterpret_cast<uintptr_t>(a->logits) % (a->in_dtype == GDN_BF16 ? 2 : 4) != 0 ||
        reinterpret_cast<uintptr_t>(a->workspace) % 16 != 0)
        return fail(GDN_EINVAL, "%s: misaligned logits or workspace", who);
    const int64_t need = logprobs_bytes(a->n_rows, a->vocab, a->top_k);
    if (a->workspace_bytes < need)
        return fail(GDN_ECAPACITY, "%s: workspace holds %lld bytes, the call needs %lld", who,
                    static_cast<long long>(a->workspace_bytes), static_cast<long long>(need));
    LogprobsParams P{};
    P.logits = a->logits;
    P.given = a->given;
    P.given_logp = a->given_logp;
    P.top_logp = a->top_logp;
    P.top_token = a->top_token;
    P.entropy = a->entropy;
    P.stride = a->logit_stride;
    P.rows = a->n_rows;
    P.V = a->vocab;
    P.pieces = pieces_of_row(a->vocab);
    P.K = a->top_k;
    P.n_given = a->n_given;
    P.stats = static_cast<float4 *>(a->workspace);
    P.group = reinterpret_cast<float *>(P.stats + int64_t(a->n_rows) * P.pieces);
    const int64_t blocks = logprobs_blocks(a->n_rows, a->vocab);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return a->in_dtype == GDN_BF16 ? launch_logprobs<bf16_t>(P, uint32_t(blocks), s)
                                   : launch_logprobs<float>(P, uint32_t(blocks), s);
}
