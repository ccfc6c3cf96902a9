// One step of beam search over logits [B, K, V]: the M best continuations of
// each batch entry's K beams by score + log-softmax, and the reordering of
// the beams' states. Two kernels for the selection, one for the reordering.
//
// Selection. With lse_k = log sum_v exp(x_kv), candidate (k, v) has the score
// s_k + x_kv - lse_k, so within a beam the order is that of the logits:
//  1. beam_scan reads every logit once. A row is split over CTAs and their
//     warps; a warp keeps the running maximum and sum of the softmax a lane,
//     and its M best logits in a sorted list over its lanes. A logit above
//     the list's last goes to a buffer in shared memory; 32 of them are
//     sorted and merged into the list by a bitonic network. A CTA joins its
//     warps' lists and sums and writes M candidates and {max, sum}.
//  2. beam_pick, a CTA a batch entry, forms the K log-sum-exps from the
//     {max, sum} in a fixed order, takes the M-th best of the lists' first
//     candidates as a bound (no list that starts below it can contribute),
//     and ranks the candidates above it by counting.
// Candidates are ordered by (score in 64 bits, then lowest k V + v), so ties
// and the order in which warps finish do not show in the result.
//
// Bound by HBM: one read of the logits.
#include <algorithm>
#include <cstdint>
#include <string>

#include "ce_kernels.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);
void record_message(const std::string& msg);

namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanVec = 4;     // 16-byte vectors a lane holds at a time
constexpr int kPickThreads = 256;
constexpr int kMaxBeams = 32;
constexpr int kMaxCandidates = 64;
constexpr int kMaxSplits = 64;  // CTAs a row
constexpr float kLowest = -3.402823466e38f;

// A candidate inside a row: the logit as an ordered integer above the
// complement of the token, so that a larger word is a better candidate (a
// larger logit, then a smaller token); 0 is none.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint64_t candidate(float x, int token) {
    return (static_cast<uint64_t>(ordered(x)) << 32) | static_cast<uint32_t>(~token);
}

struct RowSum {  // of one split of a row
    float m;     // running maximum (kLowest with no token)
    float s;     // sum of exp(x - m)
};

struct BeamArgs {
    const void* logits;       // [B, K, V]
    const float* scores;      // [B, K]
    const uint8_t* finished;  // [B, K] or nullptr
    int64_t rows;             // B K
    int64_t V;
    int K, M, splits;
    int64_t pad;
    RowSum* sums;        // [rows, splits]
    uint64_t* lists;     // [rows, splits, M]
    float* out_scores;   // [B, M]
    int64_t* out_beams;
    int64_t* out_tokens;
};

// Whether beam `row` has candidates of its own (a finite score, not finished).
__device__ __forceinline__ bool beam_lives(const BeamArgs& a, int64_t row) {
    const float s = a.scores[row];
    return isfinite(s) && !(a.finished && a.finished[row]);
}

// Sorts a word a lane in descending order over the warp.
__device__ __forceinline__ uint64_t warp_sort_desc(uint64_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const uint64_t o = __shfl_xor_sync(~0u, v, d);
            const bool up = (lane & d) == 0;
            const bool desc = (lane & size) == 0 || size == 32;
            v = ((v > o) == (up == desc)) ? v : o;
        }
    }
    return v;
}

// The M best logits a warp has seen: E words a lane, position 32 e + lane in
// descending order, and a buffer of up to 63 not yet merged.
template <int E>
struct WarpBest {
    uint64_t best[E];
    uint64_t* buf;  // 64 words of shared memory of this warp
    int count;
    uint64_t last;  // a candidate must lie above this to matter,
    float bar;      // and this is its logit
    int lane, M;

    __device__ __forceinline__ void init(uint64_t* b, int l, int m) {
#pragma unroll
        for (int e = 0; e < E; ++e) best[e] = 0;
        buf = b;
        count = 0;
        bar = -INFINITY;
        last = candidate(bar, 0);  // -inf is never a candidate
        lane = l;
        M = m;
    }

    // Merges up to 32 buffered words (0 on the lanes behind the last).
    __device__ __forceinline__ void merge(uint64_t in) {
        in = warp_sort_desc(in, lane);
        // the best 32 E of the list and the sorted words: the larger of the
        // list and the reversed words is a bitonic sequence that holds them
        const uint64_t r = __shfl_xor_sync(~0u, in, 31);
        best[E - 1] = best[E - 1] > r ? best[E - 1] : r;
        if constexpr (E == 2) {
            const uint64_t hi = best[0] > best[1] ? best[0] : best[1];
            const uint64_t lo = best[0] > best[1] ? best[1] : best[0];
            best[0] = hi;
            best[1] = lo;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const uint64_t o = __shfl_xor_sync(~0u, best[e], d);
                best[e] = ((best[e] > o) == ((lane & d) == 0)) ? best[e] : o;
            }
        }
        const uint64_t w = __shfl_sync(~0u, best[E - 1], (M - 1) & 31);  // position M - 1
        if (w) {
            last = w;
            bar = unordered(static_cast<uint32_t>(w >> 32));
        }
    }

    // Offers one logit a lane (NaN and -inf never pass).
    __device__ __forceinline__ void offer(float x, int token) {
        // logits of one block of vectors come out of the tokens' order, so an
        // equal logit counts when its token is the lower
        const uint64_t w = candidate(x, token);
        const bool in = x >= bar && w > last;
        const unsigned who = __ballot_sync(~0u, in);
        if (!who) return;
        if (in) buf[count + __popc(who & ((1u << lane) - 1u))] = w;
        count += __popc(who);
        __syncwarp();
        if (count >= 32) {
            merge(buf[lane]);
            const uint64_t rest = buf[32 + lane];
            __syncwarp();
            buf[lane] = rest;
            count -= 32;
            __syncwarp();
        }
    }

    __device__ __forceinline__ void finish() {
        __syncwarp();
        if (count) merge(lane < count ? buf[lane] : 0);
        count = 0;
    }
};

// Vector j of a row whose first element lies `lead` elements before the
// row's start (so that vectors are 16-byte aligned): whole vectors in one
// load, the row's ends element by element with -inf outside the row.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int64_t V, int lead, int64_t j, float* f) {
    constexpr int N = Vec<T>::N;
    const int64_t e = j * N - lead;
    if (e >= 0 && e + N <= V) {
        float t[N];
        Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(row + e)), t);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = t[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = (e + i >= 0 && e + i < V) ? Vec<T>::load1(row, e + i) : -INFINITY;
    }
}

template <typename T, int E>
__global__ void __launch_bounds__(kScanThreads) beam_scan(const __grid_constant__ BeamArgs a) {
    constexpr int N = Vec<T>::N;
    __shared__ uint64_t buf[kScanWarps][64];
    __shared__ uint64_t lists[kScanWarps * kMaxCandidates];
    __shared__ RowSum sums[kScanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x % a.splits);
    pdl_launch_dependents();
    if (!beam_lives(a, r)) return;
    const T* row = static_cast<const T*>(a.logits) + r * a.V;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int64_t nv = (a.V + lead + N - 1) / N;
    const int64_t per = (nv + a.splits * kScanWarps - 1) / (a.splits * kScanWarps);
    const int64_t j0 = (static_cast<int64_t>(split) * kScanWarps + warp) * per;
    const int64_t j1 = j0 + per < nv ? j0 + per : nv;

    WarpBest<E> top;
    top.init(buf[warp], lane, a.M);
    float m = kLowest, s = 0.f;
    for (int64_t j = j0; j < j1; j += 32 * kScanVec) {
        float f[kScanVec][N];
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) {
            const int64_t jk = j + 32 * k + lane;
            if (jk < j1) {
                load_vec<T>(row, a.V, lead, jk, f[k]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[k][i] = -INFINITY;
            }
        }
        float vm[kScanVec], bm = m;
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) {
            vm[k] = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[k][i] = fmaxf(f[k][i], -INFINITY);  // NaN counts as masked
                vm[k] = fmaxf(vm[k], f[k][i]);
            }
            bm = fmaxf(bm, vm[k]);
        }
        s *= ex2((m - bm) * kLog2e);
        m = bm;
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) {
#pragma unroll
            for (int i = 0; i < N; ++i) s += ex2((f[k][i] - m) * kLog2e);
        }
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) {
            // tokens of later blocks are larger: an equal logit does not matter
            if (!__any_sync(~0u, vm[k] > top.bar)) continue;
            const int t0 = static_cast<int>((j + 32 * k + lane) * N) - lead;
#pragma unroll
            for (int i = 0; i < N; ++i) top.offer(f[k][i], t0 + i);
        }
    }
    top.finish();

    // the warp's sum, then the CTA's list and sum
    float wm = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wm = fmaxf(wm, __shfl_xor_sync(~0u, wm, d));
    float ws = s * ex2((m - wm) * kLog2e);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ws += __shfl_xor_sync(~0u, ws, d);
    if (lane == 0) sums[warp] = RowSum{wm, ws};
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (32 * e + lane < a.M) lists[warp * a.M + 32 * e + lane] = top.best[e];
    __syncthreads();
    const int64_t slot = r * a.splits + split;
    if (threadIdx.x == 0) {
        RowSum t = sums[0];
        for (int w = 1; w < kScanWarps; ++w) t.m = fmaxf(t.m, sums[w].m);
        t.s = 0.f;
        for (int w = 0; w < kScanWarps; ++w) t.s += sums[w].s * ex2((sums[w].m - t.m) * kLog2e);
        a.sums[slot] = t;
    }
    uint64_t* out = a.lists + slot * a.M;
    const int n = kScanWarps * a.M;
    int filled = 0;  // candidates of all warps
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
        const uint64_t w = lists[i];
        int rank = 0;
        filled = 0;
        for (int o = 0; o < n; ++o) {
            rank += lists[o] > w;
            filled += lists[o] != 0;
        }
        if (w && rank < a.M) out[rank] = w;
    }
    // no candidate in the places behind the last
    if (threadIdx.x < a.M) {
        if (static_cast<int>(threadIdx.x) >= filled) out[threadIdx.x] = 0;
    }
}

// A candidate of a batch entry: its score in 64 bits as an ordered integer
// (0: none), then its place k V + v.
struct Pick {
    uint64_t key;
    int64_t at;
};
__device__ __forceinline__ bool better(const Pick& p, const Pick& q) {
    return p.key > q.key || (p.key == q.key && p.at < q.at);
}
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return (b >> 63) ? ~b : b | (uint64_t{1} << 63);
}
__device__ __forceinline__ double unordered64(uint64_t u) {
    return __longlong_as_double(
        static_cast<long long>((u >> 63) ? u & ~(uint64_t{1} << 63) : ~u));
}

// A row's log-sum-exp, m + logs: its parts are subtracted one after the
// other, since m may be of a size at which their sum loses logs.
struct RowLse {
    double m, logs;
};

// Candidate i of list `l` (beam l / splits) of batch entry b.
__device__ __forceinline__ Pick list_pick(const BeamArgs& a, int64_t b, int l, int i,
                                          const RowLse* lse, const uint8_t* kind) {
    const int k = l / a.splits;
    if (kind[k] != 1) {
        // a finished beam goes on with the padding token alone
        if (kind[k] == 2 && i == 0 && l % a.splits == 0)
            return Pick{ordered64(static_cast<double>(a.scores[b * a.K + k])), k * a.V + a.pad};
        return Pick{0, INT64_MAX};
    }
    const uint64_t w = a.lists[((b * a.K + k) * a.splits + l % a.splits) * a.M + i];
    if (!w) return Pick{0, INT64_MAX};
    const double x = static_cast<double>(unordered(static_cast<uint32_t>(w >> 32)));
    const int token = static_cast<int>(~static_cast<uint32_t>(w));
    return Pick{ordered64(((x - lse[k].m) - lse[k].logs) +
                          static_cast<double>(a.scores[b * a.K + k])),
                k * a.V + token};
}

__global__ void __launch_bounds__(kPickThreads) beam_pick(const __grid_constant__ BeamArgs a) {
    extern __shared__ Pick pick_smem[];
    __shared__ RowLse lse[kMaxBeams];
    __shared__ uint8_t kind[kMaxBeams];  // 0 dead, 1 alive, 2 finished
    __shared__ Pick bound;
    __shared__ int nsurv;
    Pick* heads = pick_smem;                    // [K splits]
    const int nl = a.K * a.splits;
    Pick* surv = pick_smem + nl;                // [M M]
    const int64_t b = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        bound = Pick{0, INT64_MAX};
        nsurv = 0;
    }
    pdl_wait();
    for (int k = warp; k < a.K; k += kPickThreads / 32) {
        const int64_t row = b * a.K + k;
        const bool live = beam_lives(a, row);
        if (live) {
            float m = kLowest;
            for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, a.sums[row * a.splits + i].m);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
            double s = 0.0;
            for (int i = lane; i < a.splits; i += 32) {
                const RowSum t = a.sums[row * a.splits + i];
                s += static_cast<double>(t.s * exp2f((t.m - m) * kLog2e));
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
            if (lane == 0) {
                // log s from its binary exponent and a mantissa near 1: logf there
                // is off by 2^-25 or less, the mantissa's rounding is put back
                int e = 0;
                const double f = frexp(s, &e) * 1.4142135623730951;  // [0.7, 1.42)
                const float f32 = static_cast<float>(f);
                lse[k].m = static_cast<double>(m);
                lse[k].logs = (e - 0.5) * 0.6931471805599453 +
                              static_cast<double>(logf(f32) + static_cast<float>(f - f32) / f32);
                kind[k] = isfinite(m) && s > 0.0 && isfinite(s) ? 1 : 0;
            }
        } else if (lane == 0) {
            kind[k] = isfinite(a.scores[row]) ? 2 : 0;
        }
    }
    __syncthreads();
    for (int l = threadIdx.x; l < nl; l += kPickThreads) heads[l] = list_pick(a, b, l, 0, lse, kind);
    __syncthreads();
    // the M-th best of the lists' first candidates
    for (int l = threadIdx.x; l < nl; l += kPickThreads) {
        const Pick p = heads[l];
        if (!p.key) continue;
        int rank = 0;
        for (int o = 0; o < nl; ++o) rank += better(heads[o], p);
        if (rank == a.M - 1) bound = p;
    }
    __syncthreads();
    const Pick bar = bound;
    // every candidate that is not below it: M lists at most start above it
    for (int l = threadIdx.x; l < nl; l += kPickThreads) {
        Pick p = heads[l];
        for (int i = 0; p.key && !better(bar, p);) {
            surv[atomicAdd(&nsurv, 1)] = p;
            if (++i == a.M) break;
            p = list_pick(a, b, l, i, lse, kind);
        }
    }
    __syncthreads();
    const int n = nsurv;
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
        const Pick p = surv[i];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += better(surv[o], p);
        if (rank < a.M) {
            a.out_scores[b * a.M + rank] = static_cast<float>(unordered64(p.key));
            a.out_beams[b * a.M + rank] = p.at / a.V;
            a.out_tokens[b * a.M + rank] = p.at % a.V;
        }
    }
    for (int i = n + threadIdx.x; i < a.M; i += kPickThreads) {
        a.out_scores[b * a.M + i] = -INFINITY;
        a.out_beams[b * a.M + i] = -1;
        a.out_tokens[b * a.M + i] = a.pad;
    }
}

// ---------------------------------------------------------------- states

constexpr int kReorderThreads = 256;
constexpr int kReorderTensors = 16;  // of one launch

// A state: rows [B K] of `outer` blocks of `inner` bytes each, at strides.
struct ReorderTensor {
    const char* src;
    char* dst;
    int64_t src_row, src_outer, dst_row, dst_outer;  // strides in bytes
    int64_t outer, inner;                            // blocks a row, bytes a block
    int vec;                                         // bytes a thread moves: 16, 8, 4, 2 or 1
};
struct ReorderArgs {
    ReorderTensor t[kReorderTensors];
    const int64_t* beams;  // [B, K]
    int64_t B;
    int K, inplace;
};

// A thread owns one column of `vec` bytes of all K rows: it reads the rows
// that the new order takes from elsewhere, then writes them, so that the
// order may be changed in place. K registers a thread are in flight.
template <typename U, int KMAX>
__device__ __forceinline__ void reorder_columns(const ReorderArgs& a, const ReorderTensor& t,
                                                const int* from, int64_t b, int64_t first,
                                                int64_t step) {
    const int64_t per = t.inner / static_cast<int64_t>(sizeof(U));
    const int64_t cols = t.outer * per;
    for (int64_t c = first; c < cols; c += step) {
        const int64_t o = c / per, i = (c - o * per) * static_cast<int64_t>(sizeof(U));
        const char* src = t.src + b * a.K * t.src_row + o * t.src_outer + i;
        char* dst = t.dst + b * a.K * t.dst_row + o * t.dst_outer + i;
        U v[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (k < a.K && from[k] >= 0)
                v[k] = *reinterpret_cast<const U*>(src + from[k] * t.src_row);
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
            if (k < a.K && from[k] >= 0) *reinterpret_cast<U*>(dst + k * t.dst_row) = v[k];
    }
}

template <int KMAX>
__global__ void __launch_bounds__(kReorderThreads) beam_reorder(const __grid_constant__ ReorderArgs a) {
    __shared__ int from[KMAX];  // the row that row k takes, -1: stays untouched
    const ReorderTensor& t = a.t[blockIdx.z];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kReorderThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kReorderThreads;
    pdl_wait();
    for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
        __syncthreads();
        if (threadIdx.x < KMAX) {
            const int k = threadIdx.x;
            int f = -1;
            if (k < a.K) {
                const int64_t s = a.beams[b * a.K + k];
                f = (s >= 0 && s < a.K) ? static_cast<int>(s) : k;  // anything else: stays
                if (f == k && a.inplace) f = -1;
            }
            from[k] = f;
        }
        __syncthreads();
        switch (t.vec) {
        case 16: reorder_columns<uint4, KMAX>(a, t, from, b, first, step); break;
        case 8: reorder_columns<uint2, KMAX>(a, t, from, b, first, step); break;
        case 4: reorder_columns<uint32_t, KMAX>(a, t, from, b, first, step); break;
        case 2: reorder_columns<uint16_t, KMAX>(a, t, from, b, first, step); break;
        default: reorder_columns<uint8_t, KMAX>(a, t, from, b, first, step); break;
        }
    }
}

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

ce_status sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "beam search device");
}

// CTAs a row: enough to fill the GPU four CTAs an SM deep, at least 8 KB of
// logits each.
int scan_splits(int64_t rows, int64_t row_bytes, int sms) {
    const int64_t fill = (4L * std::max(sms, 1) + rows - 1) / std::max<int64_t>(rows, 1);
    const int64_t room = std::max<int64_t>(1, row_bytes / 8192);
    return static_cast<int>(std::max<int64_t>(1, std::min({fill, room, int64_t{kMaxSplits}})));
}

template <int E>
const void* scan_fn(int dtype) {
    return dtype == CE_F32    ? (const void*)&beam_scan<float, E>
           : dtype == CE_BF16 ? (const void*)&beam_scan<__nv_bfloat16, E>
                              : (const void*)&beam_scan<__half, E>;
}

ce_status check_beam(int dtype, int64_t B, int64_t K, int64_t V, int64_t M) {
    if (dtype != CE_F32 && dtype != CE_BF16 && dtype != CE_F16) return CE_ERR_INVALID_ARG;
    if (B < 0 || K < 1 || V < 1 || M < 1) return CE_ERR_INVALID_ARG;
    if (K > kMaxBeams || M > kMaxCandidates || V > INT32_MAX - 64 || B > INT32_MAX / (kMaxBeams * kMaxSplits)) {
        record_message("beam search takes at most 32 beams, 64 candidates, 2^20 batch entries "
                       "and a vocabulary below 2^31 - 64");
        return CE_ERR_UNSUPPORTED;
    }
    return CE_OK;
}

ce_status launch_pdl(const void* fn, dim3 grid, int threads, size_t smem, cudaStream_t st, void* arg,
                     const char* what) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    void* args[] = {arg};
    const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, what);
}

}  // namespace
}  // namespace gbce

using namespace gbce;

extern "C" size_t ce_beam_workspace_bytes(int dtype, int64_t B, int64_t K, int64_t V, int64_t M) {
    if (check_beam(dtype, B, K, V, M) != CE_OK) return 0;
    // for the most CTAs a row that any device gets
    const int64_t row_bytes = V * (dtype == CE_F32 ? 4 : 2);
    const int64_t lists = B * K * std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, row_bytes / 8192));
    return static_cast<size_t>(up256(lists * static_cast<int64_t>(sizeof(RowSum))) +
                               up256(lists * M * 8) + 256);
}

extern "C" ce_status ce_beam_select(const void* logits, int dtype, int64_t B, int64_t K, int64_t V,
                                    const float* scores, const uint8_t* finished,
                                    int64_t pad_token, int64_t M, float* out_scores,
                                    int64_t* out_beams, int64_t* out_tokens, void* workspace,
                                    size_t workspace_bytes, ce_stream_t stream) {
    ce_status rc = check_beam(dtype, B, K, V, M);
    if (rc != CE_OK) return rc;
    if (pad_token < 0 || pad_token >= V) return CE_ERR_INVALID_ARG;
    if (B == 0) return CE_OK;
    if (!logits || !scores || !out_scores || !out_beams || !out_tokens) return CE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < ce_beam_workspace_bytes(dtype, B, K, V, M))
        return CE_ERR_INVALID_ARG;
    const int64_t b = dtype == CE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % static_cast<uintptr_t>(b)) return CE_ERR_INVALID_ARG;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != CE_OK) return rc;
    BeamArgs a = {};
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.rows = B * K;
    a.V = V;
    a.K = static_cast<int>(K);
    a.M = static_cast<int>(M);
    a.splits = scan_splits(a.rows, V * b, sms);
    a.pad = pad_token;
    a.sums = static_cast<RowSum*>(workspace);
    a.lists = reinterpret_cast<uint64_t*>(
        static_cast<char*>(workspace) + up256(a.rows * a.splits * static_cast<int64_t>(sizeof(RowSum))));
    a.out_scores = out_scores;
    a.out_beams = out_beams;
    a.out_tokens = out_tokens;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    cudaError_t e = cudaLaunchKernel(M <= 32 ? scan_fn<1>(dtype) : scan_fn<2>(dtype),
                                     dim3(static_cast<unsigned>(a.rows * a.splits)),
                                     dim3(kScanThreads), args, 0, st);
    if (e != cudaSuccess) return record_cuda_failure(e, "beam scan launch");
    const size_t smem = sizeof(Pick) * static_cast<size_t>(K * a.splits + M * M);
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute((const void*)&beam_pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(sizeof(Pick) * (kMaxBeams * kMaxSplits +
                                                                  kMaxCandidates * kMaxCandidates)));
        if (e != cudaSuccess) return record_cuda_failure(e, "beam pick attributes");
    }
    return launch_pdl((const void*)&beam_pick, dim3(static_cast<unsigned>(B)), kPickThreads, smem, st,
                      &a, "beam pick launch");
}

extern "C" ce_status ce_beam_reorder(const ce_beam_state* states, int n, const int64_t* beams,
                                     int64_t B, int64_t K, ce_stream_t stream) {
    if (n < 0 || B < 0 || K < 1) return CE_ERR_INVALID_ARG;
    if (K > kMaxBeams) {
        record_message("beam search takes at most 32 beams");
        return CE_ERR_UNSUPPORTED;
    }
    if (n == 0 || B == 0) return CE_OK;
    if (!states || !beams) return CE_ERR_INVALID_ARG;
    int inplace = -1;
    for (int i = 0; i < n; ++i) {
        const ce_beam_state& s = states[i];
        if (s.blocks < 0 || s.block_bytes < 0) return CE_ERR_INVALID_ARG;
        if (s.blocks == 0 || s.block_bytes == 0) continue;
        if (!s.src || !s.dst) return CE_ERR_INVALID_ARG;
        const int in = s.src == s.dst ? 1 : 0;
        if (in && (s.src_row != s.dst_row || s.src_block != s.dst_block)) return CE_ERR_INVALID_ARG;
        if (inplace < 0) inplace = in;
        if (inplace != in) return CE_ERR_INVALID_ARG;
    }
    int sms = 0;
    ce_status rc = sm_count(&sms);
    if (rc != CE_OK) return rc;
    const void* fn = K <= 4    ? (const void*)&beam_reorder<4>
                     : K <= 8  ? (const void*)&beam_reorder<8>
                     : K <= 16 ? (const void*)&beam_reorder<16>
                               : (const void*)&beam_reorder<32>;
    for (int i = 0; i < n;) {
        ReorderArgs a = {};
        a.beams = beams;
        a.B = B;
        a.K = static_cast<int>(K);
        a.inplace = inplace;
        int m = 0;
        int64_t cols = 1;
        for (; i < n && m < kReorderTensors; ++i) {
            const ce_beam_state& s = states[i];
            if (s.blocks == 0 || s.block_bytes == 0) continue;
            ReorderTensor& t = a.t[m++];
            t.src = static_cast<const char*>(s.src);
            t.dst = static_cast<char*>(s.dst);
            t.src_row = s.src_row;
            t.src_outer = s.src_block;
            t.dst_row = s.dst_row;
            t.dst_outer = s.dst_block;
            t.outer = s.blocks;
            t.inner = s.block_bytes;
            const uintptr_t bits = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
                                   static_cast<uintptr_t>(s.src_row | s.src_block | s.dst_row |
                                                          s.dst_block | s.block_bytes);
            t.vec = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
            cols = std::max<int64_t>(cols, t.outer * (t.inner / t.vec));
        }
        if (!m) break;
        const int64_t gy = std::min<int64_t>(B, 4096);
        // a column a thread, until the launch has 16 CTAs an SM of every tensor
        const int64_t gx = std::min<int64_t>((cols + kReorderThreads - 1) / kReorderThreads,
                                             std::max<int64_t>(1, 16L * sms * 8 / gy));
        rc = launch_pdl(fn, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy),
                                 static_cast<unsigned>(m)),
                        kReorderThreads, 0, reinterpret_cast<cudaStream_t>(stream), &a,
                        "beam reorder launch");
        if (rc != CE_OK) return rc;
    }
    return CE_OK;
}
