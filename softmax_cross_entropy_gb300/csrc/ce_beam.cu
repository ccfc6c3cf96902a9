// One step of beam search over logits [B, K, V]: the M best continuations of
// each batch entry's K beams by score + log-softmax, and the reordering of
// the beams' states. Two kernels for the selection, one for the reordering.
//
// Selection. With lse_k = log sum_v exp(x_kv), candidate (k, v) has the score
// s_k + x_kv - lse_k, so within a beam the order is that of the logits:
//  1. beam_scan reads every logit once, in parts of a row of up to 44 KB that
//     a CTA stages in shared memory (cp.async; four CTAs an SM, so that parts
//     are on their way while others are worked on) and passes over twice.
//     The first pass takes each thread's largest logit. From these come the
//     part's maximum and a bound that M logits reach: for M up to 16 the M-th
//     best of the 8 warps' 4 largest, else the smallest of the 8 warps'
//     ceil(M / 8)-th largest (a thread counts once). The second pass
//     sums exp(x - maximum) (one FFMA and one exp2 a logit) and lists the
//     logits that reach the bound, about M of them, which are ranked by
//     counting. The part's M best and {maximum, sum} go to the workspace.
//     Where more logits reach the bound than the list holds (equal ones), the
//     warps merge the part's logits into sorted lists instead, 32 at a time
//     by a bitonic network.
//  2. beam_pick, a CTA a batch entry, forms the K log-sum-exps from the
//     {max, sum} in a fixed order and the scores of the lists' candidates, and
//     merges the lists: a warp holds their first candidates and takes the best
//     M times. (Where the lists are many, the M-th best of their first
//     candidates bounds what can matter, and what reaches it is ranked by
//     counting.)
// Candidates are ordered by (score in 48 bits, then lowest k V + v), so ties
// and the order in which warps finish do not show in the result.
//
// One read of the logits. The scan fills neither the issue slots (54-60%
// taken; 32 logits take a warp 15 instructions in 16 bits, 20 in 32) nor HBM
// (36-49% of ncu's peak): a CTA has one stage, waits for a whole part, crosses
// about five barriers and asks for the next part after its second pass, which
// the three other CTAs of the SM hide in part: 64 x 8 x 131072 fp32 66 us (4.1
// TB/s), bf16 45 us (3 TB/s). The reordering is bound by HBM: 2 x 134 MB of
// states in 67 us.
#include <algorithm>
#include <cstdint>
#include <string>

#include "ce_kernels.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);
void record_message(const std::string& msg);
ce_status tc_smem_limit(const void* fn, size_t bytes);

namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanCtas = 4;        // CTAs an SM
constexpr int kScanMost = 2816;     // 16-byte vectors of a part at most (44 KB)
constexpr int kScanList = 512;      // logits of a part that may reach the bound
constexpr int kScanBuf = 64;        // words of a warp's buffer when merging
constexpr int kPickThreads = 256;
constexpr int kMaxBeams = 32;
constexpr int kMaxCandidates = 64;
constexpr int64_t kMaxVocab = 1 << 20;
constexpr int kMergeLists = 128;    // lists of an entry that a warp merges
// parts that a row needs (94, of 2^20 logits in fp32); with few rows a row
// has more, but an entry's K rows then no more than about two an SM
constexpr int kMostParts = (kMaxVocab / 4 + kScanMost - 1) / kScanMost;
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
    float m;     // maximum (-inf with no token)
    float s;     // sum of exp(x - m)
};

struct BeamArgs {
    const void* logits;       // [B, K, V]
    const float* scores;      // [B, K]
    const uint8_t* finished;  // [B, K] or nullptr
    int64_t rows;             // B K
    int64_t V;
    int K, M;
    int splits;        // parts of a row, the same of every row
    int part_vec;      // 16-byte vectors of a part
    int row_step, part_step;  // a CTA's step of gridDim parts: rows and parts
    int64_t pad;
    RowSum* sums;        // [rows, splits]
    uint64_t* lists;     // [rows, splits, M]
    float* out_scores;   // [B, M]
    int64_t* out_beams;
    int64_t* out_tokens;
};

// The most shared memory that beam_pick takes: the candidates of all lists
// that are merged, or the first candidates of all lists and M squared.
constexpr size_t kPickSmem = 16 * kMergeLists * kMaxCandidates;
static_assert(16 * (kMaxBeams * kMostParts + kMaxCandidates * kMaxCandidates) <= kPickSmem, "beam_pick");

// Whether beam `row` has candidates of its own (a finite score, not finished).
__device__ __forceinline__ bool beam_lives(const BeamArgs& a, int64_t row) {
    const float s = a.scores[row];
    return isfinite(s) && !(a.finished && a.finished[row]);
}

// Sorts a word a lane in descending order over the warp.
template <typename U>
__device__ __forceinline__ U warp_sort_desc(U v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const U o = __shfl_xor_sync(~0u, v, d);
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
    uint64_t* buf;  // kScanBuf words of shared memory of this warp
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
        if (w > last) {
            last = w;
            bar = unordered(static_cast<uint32_t>(w >> 32));
        }
    }

    // Merges whole warps of the buffer's words.
    __device__ __forceinline__ void drain() {
        while (count >= 32) {
            count -= 32;
            merge(buf[count + lane]);
        }
        __syncwarp();
    }

    // Offers one logit a lane, of tokens in any order (an equal logit counts
    // when its token is the lower; NaN and -inf never pass).
    __device__ __forceinline__ void offer(float x, int token) {
        const uint64_t w = candidate(x, token);
        const bool in = x >= bar && w > last;
        const unsigned who = __ballot_sync(~0u, in);
        if (in) buf[count + __popc(who & ((1u << lane) - 1u))] = w;
        count += __popc(who);
        __syncwarp();
        drain();
    }
};

// The pattern of -inf in every element of a vector.
template <typename T>
__device__ __forceinline__ uint32_t neg_inf_word();
template <>
__device__ __forceinline__ uint32_t neg_inf_word<float>() { return 0xFF800000u; }
template <>
__device__ __forceinline__ uint32_t neg_inf_word<__nv_bfloat16>() { return 0xFF80FF80u; }
template <>
__device__ __forceinline__ uint32_t neg_inf_word<__half>() { return 0xFC00FC00u; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// A part of a row: its 16-byte vectors [j0, j0 + len), vector j being the
// elements N j .. N j + N - 1 wherever the row starts in memory, so that equal
// rows are summed alike (and equal beams tie exactly).
template <typename T>
struct RowPart {
    static constexpr int N = Vec<T>::N;
    const T* row;
    int V, j0, len;
    int shift;  // bytes from the 16-byte boundary before the row to the row

    // Copies the part's aligned vectors (one more where the row is not
    // aligned) to shared memory; elements outside the row become -inf.
    __device__ __forceinline__ void fetch(uint4* stage) const {
        const int64_t bytes = static_cast<int64_t>(V) * sizeof(T) + shift;  // to the row's end
        const int n = len + (shift ? 1 : 0);
        const int lo = shift && j0 == 0 ? 1 : 0;  // vectors [lo, hi) lie in the row
        const int hi = min(n, static_cast<int>(bytes / 16) - j0);
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) - shift) + j0;
        uint32_t dst = smem_u32(stage + lo + threadIdx.x);
        src += lo + threadIdx.x;
#pragma unroll 4
        for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += kScanThreads) {
            cp_async16(dst, src);
            dst += 16 * kScanThreads;
            src += kScanThreads;
        }
        if (static_cast<int>(threadIdx.x) < lo) stage[threadIdx.x] = edge(j0);
        for (int i = max(hi, lo) + static_cast<int>(threadIdx.x); i < n; i += kScanThreads) stage[i] = edge(j0 + i);
    }
    // aligned vector w, of which only some elements lie in the row
    __device__ __forceinline__ uint4 edge(int w) const {
        const uint32_t none = neg_inf_word<T>();
        uint32_t v[4] = {none, none, none, none};
        const int64_t e0 = static_cast<int64_t>(w) * N - shift / static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t e = e0 + i;
            if (e < 0 || e >= V) continue;
            if constexpr (sizeof(T) == 4) {
                v[i] = reinterpret_cast<const uint32_t*>(row)[e];
            } else {
                const uint32_t h = reinterpret_cast<const uint16_t*>(row)[e];
                v[i / 2] = (i & 1) ? (v[i / 2] & 0xFFFFu) | (h << 16) : (v[i / 2] & 0xFFFF0000u) | h;
            }
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
    // vector j0 + i, from the staged aligned ones that it lies in (FLAT: of a
    // row that is aligned)
    template <bool FLAT>
    __device__ __forceinline__ uint4 get(const uint4* stage, int i) const {
        const uint4 a = stage[i];
        if constexpr (FLAT) return a;
        const uint4 b = stage[i + 1];
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = (shift & 8) ? w[k + 2] : w[k];
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = (shift & 4) ? w[k + 1] : w[k];
        const int bits = 8 * (shift & 3);
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
};

template <int E>
struct ScanShared {
    uint64_t list[kScanWarps * (32 * E + 32) > kScanList ? kScanWarps * (32 * E + 32) : kScanList];
    uint64_t buf[kScanWarps][kScanBuf];
    uint64_t lasts[kScanWarps];
    uint32_t tops[kScanWarps * 8];  // the warps' t largest threads, as ordered integers
    float sums[kScanWarps];
    uint32_t top, bound;
    int found;
};

// The first pass: this thread's largest logit of the part.
template <bool FLAT, typename T>
__device__ __forceinline__ float part_max(const RowPart<T>& part, const uint4* stage) {
    float m = -INFINITY;
#pragma unroll 4
    for (int i = threadIdx.x; i < part.len; i += kScanThreads)
        m = fmaxf(m, Vec<T>::vmax(part.template get<FLAT>(stage, i)));
    return m;
}

// log2 e m overflows from here on: such parts take part_sum.
constexpr float kHuge = 2e38f;

// The second pass: the thread's share of the sum of exp(x - m), and its
// logits from `bar` on into the list (what does not fit is counted only).
template <bool FLAT, typename T, int E>
__device__ __forceinline__ float part_scan(const RowPart<T>& part, const uint4* stage, float m,
                                           float bar, ScanShared<E>& sh) {
    constexpr int N = Vec<T>::N;
    const float c = m * kLog2e;
    const float2 scale = make_float2(kLog2e, kLog2e), minus = make_float2(-c, -c);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int i = threadIdx.x; i < part.len; i += kScanThreads) {
        const uint4 v = part.template get<FLAT>(stage, i);
        float f[N];
        Vec<T>::unpack(v, f);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float2 e = ffma2(make_float2(f[k], f[k + 1]), scale, minus);
            s = fadd2(s, make_float2(ex2(e.x), ex2(e.y)));
        }
        if (Vec<T>::vmax(v) >= bar) {  // few
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (f[k] >= bar && f[k] > -INFINITY) {
                    const int to = atomicAdd(&sh.found, 1);
                    if (to < kScanList) sh.list[to] = candidate(f[k], (part.j0 + i) * N + k);
                }
            }
        }
    }
    // the rounding of c is taken back
    return (s.x + s.y) * ex2(-fmaf(m, kLog2e, -c));
}

// The sum alone, without NaN logits and for any finite m.
template <typename T>
__device__ __noinline__ float part_sum(const RowPart<T>& part, const uint4* stage, float m) {
    float s = 0.f;
    for (int i = threadIdx.x; i < part.len; i += kScanThreads) {
        float f[Vec<T>::N];
        Vec<T>::unpack(part.template get<false>(stage, i), f);
#pragma unroll
        for (int k = 0; k < Vec<T>::N; ++k) s += ex2((fmaxf(f[k], -INFINITY) - m) * kLog2e);
    }
    return s;
}

// The part's best by merging, where the list overflows: each warp merges its
// own run of vectors. Leaves all that can be among the M best in sh.list.
template <typename T, int E>
__device__ __noinline__ void scan_merge(const RowPart<T>& part, const uint4* stage, int M,
                                        ScanShared<E>& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    WarpBest<E> top;
    top.init(sh.buf[warp], lane, M);
    const int per = (part.len + kScanWarps - 1) / kScanWarps;
    const int i1 = min(part.len, (warp + 1) * per);
#pragma unroll 1
    for (int i = warp * per; i < i1; i += 32) {
        float f[Vec<T>::N];
#pragma unroll
        for (int k = 0; k < Vec<T>::N; ++k) f[k] = -INFINITY;
        if (i + lane < i1) Vec<T>::unpack(part.template get<false>(stage, i + lane), f);
#pragma unroll
        for (int k = 0; k < Vec<T>::N; ++k) top.offer(f[k], (part.j0 + i + lane) * Vec<T>::N + k);
    }
    if (lane == 0) sh.lasts[warp] = top.last;
    __syncthreads();  // every thread has read the overflowed count
    if (threadIdx.x == 0) sh.found = 0;
    __syncthreads();
    // of what the warps hold only words from the highest `last` on can be
    // among the M best: M words of that warp are
    uint64_t bar = sh.lasts[0];
#pragma unroll
    for (int w = 1; w < kScanWarps; ++w) bar = sh.lasts[w] > bar ? sh.lasts[w] : bar;
#pragma unroll
    for (int e = 0; e <= E; ++e) {
        const uint64_t w = e < E ? (32 * e + lane < M ? top.best[e < E ? e : 0] : 0)
                                 : (lane < top.count ? sh.buf[warp][lane] : 0);
        const unsigned who = __ballot_sync(~0u, w >= bar);
        int to = 0;
        if (lane == 0 && who) to = atomicAdd(&sh.found, __popc(who));
        to = __shfl_sync(~0u, to, 0);
        if (w >= bar) sh.list[to + __popc(who & ((1u << lane) - 1u))] = w;
    }
    __syncthreads();
}

template <typename T, int E>
__global__ void __launch_bounds__(kScanThreads, kScanCtas) beam_scan(const __grid_constant__ BeamArgs a) {
    using VT = Vec<T>;
    constexpr int N = VT::N;
    extern __shared__ uint4 scan_stage[];  // kScanMost + 1 vectors
    __shared__ ScanShared<E> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    const int nv = (static_cast<int>(a.V) - 1) / N + 1;
    // the parts of this CTA, in steps of the grid; those of dead beams are
    // passed over
    int64_t row = blockIdx.x / static_cast<unsigned>(a.splits);
    int piece = blockIdx.x % static_cast<unsigned>(a.splits);
    const auto step = [&] {
        row += a.row_step;
        piece += a.part_step;
        if (piece >= a.splits) {
            piece -= a.splits;
            ++row;
        }
    };
    const auto here = [&] {
        RowPart<T> p;
        p.row = static_cast<const T*>(a.logits) + row * a.V;
        p.V = static_cast<int>(a.V);
        p.j0 = piece * a.part_vec;
        p.len = min(a.part_vec, nv - p.j0);
        p.shift = static_cast<int>(reinterpret_cast<uintptr_t>(p.row) & 15u);
        return p;
    };
    while (row < a.rows && !beam_lives(a, row)) step();
    if (row < a.rows) here().fetch(scan_stage);
    while (row < a.rows) {
        const RowPart<T> part = here();
        const bool flat = part.shift == 0;
        const int64_t item = row * a.splits + piece;
        do step();
        while (row < a.rows && !beam_lives(a, row));
        cp_async_wait();
        __syncthreads();  // the part is staged, and the last one's list read
        // ---- each thread's largest logit, and the warps' t largest of those
        const float lm = flat ? part_max<true>(part, scan_stage) : part_max<false>(part, scan_stage);
        const bool small = a.M <= 16;
        const int t = small ? 4 : (a.M + kScanWarps - 1) / kScanWarps;
        uint32_t mine = lm > -INFINITY ? ordered(lm) : 0u;
        for (int i = 0; i < t; ++i) {
            const uint32_t best = __reduce_max_sync(~0u, mine);
            if (__ffs(__ballot_sync(~0u, mine == best)) - 1 == lane) mine = 0u;
            if (lane == 0) sh.tops[warp * t + i] = best;
        }
        if (threadIdx.x == 0) sh.found = 0;
        __syncthreads();
        // ---- the maximum, and the bound (0: too few threads have a logit)
        uint32_t top, bound;
        if (small) {  // M of the 8 t = 32 values, sorted over a warp's lanes
            if (warp == 0) {
                const uint32_t o = warp_sort_desc(sh.tops[lane], lane);
                if (lane == 0) sh.top = o;
                if (lane == a.M - 1) sh.bound = o;
            }
            __syncthreads();
            top = sh.top;
            bound = sh.bound;
        } else {  // every warp has t such threads
            top = __reduce_max_sync(~0u, lane < kScanWarps ? sh.tops[lane * t] : 0u);
            bound = __reduce_min_sync(~0u, lane < kScanWarps ? sh.tops[lane * t + t - 1] : ~0u);
        }
        const float m = top ? unordered(top) : -INFINITY;
        // (below +0 that is not -0: equal values)
        const float bar = !bound ? -INFINITY : unordered(bound);
        // ---- the sum, and the logits that reach the bound
        float s = flat ? part_scan<true>(part, scan_stage, m, bar, sh)
                       : part_scan<false>(part, scan_stage, m, bar, sh);
        // a NaN in the sum comes from a NaN logit, which counts as masked
        const bool usual = fabsf(m) < kHuge;
        if (!usual) s = 0.f;
        if (__syncthreads_or(isnan(s) || (!usual && fabsf(m) < INFINITY)))
            s = part_sum<T>(part, scan_stage, m);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        if (lane == 0) sh.sums[warp] = s;
        if (sh.found > kScanList) scan_merge<T, E>(part, scan_stage, a.M, sh);
        __syncthreads();  // the stage is free, the list and sums are whole
        if (row < a.rows) here().fetch(scan_stage);
        if (threadIdx.x == 0) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kScanWarps; ++w) sum += sh.sums[w];
            a.sums[item] = RowSum{m, m == INFINITY ? INFINITY : sum};
        }
        uint64_t* out = a.lists + item * a.M;
        const int n = sh.found;
        for (int i = threadIdx.x; i < n; i += kScanThreads) {
            const uint64_t w = sh.list[i];
            int rank = 0;
#pragma unroll 4
            for (int o = 0; o < n; ++o) rank += sh.list[o] > w;
            if (rank < a.M) out[rank] = w;
        }
        // no candidate in the places behind the last
        for (int i = n + threadIdx.x; i < a.M; i += kScanThreads) out[i] = 0;
    }
}

// Numbers held as the exact sum of two fp32 (48 bits and more): the scores
// of candidates are formed and compared in them. (The same in fp64, which
// this GPU issues at a sixteenth of a warp a cycle, made the pick of 16 x 8
// beams 10 us instead of 4.)
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // exact (Knuth)
    const float s = a + b;
    const float t = s - a;
    return Two{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two two_add(const Two& a, const Two& b) {
    const Two s = two_sum(a.hi, b.hi);
    const float e = s.lo + (a.lo + b.lo);
    const float hi = s.hi + e;
    return Two{hi, e - (hi - s.hi)};
}

// A candidate of a batch entry: its score as ordered integers, hi above lo
// (0: none), then its beam above its token (the order of k V + v).
struct Pick {
    uint64_t key;
    uint64_t at;
};
constexpr uint64_t kNowhere = ~uint64_t{0};
__device__ __forceinline__ bool better(const Pick& p, const Pick& q) {
    return p.key > q.key || (p.key == q.key && p.at < q.at);
}
// (a score that is not finite in fp32 is no candidate's)
__device__ __forceinline__ uint64_t score_key(const Two& s) {
    return isfinite(s.hi) ? (static_cast<uint64_t>(ordered(s.hi)) << 32) | ordered(s.lo) : 0u;
}

// What beam_pick knows of a beam. The log-sum-exp is m + logs: its parts are
// subtracted one after the other, since m may be of a size at which their
// sum loses logs.
enum : int { kBeamDead = 0, kBeamAlive = 1, kBeamFinished = 2 };
struct BeamInfo {
    Two minus_logs;
    float m, score;
    int kind;
};

// The candidate of beam k that a list's word stands for; a finished beam
// goes on with the padding token alone (word 0 of its list 0).
__device__ __forceinline__ Pick word_pick(const BeamInfo& info, int k, uint64_t w, bool front,
                                          int64_t pad) {
    const uint64_t beam = static_cast<uint64_t>(k) << 32;
    if (info.kind == kBeamAlive && w) {
        const float x = unordered(static_cast<uint32_t>(w >> 32));
        const Two s = two_add(two_add(two_sum(x, -info.m), info.minus_logs), Two{info.score, 0.f});
        return Pick{score_key(s), beam | static_cast<uint32_t>(~static_cast<uint32_t>(w))};
    }
    if (info.kind == kBeamFinished && front)
        return Pick{score_key(Two{info.score, 0.f}), beam | static_cast<uint64_t>(pad)};
    return Pick{0, kNowhere};
}

// How many of n picks are better than p, counted by the four lanes of a quad
// (which all get the sum).
__device__ __forceinline__ int quad_rank(const Pick* all, int n, const Pick& p) {
    int rank = 0;
#pragma unroll 4
    for (int o = threadIdx.x & 3; o < n; o += 4) rank += better(all[o], p);
    rank += __shfl_xor_sync(~0u, rank, 1);
    return rank + __shfl_xor_sync(~0u, rank, 2);
}

// Place i of entry b has no candidate.
__device__ __forceinline__ void no_pick(const BeamArgs& a, int64_t b, int i) {
    a.out_scores[b * a.M + i] = -INFINITY;
    a.out_beams[b * a.M + i] = -1;
    a.out_tokens[b * a.M + i] = a.pad;
}

// The M best of nl sorted lists of M picks, by one warp: lane i holds the
// first of lists i, i + 32, ...
__device__ __forceinline__ int merge_lists(const BeamArgs& a, const Pick* all, int nl, int64_t b, int lane) {
    constexpr int R = kMergeLists / 32;
    Pick head[R];
    int pos[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int l = lane + 32 * q;
        pos[q] = 0;
        head[q] = l < nl ? all[l * a.M] : Pick{0, kNowhere};
    }
    for (int r = 0; r < a.M; ++r) {
        Pick best = head[0];
#pragma unroll
        for (int q = 1; q < R; ++q)
            if (better(head[q], best)) best = head[q];
        // the warp's best: by score, then (equal ones) by beam and token
        const uint32_t hi = static_cast<uint32_t>(best.key >> 32);
        const uint32_t top = __reduce_max_sync(~0u, hi);
        if (!top) return r;  // no candidate left
        bool mine = hi == top;
        unsigned who = __ballot_sync(~0u, mine);
        if (who & (who - 1)) {
            // (every lane takes part in each reduction)
            const uint32_t lo = static_cast<uint32_t>(best.key);
            const uint32_t most = __reduce_max_sync(~0u, mine ? lo : 0u);
            mine = mine && lo == most;
            const uint32_t beam = mine ? static_cast<uint32_t>(best.at >> 32) : ~0u;
            const uint32_t first = __reduce_min_sync(~0u, beam);
            mine = mine && beam == first;
            const uint32_t token = mine ? static_cast<uint32_t>(best.at) : ~0u;
            const uint32_t least = __reduce_min_sync(~0u, token);
            mine = mine && token == least;
        }
        if (mine) {
            a.out_scores[b * a.M + r] = unordered(static_cast<uint32_t>(best.key >> 32));
            a.out_beams[b * a.M + r] = static_cast<int64_t>(best.at >> 32);
            a.out_tokens[b * a.M + r] = static_cast<int64_t>(best.at & 0xFFFFFFFFu);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (head[q].at != best.at) continue;
                ++pos[q];
                head[q] = pos[q] < a.M ? all[(lane + 32 * q) * a.M + pos[q]] : Pick{0, kNowhere};
                break;
            }
        }
    }
    return a.M;
}

// MERGE: the entry has at most kMergeLists lists.
template <bool MERGE>
__global__ void __launch_bounds__(kPickThreads) beam_pick(const __grid_constant__ BeamArgs a) {
    extern __shared__ Pick pick_smem[];
    __shared__ BeamInfo info[kMaxBeams];
    __shared__ Pick bound;
    __shared__ int nsurv;
    const int nl = a.K * a.splits;
    Pick* heads = pick_smem;  // [nl], or MERGE: all candidates [nl, M]
    Pick* surv = heads + nl;  // [M M]
    const int64_t b = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t* lists = a.lists + b * nl * a.M;
    if (threadIdx.x == 0) {
        bound = Pick{0, kNowhere};
        nsurv = 0;
    }
    pdl_wait();
    // the lists' words, on their way while the log-sum-exps are formed
    constexpr int kHold = 8;
    uint64_t held[kHold];
    if (MERGE) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int at = threadIdx.x + i * kPickThreads;
            held[i] = at < nl * a.M ? lists[at] : 0;
        }
    }
    for (int k = warp; k < a.K; k += kPickThreads / 32) {
        const int64_t row = b * a.K + k;
        const float score = a.scores[row];
        const bool done = a.finished && a.finished[row];
        // (a beam that was not scanned has left its sums as they were: not used)
        const RowSum* sums = a.sums + row * a.splits;
        float m = kLowest;
        for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, sums[i].m);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        Two s{0.f, 0.f};
        for (int i = lane; i < a.splits; i += 32) {
            const RowSum t = sums[i];  // (exp2(-inf) = 0 for a part with no token)
            s = two_add(s, Two{t.s * exp2f((t.m - m) * kLog2e), 0.f});
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s = two_add(s, Two{__shfl_xor_sync(~0u, s.hi, d), __shfl_xor_sync(~0u, s.lo, d)});
        if (lane == 0) {
            // log s = e ln 2 + log f, f in [0.7, 1.42): logf there is off by
            // 2^-25 or less
            const uint32_t bits = __float_as_uint(s.hi);
            int e = static_cast<int>(bits >> 23) - 127;
            float f = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
            if (f > 1.41421356f) {
                f *= 0.5f;
                ++e;
            }
            const float ef = static_cast<float>(e);
            constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;  // ln 2 as two fp32
            const float hi = ef * kLn2;
            Two logs = two_add(Two{hi, fmaf(ef, kLn2, -hi) + ef * kLn2Lo}, two_sum(logf(f), s.lo / s.hi));
            BeamInfo w;
            w.m = m;
            w.minus_logs = Two{-logs.hi, -logs.lo};
            w.score = score;
            w.kind = !isfinite(score) ? kBeamDead
                     : done           ? kBeamFinished
                     : (isfinite(m) && s.hi > 0.f && isfinite(s.hi)) ? kBeamAlive : kBeamDead;
            info[k] = w;
        }
    }
    __syncthreads();
    const auto pick_of = [&](int l, int i, uint64_t w) {
        const int k = l / a.splits;
        return word_pick(info[k], k, w, i == 0 && l == k * a.splits, a.pad);
    };
    if constexpr (MERGE) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int at = threadIdx.x + i * kPickThreads;
            if (at < nl * a.M) heads[at] = pick_of(at / a.M, at % a.M, held[i]);
        }
        for (int at = threadIdx.x + kHold * kPickThreads; at < nl * a.M; at += kPickThreads)
            heads[at] = pick_of(at / a.M, at % a.M, lists[at]);
        __syncthreads();
        if (warp == 0) {
            const int n = merge_lists(a, heads, nl, b, lane);
            for (int i = n + lane; i < a.M; i += 32) no_pick(a, b, i);
        }
        return;
    }
    const auto at = [&](int l, int i) { return pick_of(l, i, lists[static_cast<int64_t>(l) * a.M + i]); };
    for (int l = threadIdx.x; l < nl; l += kPickThreads) heads[l] = at(l, 0);
    __syncthreads();
    // the M-th best of the lists' first candidates
    for (int l0 = 0; l0 < nl; l0 += kPickThreads / 4) {
        const int l = l0 + static_cast<int>(threadIdx.x >> 2);
        const Pick p = l < nl ? heads[l] : Pick{0, kNowhere};
        const int rank = quad_rank(heads, nl, p);
        if (p.key && rank == a.M - 1) bound = p;
    }
    __syncthreads();
    const Pick bar = bound;
    // every candidate that is not below it, a warp a list (M lists at most
    // start above it): the lanes look at the list's candidates side by side
    for (int l = warp; l < nl; l += kPickThreads / 32) {
        const Pick h = heads[l];
        if (!h.key || better(bar, h)) continue;
        for (int i = lane; i - lane < a.M; i += 32) {
            Pick p{0, kNowhere};
            if (i < a.M) p = at(l, i);
            const bool in = p.key && !better(bar, p);
            const unsigned who = __ballot_sync(~0u, in);
            int to = 0;
            if (lane == 0) to = atomicAdd(&nsurv, __popc(who));
            to = __shfl_sync(~0u, to, 0);
            if (in) surv[to + __popc(who & ((1u << lane) - 1u))] = p;
            if (who != ~0u) break;  // lists descend
        }
    }
    __syncthreads();
    const int n = nsurv;
    for (int i0 = 0; i0 < n; i0 += kPickThreads / 4) {
        const int i = i0 + static_cast<int>(threadIdx.x >> 2);
        const Pick p = i < n ? surv[i] : Pick{0, kNowhere};
        const int rank = quad_rank(surv, n, p);
        if (i < n && rank < a.M && (threadIdx.x & 3) == 0) {
            a.out_scores[b * a.M + rank] = unordered(static_cast<uint32_t>(p.key >> 32));
            a.out_beams[b * a.M + rank] = static_cast<int64_t>(p.at >> 32);
            a.out_tokens[b * a.M + rank] = static_cast<int64_t>(p.at & 0xFFFFFFFFu);
        }
    }
    for (int i = n + threadIdx.x; i < a.M; i += kPickThreads) no_pick(a, b, i);
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
    const int64_t* beams;  // [B, K], rows beams_row apart
    int64_t beams_row, B;
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
                const int64_t s = a.beams[b * a.beams_row + k];
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

// How the rows are dealt out: `splits` parts a row, over one wave of CTAs
// (kScanCtas an SM) in turn. As few parts as the stage allows, since each
// costs a bound and a ranking (16 x 8 x 128256 bf16 in 7, 10 and 12 parts: 22,
// 26 and 38 us), but, for few rows, up to two an SM of at least 1000 vectors
// (4 x 32000 in 1 and 4 parts: 8.5 and 7.9 us).
constexpr int64_t kScanMin = 1000;
struct ScanPlan {
    int64_t part_vec, grid;
    int splits;
};
ScanPlan scan_plan(int64_t rows, int64_t V, int dtype, int sms) {
    const int64_t N = dtype == CE_F32 ? 4 : 8;
    const int64_t nv = (V + N - 1) / N;
    const int64_t least = (nv + kScanMost - 1) / kScanMost;
    const int64_t fill = (2L * std::max(sms, 1) + rows - 1) / std::max<int64_t>(rows, 1);
    const int64_t s = std::max(least, std::min(fill, nv / kScanMin));
    ScanPlan p;
    p.part_vec = (nv + s - 1) / s;
    p.splits = static_cast<int>((nv + p.part_vec - 1) / p.part_vec);
    p.grid = std::min<int64_t>(rows * p.splits, int64_t{kScanCtas} * std::max(sms, 1));
    return p;
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
    if (K > kMaxBeams || M > kMaxCandidates || V > kMaxVocab || B > kMaxVocab) {
        record_message("beam search takes at most 32 beams, 64 candidates, 2^20 batch entries "
                       "and 2^20 tokens");
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
    int sms = 0;
    if (sm_count(&sms) != CE_OK) return 0;
    const int64_t lists = B * K * scan_plan(B * K, V, dtype, sms).splits;
    return static_cast<size_t>(up256(lists * static_cast<int64_t>(sizeof(RowSum))) +
                               up256(lists * M * 8));
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
    const uintptr_t b = dtype == CE_F32 ? 4 : 2;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        reinterpret_cast<uintptr_t>(logits) % b ||
        workspace_bytes < static_cast<size_t>(B * K * M * 8))  // (of one part a row)
        return CE_ERR_INVALID_ARG;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != CE_OK) return rc;
    const ScanPlan plan = scan_plan(B * K, V, dtype, sms);
    const int64_t lists = B * K * plan.splits;
    const int64_t sums_bytes = up256(lists * static_cast<int64_t>(sizeof(RowSum)));
    if (workspace_bytes < static_cast<size_t>(sums_bytes + up256(lists * M * 8)))
        return CE_ERR_INVALID_ARG;
    BeamArgs a = {};
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.rows = B * K;
    a.V = V;
    a.K = static_cast<int>(K);
    a.M = static_cast<int>(M);
    a.splits = plan.splits;
    a.part_vec = static_cast<int>(plan.part_vec);
    a.row_step = static_cast<int>(plan.grid / plan.splits);
    a.part_step = static_cast<int>(plan.grid % plan.splits);
    a.pad = pad_token;
    a.sums = static_cast<RowSum*>(workspace);
    a.lists = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + sums_bytes);
    a.out_scores = out_scores;
    a.out_beams = out_beams;
    a.out_tokens = out_tokens;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    const size_t lists_n = static_cast<size_t>(K * a.splits);
    const bool merge = lists_n <= kMergeLists;
    const size_t smem = sizeof(Pick) * static_cast<size_t>(merge ? lists_n * M : lists_n + M * M);
    if (smem > kPickSmem) {
        record_message("a batch entry's beams have more parts than the selection holds");
        return CE_ERR_UNSUPPORTED;
    }
    const void* scan = M <= 32 ? scan_fn<1>(dtype) : scan_fn<2>(dtype);
    rc = tc_smem_limit(scan, 16 * (kScanMost + 1));
    if (rc != CE_OK) return rc;
    cudaError_t e = cudaLaunchKernel(scan, dim3(static_cast<unsigned>(plan.grid)), dim3(kScanThreads), args,
                                     16 * static_cast<size_t>(plan.part_vec + 1), st);
    if (e != cudaSuccess) return record_cuda_failure(e, "beam scan launch");
    const void* pick = merge ? (const void*)&beam_pick<true> : (const void*)&beam_pick<false>;
    if (smem > 48 * 1024) {
        rc = tc_smem_limit(pick, kPickSmem);
        if (rc != CE_OK) return rc;
    }
    return launch_pdl(pick, dim3(static_cast<unsigned>(B)), kPickThreads, smem, st, &a,
                      "beam pick launch");
}

extern "C" ce_status ce_beam_reorder(const ce_beam_state* states, int n, const int64_t* beams,
                                     int64_t beams_row, int64_t B, int64_t K, ce_stream_t stream) {
    if (n < 0 || B < 0 || K < 1 || beams_row < K) return CE_ERR_INVALID_ARG;
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
        for (int j = 0; j < i; ++j)  // one state twice would be written by two
            if (states[j].dst == s.dst && states[j].blocks && states[j].block_bytes)
                return CE_ERR_INVALID_ARG;
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
        a.beams_row = beams_row;
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
