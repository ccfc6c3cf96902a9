// One step of beam search over logits [B, K, V]: the M best continuations of
// each batch entry's K beams by score + log-softmax, and the reordering of
// the beams' states. Two kernels for the selection, one for the reordering.
//
// Selection. With lse_k = log sum_v exp(x_kv), candidate (k, v) has the score
// s_k + x_kv - lse_k, so within a beam the order is that of the logits:
//  1. beam_scan reads every logit once. A row is split over CTAs and their
//     warps; a lane keeps a running maximum and sum of the softmax, a warp
//     its M best logits in a sorted list over its lanes. A logit that can
//     still matter goes to a buffer in shared memory; 32 of them are sorted
//     and merged into the list by a bitonic network. What can matter is
//     bounded from the lanes' largest logits: with m = ceil(M / 8), each of
//     the 8 warps has m lanes whose largest is at least the warp's m-th
//     largest of those, so M logits of the CTA are at least the smallest of
//     the 8 values. Formed after 1, 2, 4, ... blocks, it lets some 40
//     logits of each doubling pass, where a list that starts empty would
//     merge the first blocks whole. A CTA ranks what its warps hold by
//     counting and writes M candidates and {max, sum}.
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
constexpr int kScanCtas = 3;    // CTAs an SM
constexpr int kScanVec = 4;     // 16-byte vectors a lane holds at a time
constexpr int kScanBuf = 128;   // words of a warp's buffer (fewer than 32 at the start of a block)
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
    float m;     // maximum (kLowest with no token)
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
    int64_t pad;
    RowSum* sums;        // [rows, splits]
    uint64_t* lists;     // [rows, splits, M]
    float* out_scores;   // [B, M]
    int64_t* out_beams;
    int64_t* out_tokens;
};

// The most shared memory that beam_pick takes: 32 beams of 64 parts and 64
// candidates squared, or staged lists below that.
constexpr size_t kPickSmem = 16 * (kMaxBeams * kMaxSplits + kMaxCandidates * kMaxCandidates);

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
    uint64_t* buf;  // kScanBuf words of shared memory of this warp
    int count;
    uint64_t last;  // a candidate must lie above this to matter,
    float bar;      // a logit above this: of last, or just below the bound
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

    // At least M logits of the CTA are `least` or more.
    __device__ __forceinline__ void bound(float least) {
        if (least > -INFINITY && (static_cast<uint64_t>(ordered(least)) << 32) - 1u > last) {
            last = (static_cast<uint64_t>(ordered(least)) << 32) - 1u;
            // the next value below it (below +0 that is not -0)
            bar = least == 0.f ? -__uint_as_float(1u) : unordered(static_cast<uint32_t>(last >> 32));
        }
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

// A part of a row: vectors [j0, j1) of a warp, vector j being the elements
// N j .. N j + N - 1 wherever the row starts in memory, so that equal rows
// are summed alike (and equal beams tie exactly).
template <typename T>
struct RowPart {
    const T* row;
    int V, j0, j1;
    int in0, in1;  // the vectors in [in0, in1) are loaded whole
    int shift;     // bytes from the 16-byte boundary before the row to the row
    bool live;

    // vector j by element, with -inf outside the row and the part
    __device__ __forceinline__ uint4 edge(int j) const {
        constexpr int N = Vec<T>::N;
        const uint32_t none = neg_inf_word<T>();
        uint32_t w[4] = {none, none, none, none};
        if (j < j1) {
            const int e = j * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (e + i >= V) continue;
                if constexpr (sizeof(T) == 4) {
                    w[i] = reinterpret_cast<const uint32_t*>(row)[e + i];
                } else {
                    const uint32_t h = reinterpret_cast<const uint16_t*>(row)[e + i];
                    w[i / 2] = (i & 1) ? (w[i / 2] & 0xFFFFu) | (h << 16) : (w[i / 2] & 0xFFFF0000u) | h;
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }

    // vector j of a row that is not 16-byte aligned, from the two aligned
    // vectors that it lies in (both inside the row)
    __device__ __forceinline__ uint4 apart(int j) const {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) - shift) + j;
        const uint4 a = p[0], b = p[1];
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = (shift & 8) ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = (shift & 4) ? w[i + 1] : w[i];
        const int bits = 8 * (shift & 3);
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }

    // this lane's vectors j + lane, j + 32 + lane, ...
    template <int NV>
    __device__ __forceinline__ void load(int j, uint4 (&v)[NV]) const {
        const int lane = threadIdx.x & 31;
        if (j >= in0 && j + 32 * NV <= in1) {
            if (shift) {
#pragma unroll
                for (int k = 0; k < NV; ++k) v[k] = apart(j + 32 * k + lane);
            } else {
                const uint4* p = reinterpret_cast<const uint4*>(row) + (j + lane);
#pragma unroll
                for (int k = 0; k < NV; ++k) v[k] = __ldcs(p + 32 * k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) v[k] = edge(j + 32 * k + lane);
        }
    }
};

// A lane's part of a log-sum-exp: sum of exp2(log2e x - c) with c = log2e m
// rounded to fp32, m the running maximum: one FFMA and one exp2 a logit. The
// rounding of c is taken back when the sum is brought to another maximum.
// Logits of a size at which c overflows (kHuge) do not raise m: below it
// they add 0, as they should next to any other logit, and a warp that has no
// other, or one above it, sums again by sum_apart.
constexpr float kHuge = 2e38f;
struct LaneSum {
    float m, c, s;

    __device__ __forceinline__ void raise(float to) {
        if (to > m && to > -kHuge) {
            const float nc = to * kLog2e;
            s *= ex2(c - nc);
            m = to;
            c = nc;
        }
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&f)[N]) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) p[i & 3] += ex2(fmaf(f[i], kLog2e, -c));
        s += (p[0] + p[1]) + (p[2] + p[3]);
    }
    // the sum relative to a maximum `to` that is finite
    __device__ __forceinline__ float relative(float to) const { return s * ex2(-fmaf(to, kLog2e, -c)); }
};

// A lane's sum of exp(x - m) over its vectors of a part, without NaN logits
// and for any finite m.
template <typename T>
__device__ __noinline__ float sum_apart(const RowPart<T>& part, float m) {
    float s = 0.f;
    for (int j = part.j0; j < part.j1; j += 32) {
        uint4 v[1];
        part.load(j, v);
        float f[Vec<T>::N];
        Vec<T>::unpack(v[0], f);
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) s += ex2((fmaxf(f[i], -INFINITY) - m) * kLog2e);
    }
    return s;
}

// Part `item` mod splits of row item / splits, as this warp takes it.
template <typename T>
__device__ __forceinline__ RowPart<T> row_part(const BeamArgs& a, int64_t item) {
    constexpr int N = Vec<T>::N;
    RowPart<T> p;
    p.V = static_cast<int>(a.V);
    p.live = item < a.rows * a.splits;
    const int64_t r = p.live ? item / a.splits : 0;
    const int off = static_cast<int>(item - r * a.splits) * a.part_vec;
    p.row = static_cast<const T*>(a.logits) + r * a.V;
    p.shift = static_cast<int>(reinterpret_cast<uintptr_t>(p.row) & 15u);
    const int nv = (p.V - 1) / N + 1;
    const int end = min(off + a.part_vec, nv);
    const int per = (a.part_vec + kScanWarps - 1) / kScanWarps;
    p.j0 = off + static_cast<int>(threadIdx.x >> 5) * per;
    p.j1 = min(p.j0 + per, end);
    // an unaligned vector j lies in the aligned ones j and j + 1
    p.in0 = p.shift ? 1 : 0;
    const int whole = p.shift ? static_cast<int>((a.V * static_cast<int64_t>(sizeof(T)) + p.shift) / 16) - 1
                              : p.V / N;
    p.in1 = min(whole, p.j1);
    if (p.live) p.live = beam_lives(a, r);
    return p;
}

template <int E>
struct ScanShared {
    uint64_t buf[kScanWarps][kScanBuf];
    int count[kScanWarps];  // words in buf
    uint64_t lists[kScanWarps * (32 * E + 32)];
    uint64_t lasts[kScanWarps];
    RowSum sums[kScanWarps];
    float least[kScanWarps];
    int found;
};

// One part of a row. `next` holds its first block on entry, and that of
// `after` on return.
template <typename T, int E>
__device__ __forceinline__ void scan_part(const BeamArgs& a, const RowPart<T>& part,
                                          const RowPart<T>& after, int64_t item,
                                          uint4 (&v)[kScanVec], uint4 (&next)[kScanVec],
                                          ScanShared<E>& sh) {
    using VT = Vec<T>;
    constexpr int N = VT::N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();  // the shared arrays have been read by the part before
    if (lane == 0) sh.count[warp] = 0;  // (block 1 synchronises)
    WarpBest<E> top;
    top.init(sh.buf[warp], lane, a.M);
    LaneSum sum{-INFINITY, kLowest, 0.f};
    float lm = -INFINITY;  // the lane's maximum
    unsigned block = 1;
    for (int j = part.j0; block == 1 || j < part.j1; j += 32 * kScanVec, ++block) {
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) v[k] = next[k];
        if (j + 32 * kScanVec < part.j1) part.load(j + 32 * kScanVec, next);
        else if (after.live) after.load(after.j0, next);
        float vm[kScanVec];
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) vm[k] = VT::vmax(v[k]);
        const float bm = fmaxf(fmaxf(vm[0], vm[1]), fmaxf(vm[2], vm[3]));
        static_assert(kScanVec == 4, "four vectors a lane");
        lm = fmaxf(lm, bm);
        if ((block & (block - 1)) == 0) {
            // the m-th largest of the lanes' largest so far
            uint32_t mine = lm > -INFINITY ? ordered(lm) : 0u;
            uint32_t best = 0;
            for (int i = 0; i < (a.M + kScanWarps - 1) / kScanWarps; ++i) {
                best = __reduce_max_sync(~0u, mine);
                if (__ffs(__ballot_sync(~0u, mine == best)) - 1 == lane) mine = 0u;
            }
            volatile float* known = sh.least;
            if (lane == 0) known[warp] = best ? unordered(best) : -INFINITY;
            // every warp's first value; later ones only rise, so that an
            // older one is a bound as well
            if (block == 1) __syncthreads();
            else __syncwarp();
            float l = known[0];
#pragma unroll
            for (int w = 1; w < kScanWarps; ++w) l = fminf(l, known[w]);
            top.bound(l);
        }
        sum.raise(bm);
#pragma unroll
        for (int k = 0; k < kScanVec; ++k) {
            float f[N];
            VT::unpack(v[k], f);
            sum.add(f);
        }
        // tokens of later blocks are larger: an equal logit does not matter
        if (__any_sync(~0u, bm > top.bar)) {
#pragma unroll
            for (int k = 0; k < kScanVec; ++k) {
                if (vm[k] > top.bar) {  // few lanes
                    float f[N];
                    VT::unpack(v[k], f);
                    const int t0 = (j + 32 * k + lane) * N;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (f[i] > top.bar) {
                            const int to = atomicAdd(&sh.count[warp], 1);
                            if (to < kScanBuf) sh.buf[warp][to] = candidate(f[i], t0 + i);
                        }
                    }
                }
            }
            __syncwarp();
            const int before = top.count;
            top.count = sh.count[warp];
            if (top.count > kScanBuf) {
                // more than the buffer holds (equal or ascending logits): the
                // block once more, a logit a lane at a time
                top.count = before;
#pragma unroll 1
                for (int k = 0; k < kScanVec; ++k) {
                    const uint4 again = part.edge(j + 32 * k + lane);
                    float f[N];
                    VT::unpack(again, f);
#pragma unroll 1
                    for (int i = 0; i < N; ++i) {
                        float x = f[0];
#pragma unroll
                        for (int q = 1; q < N; ++q) x = q == i ? f[q] : x;
                        top.offer(x, (j + 32 * k + lane) * N + i);
                    }
                }
            }
            top.drain();
            if (lane == 0) sh.count[warp] = top.count;
            __syncwarp();
        }
    }
    // the warp's sum, then the CTA's list and sum
    float wm = lm;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wm = fmaxf(wm, __shfl_xor_sync(~0u, wm, d));
    float ws = 0.f;
    if (wm == INFINITY) {
        ws = wm;  // no log-sum-exp
    } else if (wm > -INFINITY) {
        // a NaN in a sum comes from a NaN logit, which counts as masked
        if (__any_sync(~0u, isnan(sum.s)) || fabsf(wm) >= kHuge)
            ws = sum_apart<T>(part, wm);
        else
            ws = sum.relative(wm);
    }
    wm = fmaxf(wm, kLowest);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ws += __shfl_xor_sync(~0u, ws, d);
    if (lane == 0) sh.sums[warp] = RowSum{wm, ws};
    if (lane == 0) sh.lasts[warp] = top.last;
    if (threadIdx.x == 0) sh.found = 0;
    __syncthreads();
    if (warp == 0) {
        RowSum t = lane < kScanWarps ? sh.sums[lane] : RowSum{kLowest, 0.f};
        float tm = t.m;
#pragma unroll
        for (int d = kScanWarps / 2; d > 0; d >>= 1) tm = fmaxf(tm, __shfl_xor_sync(~0u, tm, d));
        float ts = t.s * ex2((t.m - tm) * kLog2e);
#pragma unroll
        for (int d = kScanWarps / 2; d > 0; d >>= 1) ts += __shfl_xor_sync(~0u, ts, d);
        if (lane == 0) a.sums[item] = RowSum{tm, ts};
    }
    // The warps' lists and buffers as one: of what they hold, only words from
    // the highest `last` on can be among the M best (M words of that warp, or
    // of the CTA, are), so that about 2 M are ranked.
    uint64_t bar = sh.lasts[0];
#pragma unroll
    for (int w = 1; w < kScanWarps; ++w) bar = sh.lasts[w] > bar ? sh.lasts[w] : bar;
    __syncwarp();
#pragma unroll
    for (int e = 0; e <= E; ++e) {
        const uint64_t w = e < E ? (32 * e + lane < a.M ? top.best[e < E ? e : 0] : 0)
                                 : (lane < top.count ? sh.buf[warp][lane] : 0);
        const unsigned who = __ballot_sync(~0u, w >= bar);
        int to = 0;
        if (lane == 0 && who) to = atomicAdd(&sh.found, __popc(who));
        to = __shfl_sync(~0u, to, 0);
        if (w >= bar) sh.lists[to + __popc(who & ((1u << lane) - 1u))] = w;
    }
    __syncthreads();
    uint64_t* out = a.lists + item * a.M;
    const int n = sh.found;
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
        const uint64_t w = sh.lists[i];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < n; ++o) rank += sh.lists[o] > w;
        if (rank < a.M) out[rank] = w;
    }
    // no candidate in the places behind the last
    for (int i = n + threadIdx.x; i < a.M; i += kScanThreads) out[i] = 0;
}

template <typename T, int E>
__global__ void __launch_bounds__(kScanThreads, kScanCtas) beam_scan(const __grid_constant__ BeamArgs a) {
    __shared__ ScanShared<E> sh;
    pdl_launch_dependents();
    const int64_t items = a.rows * a.splits;
    uint4 v[kScanVec], next[kScanVec];
    RowPart<T> part = row_part<T>(a, blockIdx.x);
    if (part.live) part.load(part.j0, next);
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        // the next part's first block is loaded before this one's end is worked off
        const RowPart<T> after = row_part<T>(a, item + gridDim.x);
        if (part.live) {
            scan_part<T, E>(a, part, after, item, v, next, sh);
        } else if (after.live) {
            after.load(after.j0, next);
        }
        part = after;
    }
}

// A candidate of a batch entry: its score in 64 bits as an ordered integer
// (0: none), then its beam above its token (the order of k V + v).
struct Pick {
    uint64_t key;
    uint64_t at;
};
constexpr uint64_t kNowhere = ~uint64_t{0};
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

// What beam_pick knows of a beam. The log-sum-exp is m + logs: its parts are
// subtracted one after the other, since m may be of a size at which their
// sum loses logs.
enum : int { kBeamDead = 0, kBeamAlive = 1, kBeamFinished = 2 };
struct BeamInfo {
    double m, logs, score;
    int kind;
};

// The candidate of beam k that a list's word stands for; a finished beam
// goes on with the padding token alone (word 0 of its list 0).
__device__ __forceinline__ Pick word_pick(const BeamInfo& info, int k, uint64_t w, bool front,
                                          int64_t pad) {
    const uint64_t beam = static_cast<uint64_t>(k) << 32;
    if (info.kind == kBeamAlive && w) {
        const double x = static_cast<double>(unordered(static_cast<uint32_t>(w >> 32)));
        return Pick{ordered64(((x - info.m) - info.logs) + info.score),
                    beam | static_cast<uint32_t>(~static_cast<uint32_t>(w))};
    }
    if (info.kind == kBeamFinished && front)
        return Pick{ordered64(info.score), beam | static_cast<uint64_t>(pad)};
    return Pick{0, kNowhere};
}

// STAGED: the entry's lists are held in shared memory (all the loads at
// once); else they are read again where needed.
template <bool STAGED>
__global__ void __launch_bounds__(kPickThreads) beam_pick(const __grid_constant__ BeamArgs a) {
    extern __shared__ Pick pick_smem[];
    __shared__ BeamInfo info[kMaxBeams];
    __shared__ Pick bound;
    __shared__ int nsurv;
    const int nl = a.K * a.splits;
    Pick* heads = pick_smem;  // [nl]
    Pick* surv = heads + nl;  // [M M]
    uint64_t* words = reinterpret_cast<uint64_t*>(surv + a.M * a.M);  // [nl, M], STAGED
    const int64_t b = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t* lists = a.lists + b * nl * a.M;
    if (threadIdx.x == 0) {
        bound = Pick{0, kNowhere};
        nsurv = 0;
    }
    pdl_wait();
    if (STAGED)
        for (int i = threadIdx.x; i < nl * a.M; i += kPickThreads) words[i] = lists[i];
    for (int k = warp; k < a.K; k += kPickThreads / 32) {
        const int64_t row = b * a.K + k;
        const float score = a.scores[row];
        const bool done = a.finished && a.finished[row];
        // (a beam that was not scanned has left its sums as they were: not used)
        RowSum t{kLowest, 0.f};
        if (lane < a.splits) t = a.sums[row * a.splits + lane];
        RowSum u{kLowest, 0.f};
        if (lane + 32 < a.splits) u = a.sums[row * a.splits + 32 + lane];
        static_assert(kMaxSplits <= 64, "two parts a lane");
        float m = fmaxf(t.m, u.m);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        double s = static_cast<double>(t.s * exp2f((t.m - m) * kLog2e)) +
                   static_cast<double>(u.s * exp2f((u.m - m) * kLog2e));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        if (lane == 0) {
            // log s from its binary exponent and a mantissa near 1: logf there
            // is off by 2^-25 or less, the mantissa's rounding is put back
            const long long bits = __double_as_longlong(s);
            const int e = static_cast<int>((bits >> 52) & 0x7FF) - 1022;
            const double f = __longlong_as_double((bits & 0x000FFFFFFFFFFFFFLL) | 0x3FE0000000000000LL) *
                             1.4142135623730951;  // [0.7, 1.42)
            const float f32 = static_cast<float>(f);
            BeamInfo w;
            w.m = static_cast<double>(m);
            w.logs = (e - 0.5) * 0.6931471805599453 +
                     static_cast<double>(logf(f32) + static_cast<float>(f - f32) / f32);
            w.score = static_cast<double>(score);
            w.kind = !isfinite(score) ? kBeamDead
                     : done           ? kBeamFinished
                     : (isfinite(m) && s > 0.0 && isfinite(s)) ? kBeamAlive : kBeamDead;
            info[k] = w;
        }
    }
    __syncthreads();
    const auto at = [&](int l, int i) {
        const int k = l / a.splits;
        const uint64_t w = STAGED ? words[l * a.M + i] : lists[static_cast<int64_t>(l) * a.M + i];
        return word_pick(info[k], k, w, i == 0 && l == k * a.splits, a.pad);
    };
    for (int l = threadIdx.x; l < nl; l += kPickThreads) heads[l] = at(l, 0);
    __syncthreads();
    // the M-th best of the lists' first candidates
    for (int l = threadIdx.x; l < nl; l += kPickThreads) {
        const Pick p = heads[l];
        if (!p.key) continue;
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < nl; ++o) rank += better(heads[o], p);
        if (rank == a.M - 1) bound = p;
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
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
        const Pick p = surv[i];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < n; ++o) rank += better(surv[o], p);
        if (rank < a.M) {
            a.out_scores[b * a.M + rank] = static_cast<float>(unordered64(p.key));
            a.out_beams[b * a.M + rank] = static_cast<int64_t>(p.at >> 32);
            a.out_tokens[b * a.M + rank] = static_cast<int64_t>(p.at & 0xFFFFFFFFu);
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

// How the rows are dealt out: `splits` parts a row, all parts over one wave
// of CTAs (kScanCtas an SM) in turn. A part costs its bytes and about as
// much as another 24 KB (the first bound, the joining of the warps' lists);
// the CTAs take ceil(parts / CTAs) parts each.
constexpr int64_t kScanMin = 512;  // vectors of a part at least: 8 KB
struct ScanPlan {
    int64_t part_vec, grid;
    int splits;
};
ScanPlan scan_plan(int64_t rows, int64_t V, int dtype, int sms) {
    const int64_t N = dtype == CE_F32 ? 4 : 8;
    const int64_t nv = (V + N - 1) / N;
    const int64_t ctas = int64_t{kScanCtas} * std::max(sms, 1);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, nv / kScanMin));
    ScanPlan p{nv, 0, 1};
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s <= most; ++s) {
        const int64_t vec = (nv + s - 1) / s;
        const int64_t cost = (rows * s + ctas - 1) / ctas * (vec + 1536);
        if (cost < best) {
            best = cost;
            p.part_vec = vec;
            p.splits = static_cast<int>((nv + vec - 1) / vec);
        }
    }
    p.grid = std::min<int64_t>(rows * p.splits, ctas);
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
    a.pad = pad_token;
    a.sums = static_cast<RowSum*>(workspace);
    a.lists = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + sums_bytes);
    a.out_scores = out_scores;
    a.out_beams = out_beams;
    a.out_tokens = out_tokens;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void* args[] = {&a};
    cudaError_t e = cudaLaunchKernel(M <= 32 ? scan_fn<1>(dtype) : scan_fn<2>(dtype),
                                     dim3(static_cast<unsigned>(plan.grid)),
                                     dim3(kScanThreads), args, 0, st);
    if (e != cudaSuccess) return record_cuda_failure(e, "beam scan launch");
    size_t smem = sizeof(Pick) * static_cast<size_t>(K * a.splits + M * M);
    const size_t words = 8 * static_cast<size_t>(K * a.splits * M);
    const bool staged = smem + words <= kPickSmem;
    if (staged) smem += words;
    const void* pick = staged ? (const void*)&beam_pick<true> : (const void*)&beam_pick<false>;
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPickSmem));
        if (e != cudaSuccess) return record_cuda_failure(e, "beam pick attributes");
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
