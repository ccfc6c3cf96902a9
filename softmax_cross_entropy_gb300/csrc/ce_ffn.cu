// The gated feed-forward block y = residual + dropout(h Wd^T), h = act(x
// Wg^T) * (x Wu^T), forward and backward, on the fifth-generation tensor
// cores. x [rows, H], Wg and Wu [I, H], Wd [O, I], all bf16 or fp16 with
// fp32 accumulation.
//
// One kernel, the pipeline of the GEMM in ce_gemm_tc.cu (a TMA producer
// warp, an MMA-issuing warp, eight epilogue warps; persistent, one CTA an
// SM), in five forms (FfnMode) that differ in what a tile's K blocks are
// made of and in the epilogue:
//  * kGateUp: a tile's 256 accumulator columns are 128 columns of x Wg^T and
//    the same 128 of x Wu^T (the B tile is 128 rows of each weight), so the
//    epilogue has both and writes act(g) * u: g and u never leave the chip
//    unless a backward needs them;
//  * kDown: y = h Wd^T with dropout and the residual sum in the epilogue;
//  * kDact: dh = dz Wd; the epilogue multiplies by what the forward kept of
//    each element, s = u act'(g) and a = act(g), and writes dg = dh s and du =
//    dh a; dh itself is never stored;
//  * kDx: dx = dg Wg + du Wu as one product whose K runs over dg, then du;
//  * kDw: dWg = dg^T x, dWu = du^T x and dWd = dz^T h as one launch over the
//    tiles of all three (one tail for the SMs instead of three).
// Roundings to 16 bits: h, dg and du, which feed tensor-core products, once
// each from fp32. s and a stay in fp32 (kept in 16 bits they made the
// gradients' errors 1.7 instead of 1.4 times that of one rounding, and saved
// 60 of 2460 us of the 4096 x 4096 x 12288 training step); dropout and the residual
// are applied in fp32 before y's only rounding; dz is dy with zeros, its
// factor 1 / (1 - p) is applied to the products in fp32.
//
// The TMA wants rows of whole 16 bytes. Operands that have others (H, I or O
// not a multiple of 8) are packed into rows of such a length by a kernel of
// their own first.
//
// Bound by the tensor cores from about 300 rows on (6 rows H I operations on
// 6 H I bytes of weights); ce_ffn_rows.cu takes few rows. (Starting a launch
// early, by programmatic dependence, as the form for few rows does, gained
// nothing at 1023 rows and cost 3% of a training step, whose waiting CTAs
// draw power.)
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <string>

#include "ce_ffn.cuh"
#include "ce_philox.cuh"
#include "ce_tc.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);
void record_message(const std::string& msg);
ce_status library_status_word(cudaStream_t st, unsigned** out);
bool drop_spec(double p, uint64_t seed, uint64_t offset, const int64_t* state, DropSpec* out);
// the form for few rows (ce_ffn_rows.cu)
int64_t ffn_rows_workspace(int64_t rows, int64_t H8, int64_t I8, int64_t O, int sms);
ce_status ffn_rows_fwd(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                       const void* residual, int dtype, int64_t rows, int64_t H8, int64_t I,
                       int64_t I8, int64_t O, int act, const DropSpec& drop, void* y, void* h,
                       float* s, float* a, void* workspace, int sms, uint64_t timeout_ns,
                       unsigned* status, cudaStream_t st);

namespace {

enum FfnMode : int { kGateUp, kDown, kDact, kDx, kDw };

// Tile shapes, 256 accumulator columns wide:
//  * 128: 128 rows on one SM, 4 stages of 48 KB, two accumulators;
//  * 256: 256 rows on one SM, 3 stages of 64 KB, its two halves in all of
//    the tensor memory: the epilogue does not overlap the next tile (dx and
//    the weight gradients, whose epilogue is short);
//  * kPair: 256 rows on a pair of SMs (a cluster of two CTAs whose tensor
//    cores work as one: each holds 128 rows of A, half of B's 256 columns and
//    128 rows of the accumulator), 3 stages of 64 KB a CTA, two accumulators.
//    Each byte staged feeds twice the multiplications of the 128-row tile,
//    and the epilogue of a tile overlaps the next tile's products. A stage
//    holds two K blocks, which the products wait for together and give back
//    one by one: with a wait for each block (6 stages) a block took 620 to 650
//    cycles, of which its products are 512, whatever the tile's width. The
//    forward of 1024 rows of 4096 x 12288 205 us then, 194 with a wait and a
//    return for two, 187 so; 4096 rows 730, 680 and 655; stages of three
//    blocks 212 and 684. Where B is K-major the tile may be 224 or 192
//    columns wide.
constexpr int kPair = 2;
template <int SHAPE>
struct FfnTile {
    static constexpr bool kTwo = SHAPE == kPair;
    static constexpr int kRows = kTwo ? 256 : SHAPE;
    static constexpr int kSub = kTwo ? 2 : 1;  // K blocks of a stage
    static constexpr int kStages = kTwo ? 3 : SHAPE == 256 ? 3 : 4;
    static constexpr int kHalves = SHAPE == 256 ? 2 : 1;  // 128-row MMAs a K step
    static constexpr int kAccBufs = SHAPE == 256 ? 1 : 2;
    static constexpr uint32_t kA = (SHAPE == 256 ? 2u : 1u) * kHalfA;  // bytes of a stage, this CTA
    static constexpr uint32_t kB = kTwo ? kBBytes / 2 : kBBytes;
    static constexpr uint32_t kBlock = kA + kB;
    static constexpr uint32_t kStage = kSub * kBlock;
    static_assert(kStages * kStage == kRingBytes, "one ring for every shape");
    static_assert(kStages <= 4 && kStages * kSub <= 6, "barriers");
};
constexpr int kFfnStages = 4, kFfnBlocks = 6;

struct FfnMaps {
    CUtensorMap a[3], b[3];
};

struct FfnGemm {
    // problems (kDw), whose tiles follow one another
    int64_t M[3], N[3], tiles_m[3], tiles_n[3], tile_end[3];
    int64_t K;      // of one segment
    // outputs: of the problems (kDx, kDown: one), or of one problem (kGateUp:
    // h, and s, a in fp32; kDact: dg, du); odd: its rows are not whole
    // 16-byte vectors
    void* out[3];
    int odd[3];
    float scale[3];  // kDact, kDw: of the products
    int segs;       // segments of K (kDx: 2)
    int width;      // accumulator columns of a tile
    int m_first;    // a problem's tiles run along M first
    int outs;       // kGateUp: 3 with s and a, else 1
    int act;
    const float* s;  // kDact: u act'(g), [M, N]
    const float* a;  // kDact: act(g), [M, N]
    const void* res;  // kDown: [M, N] or nullptr
    int res_vec;      // 1: its rows are whole 16-byte vectors
    DropSpec drop;    // kDown
    uint64_t timeout_ns;
    unsigned* status;
};

// The pair's forms of the copies, products and barriers: a copy that signals
// a barrier of the pair's first CTA, a product over both CTAs' operands and
// accumulators (issued by the first), a commit that arrives in both.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    const uint16_t both = 3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(both)
        : "memory");
}
__device__ __forceinline__ void pair_arrive(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}
__device__ __forceinline__ bool pair_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// tc_wait for a barrier that the other CTA of the pair arrives on
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    if (pair_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (pair_try_wait(bar, parity)) return true;
        if ((i & 1023u) == 0 && global_timer_ns() - t0 > timeout_ns) return false;
    }
}

template <uint32_t AB>
struct FfnType {
    using T = __nv_bfloat16;
};
template <>
struct FfnType<0u> {
    using T = __half;
};

constexpr int kFfnThreads = 320;  // producer, MMA issuer, 8 epilogue warps
constexpr int kFfnEpiWarps = 8;
// epilogue staging: two boxes of 32 x 32 16-bit elements a warp
constexpr uint32_t kFfnBox = 2048;
static_assert(kFfnEpiWarps * 2 * kFfnBox == kOutBytes, "the staging area of the GEMM");

// 32 columns of 16-bit elements from column n of row `row` of [M, N] (N a
// multiple of 8) as they are; zeros outside.
template <typename T>
__device__ __forceinline__ void load_row32(const void* p, int64_t row, int64_t n, int64_t M,
                                           int64_t N, uint4 (&w)[4]) {
    const T* q = static_cast<const T*>(p) + row * N + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row < M && n + 8 * j < N) w[j] = __ldg(reinterpret_cast<const uint4*>(q + 8 * j));
    }
}
__device__ __forceinline__ void ffn_prefetch(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
template <typename T>
__device__ __forceinline__ void unpack32(const uint4 (&w)[4], float (&f)[32]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float t[8];
        Vec<T>::unpack(w[j], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * j + i] = t[i];
    }
}
template <typename T>
__device__ __forceinline__ void pack32(const float (&f)[32], uint4 (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t[8] = {f[8 * j],     f[8 * j + 1], f[8 * j + 2], f[8 * j + 3],
                            f[8 * j + 4], f[8 * j + 5], f[8 * j + 6], f[8 * j + 7]};
        w[j] = Vec<T>::pack(t);
    }
}

// An epilogue warp's way out for boxes of 32 x 32 elements, which each lane
// holds a row of: through shared memory, conflict-free, to stores of whole
// 64- or 128-byte pieces of rows. (A TMA store of the box, whose read of the
// staging area waits behind the ring's loads in the copy engine, took 346
// instead of 327 us for kDact at 4096 x 12288 x 4096 and 496 instead of 483
// for kGateUp.)
struct FfnStore {
    uint32_t stage;  // 4 KB: a box of fp32, or two of 16 bits used in turn
    uint32_t boxes;  // so far
    int lane;

    // 16-bit boxes: 16-byte chunk j of row r at chunk j ^ (r / 2 mod 4)
    __device__ __forceinline__ uint32_t at(uint32_t buf, int r, int j) const {
        return buf + static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(j ^ ((r >> 1) & 3)) << 4);
    }
    // (a buffer's last reads lie before the barrier of the box between)
    __device__ __forceinline__ uint32_t put(const uint4 (&w)[4]) {
        const uint32_t buf = stage + (boxes & 1u) * kFfnBox;
        ++boxes;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(buf, lane, j)),
                         "r"(w[j].x), "r"(w[j].y), "r"(w[j].z), "r"(w[j].w)
                         : "memory");
        __syncwarp();
        return buf;
    }
    // the box at column n, row m of [M, cols], whose rows are whole 16-byte
    // vectors
    __device__ __forceinline__ void whole(void* out, int64_t n, int64_t m, int64_t M, int64_t cols,
                                          const uint4 (&w)[4]) {
        const uint32_t buf = put(w);
        const int r0 = lane >> 2, ch = lane & 3;
        uint16_t* to = static_cast<uint16_t*>(out) + (m + r0) * cols + n + 8 * ch;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + r0;
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(at(buf, r, ch)));
            if (m + r < M && n + 8 * ch < cols) *reinterpret_cast<uint4*>(to + 8 * j * cols) = v;
        }
    }
    // the same of rows that are not: a row an instruction
    __device__ __forceinline__ void odd(void* out, int64_t n, int64_t m, int64_t M, int64_t cols,
                                        const uint4 (&w)[4]) {
        const uint32_t buf = put(w);
        uint16_t* to = static_cast<uint16_t*>(out) + m * cols + n + lane;
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at(buf, r, lane >> 3) + 2u * (lane & 7)));
            if (m + r < M && n + lane < cols) to[r * cols] = v;
        }
    }

    // fp32 boxes: chunk j of row r at chunk j ^ (r mod 8). Piece i (of 8) of a
    // lane is 4 elements: row 4 i + lane / 8, chunk lane mod 8.
    __device__ __forceinline__ void put32(const float (&v)[32]) {
        __syncwarp();  // what was staged before has been read
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stage + static_cast<uint32_t>(lane) * 128u +
                             (static_cast<uint32_t>(j ^ (lane & 7)) << 4)),
                         "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                         : "memory");
        __syncwarp();
    }
    __device__ __forceinline__ int piece_row(int i) const { return 4 * i + (lane >> 3); }
    __device__ __forceinline__ float4 piece(int i) const {
        const int r = piece_row(i);
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(stage + static_cast<uint32_t>(r) * 128u +
                           (static_cast<uint32_t>((lane & 7) ^ (r & 7)) << 4)));
        return v;
    }
    // a box of fp32 at column n, row m of [M, cols], cols a multiple of 8
    __device__ __forceinline__ void whole32(void* out, int64_t n, int64_t m, int64_t M, int64_t cols,
                                            const float (&v)[32]) {
        put32(v);
        const int64_t c = n + 4 * (lane & 7);
        float* to = static_cast<float*>(out) + m * cols + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = piece_row(i);
            const float4 p = piece(i);
            if (m + r < M && c < cols) *reinterpret_cast<float4*>(to + r * cols) = p;
        }
        __syncwarp();
    }
};

// kDact: this lane's pieces of a box of fp32 (FfnStore); zeros outside.
__device__ __forceinline__ void load_pieces(const float* p, int64_t n, int64_t m, int64_t M, int64_t cols,
                                            int lane, float4 (&w)[8]) {
    const int64_t c = n + 4 * (lane & 7);
    const float* q = p + m * cols + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m + r < M && c < cols) w[i] = __ldg(reinterpret_cast<const float4*>(q + r * cols));
    }
}

// Whether element `i` is kept.
__device__ __noinline__ bool ffn_kept(const DropSpec& d, PhiloxKey key, uint64_t i) {
    const uint4 w = philox4x32(key, i >> 2);
    const uint32_t l = static_cast<uint32_t>(i) & 3u;
    return (l == 0 ? w.x : l == 1 ? w.y : l == 2 ? w.z : w.w) >= d.threshold;
}

// Dropout of 32 columns from column n of row `row` of y, and the residual.
template <typename T>
__device__ __forceinline__ void ffn_drop_res(const FfnGemm& a, const PhiloxKey& key, int64_t row,
                                             int64_t n, float (&v)[32]) {
    const int64_t M = a.M[0], N = a.N[0];
    if (a.drop.mode == kDropSome) {
        const uint64_t at = static_cast<uint64_t>(row * N + n);
        if ((N & 3) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) drop4(a.drop, key, at / 4 + j, v + 4 * j);
        } else {  // rows that start inside a block of four words
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = ffn_kept(a.drop, key, at + j) ? v[j] * a.drop.scale : 0.f;
        }
    } else if (a.drop.mode == kDropAll) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
    }
    if (a.res) {
        if (a.res_vec) {
            uint4 raw[4];
            load_row32<T>(a.res, row, n, M, N, raw);
            float w[32];
            unpack32<T>(raw, w);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += w[j];
        } else if (row < M) {
            const T* q = static_cast<const T*>(a.res) + row * N + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (n + j < N) v[j] += Vec<T>::load1(q, j);
        }
    }
}

// The problem of tile t, and t within it.
__device__ __forceinline__ int ffn_problem(const FfnGemm& a, int64_t* t) {
    if (*t < a.tile_end[0]) return 0;
    const int p = *t < a.tile_end[1] ? 1 : 2;
    *t -= a.tile_end[p - 1];
    return p;
}
__device__ __forceinline__ int64_t ffn_tile_m(const FfnGemm& a, int p, int64_t t) {
    return a.m_first ? t % a.tiles_m[p] : t / a.tiles_n[p];
}
__device__ __forceinline__ int64_t ffn_tile_n(const FfnGemm& a, int p, int64_t t) {
    return a.m_first ? t / a.tiles_m[p] : t % a.tiles_n[p];
}

template <uint32_t AB, int MODE, int SHAPE>
__global__ void __launch_bounds__(kFfnThreads, 1)
ffn_gemm(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnGemm a) {
    using T = typename FfnType<AB>::T;
    using TT = FfnTile<SHAPE>;
    constexpr bool PAIR = TT::kTwo;
    constexpr bool A_MN = MODE == kDw;
    constexpr bool B_MN = MODE == kDact || MODE == kDx || MODE == kDw;
    // pairs' tiles may be narrower (a.width) where B is K-major
    constexpr bool NARROW = PAIR && !B_MN;
    const int width = NARROW ? a.width : kBN;
    const int cols = MODE == kGateUp ? width / 2 : width;  // output columns of a tile
    constexpr int BM = TT::kRows;
    constexpr int kStages = TT::kStages;
    constexpr int NACC = TT::kAccBufs;
    constexpr int H = TT::kHalves;
    extern __shared__ unsigned char ffn_smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kFfnStages];    // of a stage
    __shared__ __align__(8) uint64_t empty_bar[kFfnBlocks];  // of a K block
    __shared__ __align__(8) uint64_t acc_full[2];
    __shared__ __align__(8) uint64_t acc_empty[2];
    __shared__ __align__(8) uint64_t done_bar;  // every MMA of the CTA completed
    __shared__ uint32_t tmem_base_sh;
    __shared__ uint32_t s_issued[kFfnStages];  // 0, or 2 + parity of the last copy into the stage
    __shared__ int s_fail;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // a pair's CTAs work on the same tiles; the first issues the products
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int64_t tile0 = PAIR ? blockIdx.x / 2 : blockIdx.x;
    const int64_t tile_step = PAIR ? gridDim.x / 2 : gridDim.x;
    const uint32_t smem0 = (smem_u32(ffn_smem_raw) + 1023u) & ~1023u;  // 1024-byte aligned
    constexpr int kSub = TT::kSub;
    // stages of a segment (behind K the copies fill zeros)
    const int nk = static_cast<int>((a.K + kSub * kBK - 1) / (kSub * kBK));
    const int64_t ntiles = a.tile_end[2];

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            s_issued[s] = 0;
        }
        for (int s = 0; s < kStages * TT::kSub; ++s) mbar_init(smem_u32(&empty_bar[s]), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), (PAIR ? 2 : 1) * kFfnEpiWarps);
        }
        mbar_init(smem_u32(&done_bar), 1);
        s_fail = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile(
                "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                    smem_u32(&tmem_base_sh)),
                "r"(kTmemCols)
                : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile(
                "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                    smem_u32(&tmem_base_sh)),
                "r"(kTmemCols)
                : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // both CTAs' barriers and tensor memory
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer: every K block of every tile of this CTA
            const auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
                if constexpr (PAIR) pair_load_2d(dst, map, x, y, bar);
                else tma_load_2d(dst, map, x, y, bar);
            };
            const uint32_t bytes = NARROW ? kSub * (2u * TT::kA + static_cast<uint32_t>(width) * kBK * 2u)
                                          : (PAIR ? 2u : 1u) * TT::kStage;
            int s = 0;
            uint32_t ph = 0;
            bool fail = false;
            for (int64_t t = tile0; t < ntiles && !fail; t += tile_step) {
                int64_t tl = t;
                const int p = ffn_problem(a, &tl);
                // this CTA's rows of A, and its columns of B
                const int m0 = static_cast<int>(ffn_tile_m(a, p, tl) * BM + rank * kMmaM);
                const int nt = static_cast<int>(ffn_tile_n(a, p, tl) * cols);
                const int n0 = MODE == kGateUp ? nt : nt + static_cast<int>(rank) * (width / 2);
                for (int kb = 0; kb < nk * a.segs; ++kb) {
                    // the pair's copies signal its first CTA's barrier, which
                    // expects the bytes of both
                    uint32_t fb = smem_u32(&full_bar[s]);
                    if constexpr (PAIR) fb = map_to_rank(fb, 0);
                    // the operands' maps: of the problem, or of the segment
                    const int seg = kb >= nk ? 1 : 0;
                    const int i = MODE == kDx ? seg : p;
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub) {
                        if (!tc_wait(smem_u32(&empty_bar[s * kSub + sub]), ph ^ 1u, a.timeout_ns)) {
                            fail = true;
                            break;
                        }
                        if (sub == 0) {
                            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), bytes);
                            s_issued[s] = 2u + ph;
                        }
                        const int k0 = ((kb - seg * nk) * kSub + sub) * kBK;
                        const uint32_t sa = smem0 + static_cast<uint32_t>(s) * TT::kStage + sub * TT::kBlock;
                        if constexpr (A_MN) {
                            for (uint32_t j = 0; j < TT::kA / kMnBox; ++j)
                                load(sa + j * kMnBox, &maps.a[i], m0 + 64 * j, k0, fb);
                        } else {
                            load(sa, &maps.a[i], k0, m0, fb);
                        }
                        const uint32_t sb = sa + TT::kA;
                        if constexpr (MODE == kGateUp) {
                            if constexpr (PAIR) {
                                load(sb, &maps.b[rank], k0, n0, fb);
                            } else {
                                load(sb, &maps.b[0], k0, n0, fb);
                                load(sb + kBBytes / 2, &maps.b[1], k0, n0, fb);
                            }
                        } else if constexpr (B_MN) {
                            for (uint32_t j = 0; j < TT::kB / kMnBox; ++j)
                                load(sb + j * kMnBox, &maps.b[i], n0 + 64 * j, k0, fb);
                        } else {
                            load(sb, &maps.b[i], k0, n0, fb);
                        }
                    }
                    if (fail) break;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (fail) s_fail = 1;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---- MMA issuer: tile i into accumulator buffer i mod NACC
            const auto commit = [](uint32_t bar) {
                if constexpr (PAIR) pair_commit(bar);
                else tc_commit(bar);
            };
            const uint32_t idesc =
                (tc_idesc(AB, A_MN ? 1u : 0u, B_MN ? 1u : 0u) & ~(31u << 24) & ~(63u << 17)) |
                (static_cast<uint32_t>((PAIR ? 256 : 128) >> 4) << 24) |
                (static_cast<uint32_t>(width >> 3) << 17);
            // the operands' descriptors at the ring's start, whose address field
            // counts 16-byte units
            const uint64_t a0 = A_MN ? tc_smem_desc_mn(smem0) : tc_smem_desc(smem0);
            const uint64_t b0 = B_MN ? tc_smem_desc_mn(smem0 + TT::kA) : tc_smem_desc(smem0 + TT::kA);
            int s = 0;
            uint32_t ph = 0;
            int i = 0;  // tiles of this CTA so far
            bool fail = false;
            for (int64_t t = tile0; t < ntiles && !fail; t += tile_step, ++i) {
                const int b = i % NACC;
                // the epilogue has drained this buffer's previous tile
                const uint32_t drained = (static_cast<uint32_t>(i / NACC) & 1u) ^ 1u;
                if (!(PAIR ? pair_wait(smem_u32(&acc_empty[b]), drained, a.timeout_ns)
                           : tc_wait(smem_u32(&acc_empty[b]), drained, a.timeout_ns))) {
                    fail = true;
                    break;
                }
                tc_fence_after();
                // half h of the tile (rows 128 h ...) in columns (b H + h) 256
                const uint32_t acc = tmem + static_cast<uint32_t>(b * H * kBN);
                for (int kb = 0; kb < nk * a.segs; ++kb) {
                    if (!tc_wait(smem_u32(&full_bar[s]), ph, a.timeout_ns)) {
                        fail = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = static_cast<uint32_t>(s) * (TT::kStage >> 4);
#pragma unroll
                    for (int kk = 0; kk < kSub * (kBK / 16); ++kk) {
                        constexpr uint32_t kPer = kBK / 16;
                        const uint32_t block = (kk / kPer) * (TT::kBlock >> 4), k = kk % kPer;
                        // a K step of 16 further in 16-byte units
                        const uint64_t db = b0 + (at + block + k * (B_MN ? 2048u >> 4 : 32u >> 4));
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const uint64_t da = a0 + (at + block + k * (A_MN ? 2048u >> 4 : 32u >> 4) +
                                                      static_cast<uint32_t>(h) * (kHalfA >> 4));
                            const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
                            if constexpr (PAIR) pair_mma(acc, da, db, idesc, add);
                            else tc_mma(acc + static_cast<uint32_t>(h * kBN), da, db, idesc, add);
                        }
                        if (k == kPer - 1) commit(smem_u32(&empty_bar[s * kSub + kk / kPer]));
                    }
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                // every MMA of the tile issued: the epilogue may read it once
                // they complete (also after a failure, so that nothing waits)
                commit(smem_u32(&acc_full[b]));
            }
            if (fail) s_fail = 1;
            commit(smem_u32(&done_bar));  // after every MMA this thread issued
        }
    } else {
        // ---- epilogue: warp w reads accumulator lanes 32 (w mod 4) of each
        // 128-row half of the tile; of its columns warps 2-5 take the first
        // half (rounded up to whole units of 32), warps 6-9 the rest
        const int q = warp & 3, side = (warp - 2) >> 2;
        FfnStore store{smem0 + kRingBytes + static_cast<uint32_t>(warp - 2) * 2u * kFfnBox, 0u, lane};
        PhiloxKey key{};
        if constexpr (MODE == kDown) key = philox_key(a.drop);
        int i = 0;
        for (int64_t t = tile0; t < ntiles; t += tile_step, ++i) {
            const int b = i % NACC;
            int64_t tl = t;
            const int p = ffn_problem(a, &tl);
            const int64_t M = a.M[p], N = a.N[p];
            const int first = (cols / 32 + 1) / 2;  // units of the first half
            const int units = side ? cols / 32 - first : first;
            const int64_t n0 = ffn_tile_n(a, p, tl) * cols + side * first * 32;
            const int64_t mt = ffn_tile_m(a, p, tl) * BM + rank * kMmaM + q * 32;  // + 128 hh
            float4 ps[8], pa[8];  // kDact: pieces of s and a of the next unit
            if constexpr (MODE == kDact) {
                // while the tile's products run: the others into L2, the first here
                for (int hh = 0; hh < H; ++hh) {
                    const int64_t row = mt + hh * kMmaM + lane;
                    for (int c = 0; c < 32 * units; c += 32) {
                        if (row >= M || n0 + c >= N) break;
                        ffn_prefetch(a.s + row * N + n0 + c);
                        ffn_prefetch(a.a + row * N + n0 + c);
                    }
                }
                load_pieces(a.s, n0, mt, M, N, lane, ps);
                load_pieces(a.a, n0, mt, M, N, lane, pa);
            }
            const bool ok = mbar_wait_bounded(smem_u32(&acc_full[b]),
                                              static_cast<uint32_t>(i / NACC) & 1u, a.timeout_ns);
            // (the whole warp goes on or none of it: what follows takes all lanes)
            if (__any_sync(~0u, !ok || *reinterpret_cast<volatile int*>(&s_fail))) {
                if (lane == 0) s_fail = 1;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < H * units; ++x) {
                const int hh = H == 1 ? 0 : x / units, c = x - hh * units;
                const int64_t m = mt + hh * kMmaM, n = n0 + c * 32;
                // the accumulator's column of this unit
                const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                                     static_cast<uint32_t>((b * H + hh) * kBN + (side * first + c) * 32);
                // the unit after this one
                const int y = x + 1 < H * units ? x + 1 : x, yh = H == 1 ? 0 : y / units;
                const int64_t nm = mt + yh * kMmaM, nn = n0 + (y - yh * units) * 32;
                if (m >= M || n >= N) {  // the same for the whole warp
                    if constexpr (MODE == kDact) {
                        load_pieces(a.s, nn, nm, M, N, lane, ps);
                        load_pieces(a.a, nn, nm, M, N, lane, pa);
                    }
                    continue;
                }
                float v[32];
                tc_ld32(acc, v);
                uint4 w[4];
                if constexpr (MODE == kGateUp) {
                    float u[32];
                    tc_ld32(acc + static_cast<uint32_t>(width / 2), u);
                    if (a.outs == 1) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = ffn_gate<false>(a.act, v[j]).act * u[j];
                        pack32<T>(v, w);
                        store.whole(a.out[0], n, m, M, N, w);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float fh[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const FfnGate r = ffn_gate<true>(a.act, v[8 * j + e]);
                                fh[e] = r.act * u[8 * j + e];
                                u[8 * j + e] *= r.slope;  // s
                                v[8 * j + e] = r.act;     // a
                            }
                            w[j] = Vec<T>::pack(fh);
                        }
                        store.whole(a.out[0], n, m, M, N, w);
                        store.whole32(a.out[1], n, m, M, N, u);
                        store.whole32(a.out[2], n, m, M, N, v);
                    }
                } else if constexpr (MODE == kDact) {
                    store.put32(v);
                    const int64_t col = n + 4 * (lane & 7);
                    T* dg = static_cast<T*>(a.out[0]) + m * N + col;
                    T* du = static_cast<T*>(a.out[1]) + m * N + col;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = store.piece_row(i);
                        float4 d = store.piece(i);
                        d.x *= a.scale[0];
                        d.y *= a.scale[0];
                        d.z *= a.scale[0];
                        d.w *= a.scale[0];
                        if (m + r < M && col < N) {
                            const float f[8] = {d.x * ps[i].x, d.y * ps[i].y, d.z * ps[i].z, d.w * ps[i].w,
                                                d.x * pa[i].x, d.y * pa[i].y, d.z * pa[i].z, d.w * pa[i].w};
                            const uint4 o = Vec<T>::pack(f);
                            *reinterpret_cast<uint2*>(dg + r * N) = make_uint2(o.x, o.y);
                            *reinterpret_cast<uint2*>(du + r * N) = make_uint2(o.z, o.w);
                        }
                    }
                    load_pieces(a.s, nn, nm, M, N, lane, ps);
                    load_pieces(a.a, nn, nm, M, N, lane, pa);
                } else {
                    if constexpr (MODE == kDw) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= a.scale[p];
                    }
                    if constexpr (MODE == kDown) ffn_drop_res<T>(a, key, m + lane, n, v);
                    pack32<T>(v, w);
                    const int pi = MODE == kDw ? p : 0;
                    if (a.odd[pi]) store.odd(a.out[pi], n, m, M, N, w);
                    else store.whole(a.out[pi], n, m, M, N, w);
                }
            }
            // the warp's loads of the accumulator are done
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) pair_arrive(map_to_rank(smem_u32(&acc_empty[b]), 0));
                else mbar_arrive(smem_u32(&acc_empty[b]));
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // every MMA completes before the tensor memory is freed
        const bool done = mbar_wait_bounded(smem_u32(&done_bar), 0u, a.timeout_ns);
        if (s_fail || !done) {
            atomicOr(a.status, kDevErrTimeout);
            // copies still in flight land before the shared memory is released
            // (a pair's are counted by its first CTA)
            if (rank == 0)
                for (int s = 0; s < kStages; ++s)
                    if (s_issued[s])
                        (void)mbar_wait_bounded(smem_u32(&full_bar[s]), s_issued[s] & 1u,
                                                a.timeout_ns);
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) {
        cluster_sync();  // neither CTA leaves while the other may still use its memory
        if (warp == 1)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kTmemCols)
                         : "memory");
    } else if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

// Packs matrices [rows, cols] into rows of `pitch` elements (a multiple of 8,
// zeros behind the columns); `mask`: elements that the dropout drops are
// zeros too. A thread an output vector of 8 elements.
constexpr int kPackMats = 5;
struct PackArgs {
    struct {
        const void* src;
        void* dst;
        int64_t rows, cols, pitch;
        int64_t end;  // vectors of this matrix and those before it
        int vec;      // 1: the source's rows are whole 16-byte vectors
        int mask;
    } m[kPackMats];
    int n;
    DropSpec drop;
};

template <typename T>
__global__ void __launch_bounds__(256) ffn_pack(const __grid_constant__ PackArgs a) {
    const PhiloxKey key = philox_key(a.drop);
    const int64_t all = a.m[a.n - 1].end;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        int k = 0;
        while (i >= a.m[k].end) ++k;
        const auto& m = a.m[k];
        const int64_t v = i - (k ? a.m[k - 1].end : 0);
        const int64_t r = v / (m.pitch / 8), c = (v - r * (m.pitch / 8)) * 8;
        const T* src = static_cast<const T*>(m.src) + r * m.cols + c;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (m.vec) {
            w = *reinterpret_cast<const uint4*>(src);
            Vec<T>::unpack(w, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < m.cols) f[j] = Vec<T>::load1(src, j);
        }
        if (m.mask && a.drop.mode != kDropNone) {
            const uint64_t at = static_cast<uint64_t>(r * m.cols + c);
            if (a.drop.mode == kDropAll) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = 0.f;
            } else if ((m.cols & 3) == 0) {
                DropSpec d = a.drop;
                d.scale = 1.f;
                drop4(d, key, at / 4, f);
                drop4(d, key, at / 4 + 1, f + 4);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = ffn_kept(a.drop, key, at + j) ? f[j] : 0.f;
            }
        }
        // (16-bit values pass through fp32 unchanged)
        reinterpret_cast<uint4*>(m.dst)[v] = Vec<T>::pack(f);
    }
}

template <uint32_t AB, int MODE>
const void* ffn_fn(int shape) {
    if constexpr (MODE == kDx || MODE == kDw)
        if (shape == 256) return (const void*)&ffn_gemm<AB, MODE, 256>;
    return shape == kPair ? (const void*)&ffn_gemm<AB, MODE, kPair> : (const void*)&ffn_gemm<AB, MODE, 128>;
}
const void* ffn_fn(int dtype, int mode, int shape) {
    const bool bf = dtype == CE_BF16;
    switch (mode) {
    case kGateUp: return bf ? ffn_fn<1u, kGateUp>(shape) : ffn_fn<0u, kGateUp>(shape);
    case kDown: return bf ? ffn_fn<1u, kDown>(shape) : ffn_fn<0u, kDown>(shape);
    case kDact: return bf ? ffn_fn<1u, kDact>(shape) : ffn_fn<0u, kDact>(shape);
    case kDx: return bf ? ffn_fn<1u, kDx>(shape) : ffn_fn<0u, kDx>(shape);
    default: return bf ? ffn_fn<1u, kDw>(shape) : ffn_fn<0u, kDw>(shape);
    }
}

// A call's device, its status word and its wait limit.
struct FfnDevice {
    int sms;
    unsigned* status;
    uint64_t timeout_ns;
};

ce_status ffn_device(cudaStream_t st, FfnDevice* d) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    // makes the device's context this thread's (an autograd thread has none
    // yet), which encoding a tensor map needs
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return record_cuda_failure(e, "feed-forward device");
    d->sms = std::max(d->sms, 1);
    const char* env = std::getenv("GBCE_WAIT_TIMEOUT_MS");
    d->timeout_ns = ((env && *env) ? static_cast<uint64_t>(std::atoll(env)) : 2000ull) * 1000000ull;
    return library_status_word(st, &d->status);
}

// An operand of a launch: a row-major [outer, inner] matrix, as A or B.
struct FfnMatrix {
    const void* p;
    int64_t outer, inner;
};

// The tile shape of a launch of form `mode` with problems of M x N, by its
// rounds of tiles over the SMs (or pairs of SMs) and what a round was measured
// to take, that of pairs being 100 (per 4096 of K, bf16: 20.5 us). 256 rows an
// SM: 195 (4096 x 4096 x 24576 475 against 482 us for pairs, 4096 x 2048 x
// 16384 156 against 167). Where the epilogue, which that shape does not
// overlap, does more than store, its round takes 215 (4096 x 12288 x 4096 549
// against 472 us, 2048 x 4096 x 12288 136 against 130), more than two of pairs:
// only dx and the weight gradients have it. 128 rows: 115 (4096 x 4096 x 12288
// 300 against 256 us; 300 rows of the block of 4096 x 12288 117 against 135).
// Narrower tiles
// of pairs save little of a round, but a product of few tiles finds more SMs
// with them: 224 columns 95, 192 columns 91 (512 rows of 1024 x 4096 40
// against 48 us, of 4096 x 12288 131 against 137).
struct FfnForm {
    int shape, width;
    int64_t tiles;
};
FfnForm ffn_form(int mode, const int64_t* M, const int64_t* N, int problems, int sms) {
    const bool bare = mode == kDx || mode == kDw;
    const struct {
        int shape, width;
        int64_t round;
        bool taken;
    } forms[] = {{kPair, 256, 100, true},
                 {256, 256, 195, bare},
                 {128, 256, 115, true},
                 {kPair, 192, 91, mode == kDown || mode == kGateUp},
                 // (kGateUp: half the columns are whole units of 32 of the epilogue's)
                 {kPair, 224, 95, mode == kDown}};
    FfnForm best = {kPair, kBN, 0};
    int64_t least = INT64_MAX;
    for (const auto& f : forms) {
        if (!f.taken) continue;
        const int64_t rows = f.shape == 128 ? 128 : 256;
        const int64_t across = mode == kGateUp ? f.width / 2 : f.width;
        const int64_t ctas = f.shape == kPair ? std::max(sms / 2, 1) : sms;
        int64_t tiles = 0;
        for (int p = 0; p < problems; ++p)
            tiles += (M[p] + rows - 1) / rows * ((N[p] + across - 1) / across);
        const int64_t cost = (tiles + ctas - 1) / ctas * f.round;
        if (cost < least) {
            least = cost;
            best = FfnForm{f.shape, f.width, tiles};
        }
    }
    return best;
}

// One launch of form `mode`: problems or segments A[i] x B[i].
ce_status ffn_launch(int mode, int dtype, FfnGemm g, int problems, const FfnMatrix (&A)[3],
                     const FfnMatrix (&B)[3], const FfnDevice& d, cudaStream_t st) {
    g.timeout_ns = d.timeout_ns;
    g.status = d.status;
    const FfnForm form = ffn_form(mode, g.M, g.N, problems, d.sms);
    const int shape = form.shape;
    g.width = form.width;
    const int64_t cols = mode == kGateUp ? g.width / 2 : g.width;
    const int bm = shape == 128 ? 128 : 256;
    int64_t end = 0;
    for (int p = 0; p < 3; ++p) {
        if (p < problems) {
            g.tiles_m[p] = (g.M[p] + bm - 1) / bm;
            g.tiles_n[p] = (g.N[p] + cols - 1) / cols;
            end += g.tiles_m[p] * g.tiles_n[p];
        }
        g.tile_end[p] = end;
    }
    // consecutive tiles share a tile of the larger operand
    g.m_first = g.N[0] >= g.M[0] ? 1 : 0;
    FfnMaps maps = {};
    const bool a_mn = mode == kDw, b_mn = mode == kDact || mode == kDx || mode == kDw;
    for (int i = 0; i < 3; ++i) {
        ce_status rc = CE_OK;
        if (A[i].p) rc = tc_map_16bit(&maps.a[i], A[i].p, dtype, A[i].outer, A[i].inner,
                                     a_mn ? 64 : shape == kPair ? 128 : bm);
        if (rc == CE_OK && B[i].p)
            rc = tc_map_16bit(&maps.b[i], B[i].p, dtype, B[i].outer, B[i].inner,
                              b_mn ? 64 : mode == kGateUp || shape == kPair ? g.width / 2 : kBN);
        if (rc != CE_OK) return rc;
    }
    const void* fn = ffn_fn(dtype, mode, shape);
    const ce_status rc = tc_smem_limit(fn, kTcSmem);
    if (rc != CE_OK) return rc;
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    if (shape == kPair) {
        lc.gridDim = dim3(2u * static_cast<unsigned>(std::min<int64_t>(end, std::max(d.sms / 2, 1))));
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        lc.attrs = &attr;
        lc.numAttrs = 1;
    } else {
        lc.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(end, d.sms)));
    }
    lc.blockDim = dim3(kFfnThreads);
    lc.dynamicSmemBytes = kTcSmem;
    lc.stream = st;
    void* args[] = {&maps, &g};
    const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "feed-forward launch");
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

ce_status check_ffn(int dtype, int64_t rows, int64_t H, int64_t I, int64_t O, int act) {
    if (dtype != CE_BF16 && dtype != CE_F16) return dtype == CE_F32 ? CE_ERR_UNSUPPORTED : CE_ERR_INVALID_ARG;
    if (rows < 0 || H <= 0 || I <= 0 || O <= 0) return CE_ERR_INVALID_ARG;
    if (act < CE_ACT_SILU || act > CE_ACT_GELU_TANH) return CE_ERR_INVALID_ARG;
    constexpr int64_t kMost = INT32_MAX - 512;  // tile coordinates are 32-bit
    if (rows > kMost || H > kMost || I > kMost || O > kMost) {
        record_message("the feed-forward block takes rows, H, I and O below 2^31 - 512");
        return CE_ERR_UNSUPPORTED;
    }
    return CE_OK;
}

// Hands out a caller's workspace, and collects the matrices that one launch
// of ffn_pack fills there.
struct FfnPacker {
    char* ws;
    PackArgs args = {};

    void* take(int64_t rows, int64_t cols) {
        void* p = ws;
        ws += up256(rows * up8(cols) * 2);
        return p;
    }
    // `src` itself where the TMA can read it, else its packed copy
    const void* operand(const void* src, int64_t rows, int64_t cols, bool mask = false) {
        const bool whole = cols % 8 == 0 && aligned(src);
        if (whole && !mask) return src;
        void* dst = take(rows, cols);
        auto& m = args.m[args.n];
        m.src = src;
        m.dst = dst;
        m.rows = rows;
        m.cols = cols;
        m.pitch = up8(cols);
        m.end = (args.n ? args.m[args.n - 1].end : 0) + rows * (m.pitch / 8);
        m.vec = whole ? 1 : 0;
        m.mask = mask ? 1 : 0;
        ++args.n;
        return dst;
    }
    ce_status run(int dtype, const DropSpec& drop, const FfnDevice& d, cudaStream_t st) {
        if (!args.n) return CE_OK;
        args.drop = drop;
        const int64_t grid = std::min<int64_t>((args.m[args.n - 1].end + 255) / 256, 16L * d.sms);
        void* p[] = {&args};
        const void* fn = dtype == CE_BF16 ? (const void*)&ffn_pack<__nv_bfloat16>
                                          : (const void*)&ffn_pack<__half>;
        const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(256), p, 0, st);
        return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "feed-forward pack launch");
    }
};

// The most rows that take the form for few rows, whose products have at most
// 256 columns. Measured, bf16, forward with residual: H 4096, I 12288: 1 row
// 59 against 109 us for the tiles, 64 rows 68 / 97, 256 rows 91 / 103; H
// 1024, I 4096: 13 / 37, 16 / 37 and 26 / 38.
constexpr int64_t kFewRows = 256;

// Output i of a launch, with rows of `cols` elements.
void ffn_output(FfnGemm* g, int i, void* p, int64_t cols) {
    g->out[i] = p;
    g->odd[i] = cols % 8 == 0 && aligned(p) ? 0 : 1;
}

// What a packed copy of [rows, cols] takes; 0 where the TMA reads the
// original, if its base is aligned.
int64_t pack_bytes(int64_t rows, int64_t cols) { return up256(rows * up8(cols) * 2); }

}  // namespace
}  // namespace gbce

using namespace gbce;

extern "C" size_t ce_ffn_fwd_workspace_bytes(int64_t rows, int64_t H, int64_t I, int64_t O) {
    if (rows < 0 || H <= 0 || I <= 0 || O <= 0) return 0;
    const int64_t x = H % 8 ? pack_bytes(rows, H) + 2 * pack_bytes(I, H) : 0;
    const int64_t packed = x + (I % 8 ? pack_bytes(O, I) : 0);
    int dev = 0, sms = 0;
    if (rows > kFewRows || cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return static_cast<size_t>(packed);
    return static_cast<size_t>(packed + ffn_rows_workspace(rows, up8(H), up8(I), O, std::max(sms, 1)));
}

extern "C" ce_status ce_ffn_fwd(const void* x, const void* w_gate, const void* w_up,
                                const void* w_down, const void* residual, int dtype, int64_t rows,
                                int64_t H, int64_t I, int64_t O, int act, double p, uint64_t seed,
                                uint64_t offset, const int64_t* state, void* y, void* h, float* s,
                                float* a, void* workspace, size_t workspace_bytes,
                                ce_stream_t stream) {
    ce_status rc = check_ffn(dtype, rows, H, I, O, act);
    if (rc != CE_OK) return rc;
    FfnGemm base = {};
    if (!drop_spec(p, seed, offset, state, &base.drop)) return CE_ERR_INVALID_ARG;
    if (!w_gate || !w_up || !w_down || (s == nullptr) != (a == nullptr)) return CE_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y || !h)) return CE_ERR_INVALID_ARG;
    if (!aligned(h) || !aligned(s) || !aligned(a)) return CE_ERR_INVALID_ARG;
    for (const void* q : {x, w_gate, w_up, w_down})
        if (reinterpret_cast<uintptr_t>(q) & 1u) return CE_ERR_INVALID_ARG;
    if ((H % 8 == 0 && !(aligned(x) && aligned(w_gate) && aligned(w_up))) ||
        (I % 8 == 0 && !aligned(w_down))) {
        record_message("rows of whole 16-byte vectors need a 16-byte aligned base");
        return CE_ERR_UNSUPPORTED;
    }
    const size_t need = ce_ffn_fwd_workspace_bytes(rows, H, I, O);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need))
        return CE_ERR_INVALID_ARG;
    if (rows == 0) return CE_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    FfnDevice d;
    rc = ffn_device(st, &d);
    if (rc != CE_OK) return rc;
    const int64_t H8 = up8(H), I8 = up8(I);
    FfnPacker pack{static_cast<char*>(workspace)};
    x = pack.operand(x, rows, H);
    w_gate = pack.operand(w_gate, I, H);
    w_up = pack.operand(w_up, I, H);
    w_down = pack.operand(w_down, O, I);
    rc = pack.run(dtype, base.drop, d, st);
    if (rc != CE_OK) return rc;
    if (rows <= kFewRows)
        return ffn_rows_fwd(x, w_gate, w_up, w_down, residual, dtype, rows, H8, I, I8, O, act,
                            base.drop, y, h, s, a, pack.ws, d.sms, d.timeout_ns, d.status, st);
    base.segs = 1;
    base.act = act;
    FfnGemm up = base;
    up.M[0] = rows;
    up.N[0] = I8;
    up.K = H8;
    up.outs = s ? 3 : 1;
    up.out[0] = h;
    up.out[1] = s;
    up.out[2] = a;
    rc = ffn_launch(kGateUp, dtype, up, 1, {{x, rows, H8}}, {{w_gate, I, H8}, {w_up, I, H8}}, d, st);
    if (rc != CE_OK) return rc;
    FfnGemm down = base;
    down.M[0] = rows;
    down.N[0] = O;
    down.K = I8;
    down.res = residual;
    down.res_vec = O % 8 == 0 && aligned(residual) ? 1 : 0;
    ffn_output(&down, 0, y, O);
    return ffn_launch(kDown, dtype, down, 1, {{h, rows, I8}}, {{w_down, O, I8}}, d, st);
}

extern "C" ce_status ce_ffn_tiles(int product, int64_t rows, int64_t H, int64_t I, int64_t O, int sms,
                                  int64_t* tile) {
    if (product < kGateUp || product > kDw || sms < 1 || !tile) return CE_ERR_INVALID_ARG;
    const ce_status rc = check_ffn(CE_BF16, rows, H, I, O, CE_ACT_SILU);
    if (rc != CE_OK) return rc;
    const int64_t I8 = up8(I);
    const int64_t n[] = {I8, O, I8, H};
    const bool dw = product == kDw;
    const int64_t M[3] = {dw ? I : rows, I, O}, N[3] = {dw ? H : n[product], H, I};
    const FfnForm f = ffn_form(product, M, N, dw ? 3 : 1, sms);
    tile[0] = f.shape == 128 ? 128 : 256;
    tile[1] = product == kGateUp ? f.width / 2 : f.width;
    tile[2] = f.shape == kPair ? 2 : 1;
    tile[3] = f.tiles;
    return CE_OK;
}

extern "C" size_t ce_ffn_bwd_workspace_bytes(int64_t rows, int64_t H, int64_t I, int64_t O, double p) {
    if (rows < 0 || H <= 0 || I <= 0 || O <= 0) return 0;
    const int64_t x = H % 8 ? pack_bytes(rows, H) + 2 * pack_bytes(I, H) : 0;
    const int64_t wd = I % 8 ? pack_bytes(O, I) : 0;
    const int64_t dz = O % 8 || p > 0.0 ? pack_bytes(rows, O) : 0;
    return static_cast<size_t>(2 * pack_bytes(rows, I) + x + wd + dz);
}

extern "C" ce_status ce_ffn_bwd(const void* dy, const void* x, const void* w_gate,
                                const void* w_up, const void* w_down, const void* h,
                                const float* s, const float* a, int dtype, int64_t rows, int64_t H,
                                int64_t I, int64_t O, int act, double p, uint64_t seed,
                                uint64_t offset, const int64_t* state, void* dx, void* dw_gate,
                                void* dw_up, void* dw_down, void* workspace,
                                size_t workspace_bytes, ce_stream_t stream) {
    ce_status rc = check_ffn(dtype, rows, H, I, O, act);
    if (rc != CE_OK) return rc;
    FfnGemm base = {};
    if (!drop_spec(p, seed, offset, state, &base.drop)) return CE_ERR_INVALID_ARG;
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return CE_ERR_INVALID_ARG;
    if (!w_gate || !w_up || !w_down) return CE_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !h || !s || !a)) return CE_ERR_INVALID_ARG;
    if (!aligned(h) || !aligned(s) || !aligned(a)) return CE_ERR_INVALID_ARG;
    for (const void* q : {dy, x, w_gate, w_up, w_down})
        if (reinterpret_cast<uintptr_t>(q) & 1u) return CE_ERR_INVALID_ARG;
    if ((H % 8 == 0 && !(aligned(x) && aligned(w_gate) && aligned(w_up))) ||
        (I % 8 == 0 && !aligned(w_down)) || (O % 8 == 0 && !aligned(dy))) {
        record_message("rows of whole 16-byte vectors need a 16-byte aligned base");
        return CE_ERR_UNSUPPORTED;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: zero gradients of the weights
        cudaError_t e = cudaSuccess;
        if (dw_gate) e = cudaMemsetAsync(dw_gate, 0, static_cast<size_t>(I * H * 2), st);
        if (e == cudaSuccess && dw_up) e = cudaMemsetAsync(dw_up, 0, static_cast<size_t>(I * H * 2), st);
        if (e == cudaSuccess && dw_down)
            e = cudaMemsetAsync(dw_down, 0, static_cast<size_t>(O * I * 2), st);
        return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "cudaMemsetAsync(weight gradients)");
    }
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < ce_ffn_bwd_workspace_bytes(rows, H, I, O, p))
        return CE_ERR_INVALID_ARG;
    if (!dx && !dw_gate && !dw_down) return CE_OK;
    FfnDevice d;
    rc = ffn_device(st, &d);
    if (rc != CE_OK) return rc;
    const int64_t H8 = up8(H), I8 = up8(I), O8 = up8(O);
    FfnPacker pack{static_cast<char*>(workspace)};
    void* dg = pack.take(rows, I);
    void* du = pack.take(rows, I);
    const void* dz = pack.operand(dy, rows, O, base.drop.mode != kDropNone);
    const float scale = base.drop.mode == kDropNone ? 1.f : base.drop.scale;
    if (dx || dw_gate) w_down = pack.operand(w_down, O, I);
    if (dw_gate) x = pack.operand(x, rows, H);
    if (dx) {
        w_gate = pack.operand(w_gate, I, H);
        w_up = pack.operand(w_up, I, H);
    }
    rc = pack.run(dtype, base.drop, d, st);
    if (rc != CE_OK) return rc;
    base.segs = 1;
    base.act = act;
    if (dx || dw_gate) {
        FfnGemm t = base;
        t.M[0] = rows;
        t.N[0] = I8;
        t.K = O8;
        t.s = s;
        t.a = a;
        t.scale[0] = scale;
        t.out[0] = dg;
        t.out[1] = du;
        rc = ffn_launch(kDact, dtype, t, 1, {{dz, rows, O8}}, {{w_down, O, I8}}, d, st);
        if (rc != CE_OK) return rc;
    }
    if (dx) {
        FfnGemm t = base;
        t.M[0] = rows;
        t.N[0] = H;
        t.K = I8;
        t.segs = 2;
        ffn_output(&t, 0, dx, H);
        rc = ffn_launch(kDx, dtype, t, 1, {{dg, rows, I8}, {du, rows, I8}}, {{w_gate, I, H8}, {w_up, I, H8}},
                        d, st);
        if (rc != CE_OK) return rc;
    }
    if (dw_gate || dw_down) {
        FfnGemm t = base;
        t.K = rows;
        FfnMatrix A[3] = {}, B[3] = {};
        int n = 0;
        // left^T right: [rows, m] and [rows, cols], their rows of m8 and cols8 elements
        const auto add = [&](const void* left, int64_t m, const void* right, int64_t cols, void* out,
                             float factor) {
            t.M[n] = m;
            t.N[n] = cols;
            t.scale[n] = factor;
            A[n] = FfnMatrix{left, rows, up8(m)};
            B[n] = FfnMatrix{right, rows, up8(cols)};
            ffn_output(&t, n, out, cols);
            ++n;
        };
        if (dw_gate) {
            add(dg, I, x, H, dw_gate, 1.f);
            add(du, I, x, H, dw_up, 1.f);
        }
        if (dw_down) add(dz, O, h, I, dw_down, scale);
        rc = ffn_launch(kDw, dtype, t, n, A, B, d, st);
        if (rc != CE_OK) return rc;
    }
    return CE_OK;
}
