// The tensor-core GEMMs' common parts (ce_gemm_tc.cu, ce_ffn.cu): tile
// shapes, shared-memory and instruction descriptors, and the tcgen05, TMA and
// bulk-group instructions as inline PTX.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "ce_kernels.cuh"
#include "gbce.h"

namespace gbce {

// Tiles of BM x 256 (BM = 128 or 256) with K blocks of 64, one CTA an SM:
//  * BM = 128: 4 stages of 128 x 64 + 256 x 64 (48 KB each); two 256-column
//    accumulators, so the epilogue of a tile overlaps the next tile's MMAs;
//  * BM = 256: 3 stages of 256 x 64 + 256 x 64 (64 KB each); the tile's two
//    128-row halves take the 512 columns, the epilogue does not overlap,
//    but each stage's bytes feed twice the MMA work (the TMA latency is
//    what limits the 128-row tiles: a third fewer bytes a flop).
constexpr int kMmaM = 128, kBN = 256, kBK = 64, kTcMaxStages = 4;
constexpr int kTcThreads = 192;  // producer, MMA issuer, 4 epilogue warps
constexpr uint32_t kBBytes = kBN * kBK * 2;
constexpr uint32_t kHalfA = kMmaM * kBK * 2;  // 128 rows of A (16 KB)
constexpr uint32_t kMnBox = 64 * kBK * 2;  // one 64 (MN) x 64 (K) box of an MN-major tile
constexpr uint32_t kTmemCols = 2 * kBN;    // 512 columns
template <int BM>
struct TcTile {
    static constexpr int kStages = BM == 256 ? 3 : 4;
    static constexpr int kHalves = BM / kMmaM;      // 128-row MMAs a K step
    static constexpr int kAccBufs = BM == 256 ? 1 : 2;
    static constexpr uint32_t kABytes = BM * kBK * 2;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes;
};
constexpr uint32_t kRingBytes = 4 * (kHalfA + kBBytes);  // the same for both BM
static_assert(TcTile<128>::kStages * TcTile<128>::kStageBytes == kRingBytes &&
                  TcTile<256>::kStages * TcTile<256>::kStageBytes == kRingBytes,
              "both tile shapes use the same ring");
// epilogue staging for TMA stores: per epilogue warp two 32-row x 128-byte
// boxes (4 KB each, 128-byte swizzle)
constexpr uint32_t kStageOut = 4096;
constexpr uint32_t kOutBytes = 4 * 2 * kStageOut;
constexpr size_t kTcSmem = static_cast<size_t>(kRingBytes) + kOutBytes + 1024;

// Shared-memory matrix descriptor of a K-major operand tile stored as
// 128-byte rows with the 128-byte swizzle (8-row atoms of 1024 bytes):
// start address, leading offset (unused for this layout: 1), stride
// between 8-row atoms 1024 bytes, descriptor version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t tc_smem_desc(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// The same for an MN-major operand tile stored as boxes of 64 MN elements
// (one 128-byte swizzled row) x 64 K rows, 8 KB each, side by side along
// MN: 8-row (K) atoms of 1024 bytes, the stride between atoms along K (the
// stride dimension offset) 1024 bytes, between 64-element blocks along MN
// (the leading dimension offset) one box, 8 KB.
__device__ __forceinline__ uint64_t tc_smem_desc_mn(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kMnBox >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B of the
// given type (0 fp16, 1 bf16), A and B K-major (0) or MN-major (1, the
// transpose bits 15 and 16), N = kBN, M = kMmaM.
__host__ __device__ constexpr uint32_t tc_idesc(uint32_t ab, uint32_t a_mn = 0, uint32_t b_mn = 0) {
    return (1u << 4) | (ab << 7) | (ab << 10) | (a_mn << 15) | (b_mn << 16) |
           (static_cast<uint32_t>(kBN >> 3) << 17) | (static_cast<uint32_t>(kMmaM >> 4) << 24);
}

// Bounded wait for the producer and MMA threads of the tight GEMM pipeline:
// poll without a suspend hint (a suspended thread may wake late), reading
// the global timer only every 1024 polls.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 1023u) == 0 && global_timer_ns() - t0 > timeout_ns) return false;
    }
}

// TMA store and reduce-add of a 2-D box from this CTA's shared memory, in
// a bulk group (commit, then wait for the reads before reusing the buffer)
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int x,
                                                  int y) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// at most one bulk group still reading shared memory
__device__ __forceinline__ void bulk_wait_read_1() {
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// this thread's shared-memory writes visible to the TMA (async proxy)
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` once every tcgen05 operation this thread issued so far
// has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 consecutive fp32 columns of this thread's accumulator row.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Raises a kernel's limit of dynamic shared memory to `bytes`, once a device
// (the current one).
ce_status tc_smem_limit(const void* fn, size_t bytes);

// A 2-D map of a row-major [outer, inner] matrix of 16-bit elements, boxes of
// box_outer x 64 elements (128 bytes: the swizzle width), 128-byte swizzle,
// zeros outside the matrix (ce_gemm_tc.cu). A K-major operand is [MN, K] with
// boxes of 128 or 256 rows, an MN-major one [K, MN] with boxes of 64 K rows.
ce_status tc_map_16bit(CUtensorMap* map, const void* p, int dtype, int64_t outer, int64_t inner,
                       uint32_t box_outer);

}  // namespace gbce
