// The gated feed-forward block for few rows (the tokens of a batch that is
// being generated): the weights are the large operand, so they are the rows
// of the tensor-core products and the tokens their columns.
//
// Bound by HBM: every weight is read once, 6 H I bytes. Two products,
// each split so that every SM reads the same number of weight bytes:
//  * ffn_rows: tiles of 128 weight rows (of Wg, then Wu; or of Wd) x K blocks
//    of 64 are units of 16 KB, dealt out in equal runs to one CTA an SM. A
//    TMA producer keeps a ring of units in flight (about 100 KB an SM); an MMA
//    thread multiplies each by the tokens' block of x (or h), N = rows
//    rounded up to 16; four epilogue warps write the sums of a tile's part,
//    fp32, to the workspace. A run may start and end inside a tile, so a
//    tile has a few parts.
//  * ffn_rows_act and ffn_rows_out add a tile's parts in order (results do
//    not depend on which SM finishes first) and apply the activation and
//    product, or the dropout and residual, in fp32, rounding once.
// The four launches overlap (programmatic dependent launch): the second
// product fills its ring with weights, which no launch of this call writes,
// while the first still runs and its sums are added. (Bringing more of them
// to L2 at the first product's end changed nothing: 61 us either way.)
#include <algorithm>
#include <cstdint>
#include <string>

#include "ce_ffn.cuh"
#include "ce_philox.cuh"
#include "ce_tc.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);

namespace {

constexpr int kRowsThreads = 192;  // producer, MMA issuer, 4 epilogue warps
constexpr int kRowsTile = 128;     // weight rows of a tile
constexpr uint32_t kRowsA = kRowsTile * kBK * 2;  // 16 KB
constexpr int kRowsStages = 7;  // units of the ring at most (of 18 KB, up to 16 tokens)
// The ring: where three units or more fit in the smaller (up to 112 tokens),
// two CTAs an SM, so that the second product's ring fills while the first
// product still runs; else one. (Rings of 110 KB each: 60 us for 1 token of
// 4096 x 12288, 130 and 92 KB 59 us, 148 and 74 KB 60 us.)
constexpr uint32_t kRowsSmemUp = 130 * 1024, kRowsSmemDown = 92 * 1024, kRowsSmemOne = 200 * 1024;

struct RowsArgs {
    int64_t units, per;  // tiles x K blocks; of a CTA
    int64_t tiles0;      // tiles of the first weight matrix
    int nk;              // K blocks of a tile
    int rows, nt;        // tokens; rounded up to a multiple of 16
    int stages, parts;   // ring slots; parts of a tile at most
    uint32_t stage_bytes, acc_cols, tmem_cols;  // of a unit; of an accumulator; of both
    float* sums;  // [tiles, parts, rows, 128]
    uint64_t timeout_ns;
    unsigned* status;
};

// The first CTA of tile t, and the CTAs that share it.
__host__ __device__ inline int64_t rows_first(int64_t t, int nk, int64_t per) { return t * nk / per; }
__host__ __device__ inline int rows_parts(int64_t t, int nk, int64_t per) {
    return static_cast<int>(((t + 1) * nk - 1) / per - t * nk / per) + 1;
}

__device__ __forceinline__ void rows_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A copy of weights, which are read once: the first to leave L2.
__device__ __forceinline__ void rows_load_once(uint32_t dst, const CUtensorMap* map, int x, int y,
                                               uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}
template <uint32_t AB>
__global__ void __launch_bounds__(kRowsThreads, 2)
ffn_rows(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
         const __grid_constant__ CUtensorMap mapx, const __grid_constant__ RowsArgs a) {
    extern __shared__ unsigned char rows_smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kRowsStages];
    __shared__ __align__(8) uint64_t empty_bar[kRowsStages];
    __shared__ __align__(8) uint64_t acc_full[2];
    __shared__ __align__(8) uint64_t acc_empty[2];
    __shared__ __align__(8) uint64_t done_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ uint32_t s_issued[kRowsStages];  // 0, or 2 + parity of the last copy into the stage
    __shared__ int s_fail;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem0 = (smem_u32(rows_smem_raw) + 1023u) & ~1023u;
    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * a.per;
    const int64_t u1 = u0 + a.per < a.units ? u0 + a.per : a.units;
    // the units of the ring's first round; a unit as its tile and K block,
    // stepped without divisions (H 1024, I 4096: 13.4 instead of 14.7 us)
    const int pre = static_cast<int>(u1 - u0 < a.stages ? u1 - u0 : a.stages);
    const int64_t tile_first = u0 / a.nk;
    const int kb_first = static_cast<int>(u0 - tile_first * a.nk);
    const uint64_t once = l2_evict_first_policy();
    const auto load_a = [&](int64_t t, int kb, uint32_t slot, uint32_t bar) {
        const bool second = t >= a.tiles0;
        rows_load_once(slot, second ? &map1 : &map0, kb * kBK,
                       static_cast<int>((second ? t - a.tiles0 : t) * kRowsTile), bar, once);
    };
    if (threadIdx.x == 0) {
        rows_prefetch_map(&map0);
        rows_prefetch_map(&map1);
        rows_prefetch_map(&mapx);
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
            s_issued[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 128);
        }
        mbar_init(smem_u32(&done_bar), 1);
        s_fail = 0;
        fence_mbar_init();
        // the first round's weights, before anything else is set up
        int64_t t = tile_first;
        for (int s = 0, kb = kb_first; s < pre; ++s) {
            const uint32_t fb = smem_u32(&full_bar[s]);
            mbar_arrive_expect_tx(fb, a.stage_bytes);
            load_a(t, kb, smem0 + static_cast<uint32_t>(s) * a.stage_bytes, fb);
            s_issued[s] = 2u;
            if (++kb == a.nk) {
                kb = 0;
                ++t;
            }
        }
    }
    if (warp == 1) {
        asm volatile(
            "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                smem_u32(&tmem_base_sh)),
            "r"(a.tmem_cols)
            : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_base_sh;

    if (warp == 0) {
        if (lane == 0) {
            const auto load_x = [&](int kb, uint32_t slot, uint32_t bar) {
                tma_load_2d(slot + kRowsA, &mapx, kb * kBK, 0, bar);
            };
            int64_t t = tile_first;
            int kb = kb_first;
            const auto step = [&] {
                if (++kb == a.nk) {
                    kb = 0;
                    ++t;
                }
            };
            // the tokens of the ring's first round, once the launch that writes
            // them is done
            pdl_wait();
            for (int s = 0; s < pre; ++s, step())
                load_x(kb, smem0 + static_cast<uint32_t>(s) * a.stage_bytes, smem_u32(&full_bar[s]));
            int s = 0;
            uint32_t ph = 1;
            bool fail = false;
            for (int64_t u = u0 + pre; u < u1; ++u, step()) {
                if (!tc_wait(smem_u32(&empty_bar[s]), ph ^ 1u, a.timeout_ns)) {
                    fail = true;
                    break;
                }
                const uint32_t fb = smem_u32(&full_bar[s]);
                const uint32_t slot = smem0 + static_cast<uint32_t>(s) * a.stage_bytes;
                mbar_arrive_expect_tx(fb, a.stage_bytes);
                load_a(t, kb, slot, fb);
                load_x(kb, slot, fb);
                s_issued[s] = 2u + ph;
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (fail) s_fail = 1;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = (1u << 4) | (AB << 7) | (AB << 10) |
                                   (static_cast<uint32_t>(a.nt >> 3) << 17) |
                                   (static_cast<uint32_t>(kRowsTile >> 4) << 24);
            int s = 0, run = 0;
            uint32_t ph = 0;
            bool fail = false;
            int kb = kb_first;
            for (int64_t u = u0; u < u1; ++u) {
                const int b = run & 1;
                const uint32_t acc = tmem + static_cast<uint32_t>(b) * a.acc_cols;
                const bool start = u == u0 || kb == 0;
                if (start && !tc_wait(smem_u32(&acc_empty[b]),
                                      (static_cast<uint32_t>(run >> 1) & 1u) ^ 1u, a.timeout_ns)) {
                    fail = true;
                    break;
                }
                if (!tc_wait(smem_u32(&full_bar[s]), ph, a.timeout_ns)) {
                    fail = true;
                    break;
                }
                tc_fence_after();
                const uint32_t slot = smem0 + static_cast<uint32_t>(s) * a.stage_bytes;
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    tc_mma(acc, tc_smem_desc(slot + 32u * k), tc_smem_desc(slot + kRowsA + 32u * k),
                           idesc, (start && k == 0) ? 0u : 1u);
                tc_commit(smem_u32(&empty_bar[s]));
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++kb == a.nk) kb = 0;
                if (kb == 0 || u + 1 == u1) {
                    tc_commit(smem_u32(&acc_full[b]));
                    ++run;
                }
            }
            if (fail) {
                s_fail = 1;
                tc_commit(smem_u32(&acc_full[run & 1]));  // so that nothing waits
            }
            tc_commit(smem_u32(&done_bar));
        }
    } else {
        const int q = warp & 3;
        int run = 0;
        int64_t t = tile_first;
        for (int64_t u = u0; u < u1; ++run, ++t) {
            const int64_t part = blockIdx.x - rows_first(t, a.nk, a.per);
            const int b = run & 1;
            const bool ok = tc_wait(smem_u32(&acc_full[b]), static_cast<uint32_t>(run >> 1) & 1u,
                                    a.timeout_ns);
            // (the whole warp goes on or none of it: what follows takes all lanes)
            if (__any_sync(~0u, !ok || *reinterpret_cast<volatile int*>(&s_fail))) {
                if (lane == 0) s_fail = 1;
                break;
            }
            tc_fence_after();
            const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b) * a.acc_cols;
            float* out = a.sums + ((t * a.parts + part) * a.rows) * kRowsTile + q * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < a.rows; c += 32) {
                float v[32];
                tc_ld32(trow + static_cast<uint32_t>(c), v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j < a.rows) out[static_cast<int64_t>(c + j) * kRowsTile] = v[j];
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&acc_empty[b]));
            u = (t + 1) * a.nk;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool done = mbar_wait_bounded(smem_u32(&done_bar), 0u, a.timeout_ns);
        if (s_fail || !done) {
            atomicOr(a.status, kDevErrTimeout);
            for (int s = 0; s < a.stages; ++s)
                if (s_issued[s])
                    (void)mbar_wait_bounded(smem_u32(&full_bar[s]), s_issued[s] & 1u, a.timeout_ns);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(a.tmem_cols)
                     : "memory");
}

struct RowsJoin {
    const float* sums;
    int64_t per, tiles0;
    int nk, parts, rows;
    int vec;  // y's rows are whole 8-byte vectors
    int64_t cols, pitch;  // I and I8, or O and O
    int act;
    void* out;  // h or y
    float* s;   // or nullptr
    float* a;
    const void* res;
    DropSpec drop;
};

// The parts of tile t for one token, added in order: this lane's four
// columns. The loads of the first eight are on their way together.
__device__ __forceinline__ void join_parts(const RowsJoin& j, int64_t t, int n, int row, int lane,
                                           float (&sum)[4]) {
    const float4* p = reinterpret_cast<const float4*>(j.sums + ((t * j.parts) * j.rows + row) * kRowsTile) + lane;
    const int64_t step = static_cast<int64_t>(j.rows) * (kRowsTile / 4);
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __ldcg(p + i * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 s = v[0];
    const auto add = [&s](const float4& q) {
        s.x += q.x;
        s.y += q.y;
        s.z += q.z;
        s.w += q.w;
    };
#pragma unroll
    for (int i = 1; i < 8; ++i) add(v[i]);
    for (int i = 8; i < n; ++i) add(__ldcg(p + i * step));
    sum[0] = s.x;
    sum[1] = s.y;
    sum[2] = s.z;
    sum[3] = s.w;
}

// Four values as 16 bits each.
template <typename T>
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
    const float t[8] = {f[0], f[1], f[2], f[3], 0.f, 0.f, 0.f, 0.f};
    const uint4 w = Vec<T>::pack(t);
    return make_uint2(w.x, w.y);
}

// A warp a (token, 128 columns), a lane four columns.
constexpr int kJoinThreads = 256;

// h = act(g) u (and s, a).
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) ffn_rows_act(const __grid_constant__ RowsJoin j) {
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(i / j.tiles0);
    const int64_t tile = i - row * j.tiles0;
    const int64_t c = tile * kRowsTile + 4 * lane;
    const int ng = rows_parts(tile, j.nk, j.per), nu = rows_parts(j.tiles0 + tile, j.nk, j.per);
    pdl_wait();
    if (row >= j.rows || c >= j.pitch) return;
    float g[4], u[4], h[4];
    join_parts(j, tile, ng, row, lane, g);
    join_parts(j, j.tiles0 + tile, nu, row, lane, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // (columns behind the last: rows of weights that are not there, zeros)
        const FfnGate r = ffn_gate<true>(j.act, g[e]);
        const bool in = c + e < j.cols;
        h[e] = in ? r.act * u[e] : 0.f;
        u[e] = in ? u[e] * r.slope : 0.f;
        g[e] = in ? r.act : 0.f;
    }
    const int64_t at = row * j.pitch + c;
    *reinterpret_cast<uint2*>(static_cast<T*>(j.out) + at) = pack4<T>(h);
    if (j.s) {
        *reinterpret_cast<float4*>(j.s + at) = make_float4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<float4*>(j.a + at) = make_float4(g[0], g[1], g[2], g[3]);
    }
}

// y = residual + dropout(z).
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) ffn_rows_out(const __grid_constant__ RowsJoin j) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(i / j.tiles0);
    const int64_t tile = i - row * j.tiles0;
    const int64_t c = tile * kRowsTile + 4 * lane;
    if (row >= j.rows || c >= j.cols) return;
    const int64_t at = row * j.cols + c;
    const int n = j.cols - c < 4 ? static_cast<int>(j.cols - c) : 4;
    // what no launch of this call writes, before the wait
    float res[4] = {0.f, 0.f, 0.f, 0.f}, factor[4];
    const bool drop = j.drop.mode != kDropNone;
    PhiloxKey key{};
    if (j.drop.mode == kDropSome) key = philox_key(j.drop);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (j.res && e < n) res[e] = Vec<T>::load1(j.res, at + e);
        factor[e] = j.drop.mode == kDropNone ? 1.f : 0.f;
    }
    if (j.drop.mode == kDropSome) {
        uint64_t block = static_cast<uint64_t>(at) >> 2;
        uint4 w = philox4x32(key, block);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t k = static_cast<uint64_t>(at + e);
            if (k >> 2 != block) {
                block = k >> 2;
                w = philox4x32(key, block);
            }
            const uint32_t l = static_cast<uint32_t>(k) & 3u;
            const uint32_t word = l == 0 ? w.x : l == 1 ? w.y : l == 2 ? w.z : w.w;
            factor[e] = word >= j.drop.threshold ? j.drop.scale : 0.f;
        }
    }
    const int parts = rows_parts(tile, j.nk, j.per);
    pdl_wait();
    float z[4];
    join_parts(j, tile, parts, row, lane, z);
#pragma unroll
    for (int e = 0; e < 4; ++e)  // (a dropped element leaves nothing, whatever it holds)
        z[e] = (drop ? (factor[e] != 0.f ? z[e] * factor[e] : 0.f) : z[e]) + res[e];
    if (j.vec && n == 4) {
        *reinterpret_cast<uint2*>(static_cast<T*>(j.out) + at) = pack4<T>(z);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) Vec<T>::store1(j.out, at + e, z[e]);
    }
}

int64_t up256r(int64_t b) { return (b + 255) / 256 * 256; }

unsigned join_grid(int64_t tiles, int64_t rows) {
    return static_cast<unsigned>((tiles * rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
}

// How a product of `tiles` weight tiles and K columns is dealt out to `sms`.
struct RowsPlan {
    int64_t units, per, grid;
    int nk, parts;
    int64_t bytes;  // of the sums
};
RowsPlan rows_plan(int64_t tiles, int64_t K, int64_t rows, int sms) {
    RowsPlan p;
    p.nk = static_cast<int>((K + kBK - 1) / kBK);
    p.units = tiles * p.nk;
    p.per = (p.units + sms - 1) / sms;
    p.grid = (p.units + p.per - 1) / p.per;
    p.parts = static_cast<int>((p.nk + p.per - 1) / p.per + 1);
    p.bytes = up256r(tiles * p.parts * rows * kRowsTile * 4);
    return p;
}

ce_status rows_pdl(const void* fn, dim3 grid, int threads, size_t smem, bool pdl, void** args,
                   cudaStream_t st, const char* what) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = &attr;
    lc.numAttrs = pdl ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, what);
}

// sums = [W0; W1] x^T
ce_status rows_product(const RowsPlan& p, int dtype, const void* w0, const void* w1, int64_t wrows,
                       const void* x, int64_t rows, int64_t K, float* sums, bool pdl,
                       uint64_t timeout_ns, unsigned* status, cudaStream_t st) {
    RowsArgs a = {};
    a.units = p.units;
    a.per = p.per;
    a.tiles0 = (wrows + kRowsTile - 1) / kRowsTile;
    a.nk = p.nk;
    a.rows = static_cast<int>(rows);
    a.nt = static_cast<int>((rows + 15) / 16 * 16);
    a.stage_bytes = kRowsA + static_cast<uint32_t>(a.nt) * kBK * 2;
    const uint32_t two = pdl ? kRowsSmemDown : kRowsSmemUp;
    const uint32_t ring = kRowsSmemDown / a.stage_bytes >= 3 ? two : kRowsSmemOne;
    a.stages = std::min<int>(kRowsStages, static_cast<int>(ring / a.stage_bytes));
    a.acc_cols = static_cast<uint32_t>(std::max(a.nt, 32));
    a.tmem_cols = 64;  // a power of two
    while (a.tmem_cols < 2 * a.acc_cols) a.tmem_cols *= 2;
    a.parts = p.parts;
    a.sums = sums;
    a.timeout_ns = timeout_ns;
    a.status = status;
    CUtensorMap m0, m1, mx;  // weights, tokens
    ce_status rc = tc_map_16bit(&m0, w0, dtype, wrows, K, kRowsTile);
    m1 = m0;
    if (rc == CE_OK && w1) rc = tc_map_16bit(&m1, w1, dtype, wrows, K, kRowsTile);
    if (rc == CE_OK) rc = tc_map_16bit(&mx, x, dtype, rows, K, static_cast<uint32_t>(a.nt));
    if (rc != CE_OK) return rc;
    const void* fn = dtype == CE_BF16 ? (const void*)&ffn_rows<1u> : (const void*)&ffn_rows<0u>;
    const size_t smem = static_cast<size_t>(a.stages) * a.stage_bytes + 1024;
    rc = tc_smem_limit(fn, kRowsSmemOne + 1024);
    if (rc != CE_OK) return rc;
    void* args[] = {&m0, &m1, &mx, &a};
    return rows_pdl(fn, dim3(static_cast<unsigned>(p.grid)), kRowsThreads, smem, pdl, args, st,
                    "feed-forward rows launch");
}

}  // namespace

int64_t ffn_rows_workspace(int64_t rows, int64_t H8, int64_t I8, int64_t O, int sms) {
    const int64_t ti = (I8 + kRowsTile - 1) / kRowsTile, to = (O + kRowsTile - 1) / kRowsTile;
    return rows_plan(2 * ti, H8, rows, sms).bytes + rows_plan(to, I8, rows, sms).bytes;
}

// The block's forward for at most 256 rows: operands as ce_ffn_fwd has
// packed them (x [rows, H8], Wg and Wu [I, H8], Wd [O, I8], h, s, a [rows,
// I8]); y and residual [rows, O].
ce_status ffn_rows_fwd(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                       const void* residual, int dtype, int64_t rows, int64_t H8, int64_t I,
                       int64_t I8, int64_t O, int act, const DropSpec& drop, void* y, void* h,
                       float* s, float* a, void* workspace, int sms, uint64_t timeout_ns,
                       unsigned* status, cudaStream_t st) {
    const int64_t ti = (I8 + kRowsTile - 1) / kRowsTile, to = (O + kRowsTile - 1) / kRowsTile;
    const RowsPlan up = rows_plan(2 * ti, H8, rows, sms), down = rows_plan(to, I8, rows, sms);
    float* sums_up = static_cast<float*>(workspace);
    float* sums_down = reinterpret_cast<float*>(static_cast<char*>(workspace) + up.bytes);
    // the first launch waits for all work before it: what the others read
    // early (the weights) is then written
    ce_status rc = rows_product(up, dtype, w_gate, w_up, I, x, rows, H8, sums_up, false, timeout_ns,
                                status, st);
    if (rc != CE_OK) return rc;
    const bool bf = dtype == CE_BF16;
    RowsJoin j = {};
    j.sums = sums_up;
    j.per = up.per;
    j.nk = up.nk;
    j.parts = up.parts;
    j.tiles0 = ti;
    j.rows = static_cast<int>(rows);
    j.cols = I;
    j.pitch = I8;
    j.act = act;
    j.out = h;
    j.s = s;
    j.a = a;
    void* args[] = {&j};
    rc = rows_pdl(bf ? (const void*)&ffn_rows_act<__nv_bfloat16> : (const void*)&ffn_rows_act<__half>,
                  dim3(join_grid(ti, rows)), kJoinThreads, 0, true, args, st,
                  "feed-forward activation launch");
    if (rc != CE_OK) return rc;
    rc = rows_product(down, dtype, w_down, nullptr, O, h, rows, I8, sums_down, true, timeout_ns,
                      status, st);
    if (rc != CE_OK) return rc;
    j.sums = sums_down;
    j.per = down.per;
    j.nk = down.nk;
    j.parts = down.parts;
    j.tiles0 = to;
    j.cols = j.pitch = O;
    j.vec = O % 4 == 0 && reinterpret_cast<uintptr_t>(y) % 8 == 0 ? 1 : 0;
    j.out = y;
    j.res = residual;
    j.drop = drop;
    return rows_pdl(bf ? (const void*)&ffn_rows_out<__nv_bfloat16> : (const void*)&ffn_rows_out<__half>,
                    dim3(join_grid(to, rows)), kJoinThreads, 0, true, args, st,
                    "feed-forward output launch");
}

}  // namespace gbce
