// Dropout: y = residual + keep * x / (1 - p), keep from counter-based random
// words (ce_philox.cuh), so that the backward, dx = keep * dy / (1 - p), is
// the same kernel on dy with no stored mask. Arithmetic in fp32, one
// rounding into the storage type.
//
// One read of x (and of the residual) and one write of y; the words cost 10
// rounds of two 32 x 32 -> 64 multiplies for 4 elements. So what is the same
// for every thread of a launch is kept out of it: the round keys come with the
// arguments (constant operands), the counter's three upper words are the
// launch's (it covers 2^31 blocks), which leaves 18 of the 20 multiplies, and
// indexes are 32-bit steps from moving pointers.
// fp32 is bound by HBM (ncu: 74% of its peak, the multiplies' pipe active 45%
// of the time). 16-bit types are not (47%), and the pipe is active 63%: of a
// grid of 8 CTAs an SM 5 fit at 42 registers, and the 3 that follow have fewer
// warps to overlap loads and multiplies in.
// Measured, p = 0.1, 16384 x 8192: fp32 168 us (6.4 TB/s of reads and
// writes), bf16 110 us (4.9 TB/s; 84 us, 6.4 TB/s, with no words to form), with
// the residual 243 us and 127 us (6.6 and 6.3 TB/s).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ce_kernels.cuh"
#include "ce_philox.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);

namespace {

constexpr int kDropThreads = 256;
constexpr int kDropVec = 2;  // 16-byte vectors a thread holds at a time
constexpr int kDropRounds = 10;
constexpr int64_t kDropMost = int64_t{1} << 33;  // elements of a launch: 2^31 blocks of words

struct DropKeys {
    uint32_t k[2 * kDropRounds];  // of round r at 2 r and 2 r + 1
    uint32_t o0, o1;              // the offset
};

struct DropArgs {
    const void* x;
    const void* res;  // or nullptr
    void* y;
    int64_t n;       // at most kDropMost
    uint32_t base, upper;  // the block counter of element 0
    DropSpec d;
    DropKeys keys;  // of d.seed and d.offset, where d.state is nullptr
    int64_t* used;  // the {seed, offset} this call drew from, or nullptr
};

__host__ __device__ inline void drop_keys(uint64_t seed, uint64_t offset, DropKeys* out) {
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#ifdef __CUDA_ARCH__
#pragma unroll
#endif
    for (int r = 0; r < kDropRounds; ++r) {
        out->k[2 * r] = k0;
        out->k[2 * r + 1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out->o0 = static_cast<uint32_t>(offset);
    out->o1 = static_cast<uint32_t>(offset >> 32);
}

// The words of block `group` (its counter's lowest word), as philox4x32 forms
// them.
__device__ __forceinline__ uint4 drop_words(const DropKeys& key, uint32_t upper, uint32_t group) {
    uint32_t c0 = group, c1 = upper, c2 = key.o0, c3 = key.o1;
#pragma unroll
    for (int r = 0; r < kDropRounds; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ key.k[2 * r];
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ key.k[2 * r + 1];
        c3 = static_cast<uint32_t>(a);
    }
    return make_uint4(c0, c1, c2, c3);
}
__device__ __forceinline__ void drop_block(const DropArgs& a, const DropKeys& key, uint32_t group,
                                           float* v) {
    const uint4 w = drop_words(key, a.upper, group);
    v[0] = w.x >= a.d.threshold ? v[0] * a.d.scale : 0.f;
    v[1] = w.y >= a.d.threshold ? v[1] * a.d.scale : 0.f;
    v[2] = w.z >= a.d.threshold ? v[2] * a.d.scale : 0.f;
    v[3] = w.w >= a.d.threshold ? v[3] * a.d.scale : 0.f;
}

// One block of elements by single loads (tensors that are not 16-byte
// aligned, and the end of those that are).
template <typename T>
__device__ __forceinline__ void drop_group(const DropArgs& a, const DropKeys& key, int64_t g) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 4 * g + j < a.n ? Vec<T>::load1(a.x, 4 * g + j) : 0.f;
    if (a.d.mode == kDropSome) drop_block(a, key, a.base + static_cast<uint32_t>(g), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = 4 * g + j;
        if (i >= a.n) break;
        float o = a.d.mode == kDropAll ? 0.f : v[j];
        if (a.res) o += Vec<T>::load1(a.res, i);
        Vec<T>::store1(a.y, i, o);
    }
}

// STATE: seed and offset are read from the device when the kernel runs.
template <typename T, bool VEC, bool STATE>
__global__ void __launch_bounds__(kDropThreads) ce_dropout_kernel(const __grid_constant__ DropArgs a) {
    constexpr int N = Vec<T>::N;
    DropKeys own;
    if constexpr (STATE) {
        const uint64_t seed = static_cast<uint64_t>(a.d.state[0]);
        const uint64_t offset = a.d.offset + static_cast<uint64_t>(a.d.state[1]);
        drop_keys(seed, offset, &own);
        if (a.used && blockIdx.x == 0 && threadIdx.x == 0) {
            a.used[0] = static_cast<int64_t>(seed);
            a.used[1] = static_cast<int64_t>(offset);
        }
    } else if (a.used && blockIdx.x == 0 && threadIdx.x == 0) {
        a.used[0] = static_cast<int64_t>(a.d.seed);
        a.used[1] = static_cast<int64_t>(a.d.offset);
    }
    const DropKeys& key = STATE ? own : a.keys;
    if constexpr (!VEC) {
        const int64_t tid = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x;
        const int64_t threads = static_cast<int64_t>(gridDim.x) * kDropThreads;
        for (int64_t g = tid; g < (a.n + 3) / 4; g += threads) drop_group<T>(a, key, g);
        return;
    }
    // a CTA's vectors are kDropVec x kDropThreads in a row
    constexpr uint32_t kStep = kDropVec * kDropThreads;
    const uint32_t nv = static_cast<uint32_t>(a.n / N);
    uint32_t i = blockIdx.x * kStep + threadIdx.x;
    const uint32_t stride = gridDim.x * kStep;
    const uint4* x = static_cast<const uint4*>(a.x) + i;
    const uint4* res = static_cast<const uint4*>(a.res) + (a.res ? i : 0u);
    uint4* y = static_cast<uint4*>(a.y) + i;
    for (; i < nv; i += stride) {
        uint4 vx[kDropVec], vr[kDropVec];
#pragma unroll
        for (int k = 0; k < kDropVec; ++k) {
            if (i + k * kDropThreads < nv) {
                vx[k] = x[k * kDropThreads];
                if (a.res) vr[k] = res[k * kDropThreads];
            }
        }
#pragma unroll
        for (int k = 0; k < kDropVec; ++k) {
            if (i + k * kDropThreads >= nv) break;
            float f[N];
            Vec<T>::unpack(vx[k], f);
            if (a.d.mode == kDropSome) {
#pragma unroll
                for (int j = 0; j < N / 4; ++j)
                    drop_block(a, key, a.base + (i + k * kDropThreads) * (N / 4) + j, f + 4 * j);
            } else if (a.d.mode == kDropAll) {
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = 0.f;
            }
            if (a.res) {
                float r[N];
                Vec<T>::unpack(vr[k], r);
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] += r[j];
            }
            y[k * kDropThreads] = Vec<T>::pack(f);
        }
        if (nv - i <= stride) break;  // (i + stride may pass 32 bits)
        x += stride;
        y += stride;
        if (a.res) res += stride;
    }
    // the elements behind the last whole vector: nv * N is a multiple of 4
    const int64_t g = static_cast<int64_t>(nv) * (N / 4) + blockIdx.x * kDropThreads + threadIdx.x;
    if (g < (a.n + 3) / 4) drop_group<T>(a, key, g);
}

template <bool VEC, bool STATE>
const void* dropout_fn(int dtype) {
    return dtype == CE_F32    ? (const void*)&ce_dropout_kernel<float, VEC, STATE>
           : dtype == CE_BF16 ? (const void*)&ce_dropout_kernel<__nv_bfloat16, VEC, STATE>
                              : (const void*)&ce_dropout_kernel<__half, VEC, STATE>;
}
const void* dropout_fn(int dtype, bool vec, bool state) {
    return vec ? (state ? dropout_fn<true, true>(dtype) : dropout_fn<true, false>(dtype))
               : (state ? dropout_fn<false, true>(dtype) : dropout_fn<false, false>(dtype));
}

}  // namespace

// What p, seed and offset ask for; false where p is not a probability.
bool drop_spec(double p, uint64_t seed, uint64_t offset, const int64_t* state, DropSpec* out) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    out->seed = seed;
    out->offset = offset;
    out->state = state;
    out->mode = p == 0.0 ? kDropNone : p == 1.0 ? kDropAll : kDropSome;
    out->threshold = p == 1.0 ? 0u : static_cast<uint32_t>(std::floor(p * 4294967296.0));
    out->scale = p == 1.0 ? 0.f : static_cast<float>(1.0 / (1.0 - p));
    return true;
}

}  // namespace gbce

using namespace gbce;

extern "C" ce_status ce_dropout(const void* x, const void* residual, void* y, int dtype, int64_t n,
                                double p, uint64_t seed, uint64_t offset, const int64_t* state,
                                int64_t* used, ce_stream_t stream) {
    if (dtype != CE_F32 && dtype != CE_BF16 && dtype != CE_F16) return CE_ERR_INVALID_ARG;
    DropArgs a = {};
    if (n < 0 || !drop_spec(p, seed, offset, state, &a.d)) return CE_ERR_INVALID_ARG;
    if (n > 0 && (!x || !y)) return CE_ERR_INVALID_ARG;
    if (n == 0 && !used) return CE_OK;
    drop_keys(seed, offset, &a.keys);
    a.used = used;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return record_cuda_failure(e, "dropout device");
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                           reinterpret_cast<uintptr_t>(y);
    const bool vec = bits % 16 == 0;
    const int64_t bytes = dtype == CE_F32 ? 4 : 2;
    const int64_t per = vec ? int64_t{kDropVec} * 16 / bytes : 4;
    for (int64_t at = 0; at == 0 || at < n; at += kDropMost) {
        a.n = std::min(n - at, kDropMost);
        a.base = static_cast<uint32_t>(at >> 2);
        a.upper = static_cast<uint32_t>(at >> 34);
        a.x = static_cast<const char*>(x) + at * bytes;
        a.res = residual ? static_cast<const char*>(residual) + at * bytes : nullptr;
        a.y = static_cast<char*>(y) + at * bytes;
        const int64_t want = (a.n + kDropThreads * per - 1) / (kDropThreads * per);
        const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(want, 8L * sms));
        void* args[] = {&a};
        e = cudaLaunchKernel(dropout_fn(dtype, vec, state != nullptr), dim3(static_cast<unsigned>(grid)),
                             dim3(kDropThreads), args, 0, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return record_cuda_failure(e, "dropout launch");
    }
    return CE_OK;
}
