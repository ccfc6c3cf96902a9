// Dropout: y = residual + keep * x / (1 - p), keep from counter-based random
// words (ce_philox.cuh), so that the backward, dx = keep * dy / (1 - p), is
// the same kernel on dy with no stored mask. Arithmetic in fp32, one
// rounding into the storage type.
//
// Bound by HBM: one read of x (and of the residual) and one write of y; the
// words cost 10 rounds of two 32 x 32 -> 64 multiplies for 4 elements.
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

struct DropArgs {
    const void* x;
    const void* res;  // or nullptr
    void* y;
    int64_t n;
    DropSpec d;
    int64_t* used;  // the {seed, offset} this call drew from, or nullptr
};

// One element's group, by single loads (tensors that are not 16-byte
// aligned, and the end of those that are).
template <typename T>
__device__ __forceinline__ void drop_group(const DropArgs& a, const PhiloxKey& key, int64_t g) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 4 * g + j < a.n ? Vec<T>::load1(a.x, 4 * g + j) : 0.f;
    if (a.d.mode == kDropSome) drop4(a.d, key, static_cast<uint64_t>(g), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = 4 * g + j;
        if (i >= a.n) break;
        float o = a.d.mode == kDropAll ? 0.f : v[j];
        if (a.res) o += Vec<T>::load1(a.res, i);
        Vec<T>::store1(a.y, i, o);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads) ce_dropout_kernel(const __grid_constant__ DropArgs a) {
    constexpr int N = Vec<T>::N;
    const PhiloxKey key = philox_key(a.d);
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(gridDim.x) * kDropThreads;
    if (a.used && tid == 0) {
        a.used[0] = static_cast<int64_t>((static_cast<uint64_t>(key.k1) << 32) | key.k0);
        a.used[1] = static_cast<int64_t>((static_cast<uint64_t>(key.o1) << 32) | key.o0);
    }
    if constexpr (!VEC) {
        for (int64_t g = tid; g < (a.n + 3) / 4; g += threads) drop_group<T>(a, key, g);
        return;
    }
    const int64_t nv = a.n / N;
    const uint4* x = static_cast<const uint4*>(a.x);
    const uint4* res = static_cast<const uint4*>(a.res);
    uint4* y = static_cast<uint4*>(a.y);
    for (int64_t i0 = tid; i0 < nv; i0 += threads * kDropVec) {
        uint4 vx[kDropVec], vr[kDropVec];
#pragma unroll
        for (int k = 0; k < kDropVec; ++k) {
            const int64_t i = i0 + k * threads;
            if (i < nv) {
                vx[k] = x[i];
                if (res) vr[k] = res[i];
            }
        }
#pragma unroll
        for (int k = 0; k < kDropVec; ++k) {
            const int64_t i = i0 + k * threads;
            if (i >= nv) break;
            float f[N];
            Vec<T>::unpack(vx[k], f);
            if (a.d.mode == kDropSome) {
#pragma unroll
                for (int j = 0; j < N / 4; ++j)
                    drop4(a.d, key, static_cast<uint64_t>(i * (N / 4) + j), f + 4 * j);
            } else if (a.d.mode == kDropAll) {
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = 0.f;
            }
            if (res) {
                float r[N];
                Vec<T>::unpack(vr[k], r);
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] += r[j];
            }
            y[i] = Vec<T>::pack(f);
        }
    }
    // the elements behind the last whole vector: nv * N is a multiple of 4
    const int64_t g = nv * (N / 4) + tid;
    if (g < (a.n + 3) / 4) drop_group<T>(a, key, g);
}

template <bool VEC>
const void* dropout_fn(int dtype) {
    return dtype == CE_F32    ? (const void*)&ce_dropout_kernel<float, VEC>
           : dtype == CE_BF16 ? (const void*)&ce_dropout_kernel<__nv_bfloat16, VEC>
                              : (const void*)&ce_dropout_kernel<__half, VEC>;
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
    a.x = x;
    a.res = residual;
    a.y = y;
    a.n = n;
    a.used = used;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return record_cuda_failure(e, "dropout device");
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                           reinterpret_cast<uintptr_t>(y);
    const bool vec = bits % 16 == 0;
    const int64_t per = vec ? int64_t{kDropVec} * (dtype == CE_F32 ? 4 : 8) : 4;
    const int64_t want = (n + kDropThreads * per - 1) / (kDropThreads * per);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(want, 8L * sms));
    void* args[] = {&a};
    e = cudaLaunchKernel(vec ? dropout_fn<true>(dtype) : dropout_fn<false>(dtype),
                         dim3(static_cast<unsigned>(grid)), dim3(kDropThreads), args, 0,
                         reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return record_cuda_failure(e, "dropout launch");
    return CE_OK;
}
