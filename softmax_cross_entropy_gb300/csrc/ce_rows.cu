// The token losses' forward: the choice of a row's layout, and the launch of
// the kernel (ce_rows_kernel.cuh).
#include <algorithm>
#include <cstdlib>
#include <map>
#include <mutex>
#include <string>
#include <tuple>

#include "ce_rows.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);
const void* rows_kernel_f32(int op, bool ent, int nt);
const void* rows_kernel_bf16(int op, bool ent, int nt);
const void* rows_kernel_f16(int op, bool ent, int nt);

namespace {

// dynamic shared memory that leaves room for a second CTA on the SM
constexpr size_t kHalfSm = 109 * 1000;
constexpr int64_t kKeepBytes = int64_t{96} << 20;  // of the 129 MB L2

// How many clusters of C CTAs fit the device at once.
std::mutex g_fit_mu;
std::map<std::tuple<int, const void*, int, size_t>, int> g_fit;

ce_status clusters_that_fit(const void* fn, int C, int threads, size_t smem, int sms, int* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_cuda_failure(e, "token loss device");
    std::lock_guard<std::mutex> lock(g_fit_mu);
    const auto key = std::make_tuple(dev, fn, C, smem);
    const auto it = g_fit.find(key);
    if (it != g_fit.end()) {
        *out = it->second;
        return CE_OK;
    }
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 most - static_cast<int>(fa.sharedSizeBytes));
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    int fit = 0;
    if (e == cudaSuccess && C == 1) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, threads, smem);
        fit *= sms;
    } else if (e == cudaSuccess) {
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(static_cast<unsigned>(C * sms));
        lc.blockDim = dim3(static_cast<unsigned>(threads));
        lc.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(C);
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        lc.attrs = &attr;
        lc.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&fit, fn, &lc);
    }
    if (e != cudaSuccess) return record_cuda_failure(e, "token loss occupancy");
    g_fit[key] = *out = std::max(fit, 1);
    return CE_OK;
}

int env_int(const char* name, int fallback) {
    const char* v = std::getenv(name);
    return (v && *v) ? std::atoi(v) : fallback;
}

}  // namespace

// Launches the forward of `op`; ent: entropies are formed; after_count: it
// follows rows_count, which it overlaps.
ce_status rows_launch(int op, bool ent, int dtype, const RowArgs& args, int sms, bool after_count,
                      cudaStream_t st) {
    RowArgs a = args;
    const int64_t esz = dtype == CE_F32 ? 4 : 2;
    // vectors of a row, wherever it starts
    const bool whole = (reinterpret_cast<uintptr_t>(a.p.x) | static_cast<uintptr_t>(a.p.step * esz) |
                        static_cast<uintptr_t>(a.p.outer * esz)) % 16 == 0;
    const int64_t nv = (a.p.V * esz + (whole ? 15 : 30)) / 16;
    const int64_t most = env_int("GBCE_ROWS_SLICE", 36864) / 16;
    int C = 1;
    auto slice = [&]() { return ((nv + C - 1) / C + 7) / 8 * 8; };
    while (C < kMaxRowCluster && slice() > most) C *= 2;
    while (C < kMaxRowCluster && a.p.rows * C * 2 <= sms && slice() > 256) C *= 2;
    if (const int forced = env_int("GBCE_ROWS_CLUSTER", 0)) C = forced;
    a.cluster = C;
    a.slice_vec = static_cast<int>(slice());
    a.buf_bytes = static_cast<uint32_t>((a.slice_vec * 16 + 127) / 128 * 128);
    const int nt = env_int("GBCE_ROWS_THREADS", a.slice_vec > 1152 ? 256
                                                : a.slice_vec > 576 || op == kRowDistill ? 64
                                                                                         : 32);
    a.nbuf = env_int("GBCE_ROWS_BUFFERS", kMaxBuf);
    while (a.nbuf > 1 && a.nbuf * a.buf_bytes > 200 * 1024) --a.nbuf;
    const size_t list = op == kRowDistill ? 4 * kListWords * static_cast<size_t>(a.K) : 0;
    a.nlist = kMaxLists;
    while (a.nlist > kListWarps && a.nbuf * a.buf_bytes + a.nlist * list > kHalfSm) --a.nlist;
    const size_t smem = a.nbuf * a.buf_bytes + (op == kRowDistill ? a.nlist : 0) * list;
    const void* fn = dtype == CE_F32    ? rows_kernel_f32(op, ent, nt)
                     : dtype == CE_BF16 ? rows_kernel_bf16(op, ent, nt)
                                        : rows_kernel_f16(op, ent, nt);
    const int threads = nt + 96 + (op == kRowDistill ? 32 * kListWarps : 0);
    int fit = 0;
    ce_status rc = clusters_that_fit(fn, C, threads, smem, sms, &fit);
    if (rc != CE_OK) return rc;
    const int64_t clusters =
        std::max<int64_t>(1, std::min<int64_t>({a.p.rows, int64_t{fit}, int64_t{kRowsMaxCtas}}));
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(clusters * C));
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (C > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(C);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after_count) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    lc.attrs = attr;
    lc.numAttrs = n;
    void* kargs[] = {&a};
    const cudaError_t e = cudaLaunchKernelExC(&lc, fn, kargs);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "token loss launch");
}

}  // namespace gbce
