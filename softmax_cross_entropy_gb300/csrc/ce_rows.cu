// The token losses' forward over rows of logits: one kernel in three forms
// (log-probabilities of given tokens; the clipped policy loss; distillation
// from a teacher's top logits). Each forms a row's softmax statistics in one
// pass and, where a gradient is asked for, writes it in a second pass over the
// row (which then comes from L2).
#include <algorithm>

#include "ce_rows.cuh"
#include "gbce.h"

namespace gbce {
ce_status record_cuda_failure(cudaError_t e, const char* what);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Entry {
    float x, q;     // the logit, the teacher's probability
    float lq, qs;   // log q; the sum of q over entries of this class (its first entry)
    int64_t j;      // the class, -1: no entry, or not the first of its class
};

template <typename T, int OP, bool ENT>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a) {
    using VT = Vec<T>;
    constexpr int VE = VT::N;
    extern __shared__ uint32_t listed[];  // a bit a class: it is in the teacher's list
    __shared__ RowPart red[kWarps];
    __shared__ double red_d[kWarps];
    __shared__ int s_flag;
    __shared__ Entry ent[OP == kRowDistill ? kTopMax : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool tail_mode = OP == kRowDistill && a.teacher_lse != nullptr;
    if (tail_mode) {
        for (int i = tid; i < (a.p.V + 31) / 32; i += kThreads) listed[i] = 0u;
        __syncthreads();
    }
    if (OP == kRowLogp && a.ticket && blockIdx.x == 0 && tid == 0) *a.ticket = 0u;
    double sum = 0.0;
    for (int64_t r = blockIdx.x; r < a.p.rows; r += gridDim.x) {
        const int64_t at = a.p.at(r);
        const T* x = reinterpret_cast<const T*>(a.p.x) + at;
        T* dx = a.p.dx ? reinterpret_cast<T*>(a.p.dx) + at : nullptr;
        const RowSpan sp = row_span<T>(x, a.p.V);
        const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
        uint4* dv = dx ? reinterpret_cast<uint4*>(dx + sp.head) : nullptr;
        const int edges = sp.head + sp.tail;  // at most 14 single elements, one a thread
        const int64_t edge = tid < sp.head ? tid : a.p.V - sp.tail + (tid - sp.head);
        const int64_t t = OP == kRowDistill ? load_index(a.index, a.idx64, r * a.K)
                                            : load_index(a.tokens, a.tok64, r);
        const bool in_range = t >= 0 && t < a.p.V;
        const bool counts = in_range && (OP == kRowDistill || t != a.ignore_index);
        if (!counts) {
            if (tid == 0) {
                if (!in_range && (OP == kRowDistill ? t >= 0 : t != a.ignore_index))
                    atomicOr(a.status, kDevErrTarget);
                if (OP != kRowLogp && a.reduction == kRedNone) a.loss[r] = 0.f;
                if (OP != kRowDistill) {
                    if (a.logp) a.logp[r] = 0.f;
                    if (a.entropy) a.entropy[r] = 0.f;
                    if (a.kl_out) a.kl_out[r] = 0.f;
                    if (a.clipped) a.clipped[r] = 0;
                }
            }
            if (dx) {
                for (int v = tid; v < sp.nvec; v += kThreads) dv[v] = make_uint4(0u, 0u, 0u, 0u);
                if (tid < edges) VT::store1(dx, edge, 0.f);
            }
            continue;
        }
        // ---- the teacher's list, by warp 0
        __shared__ double s_mass, s_rest;
        if (OP == kRowDistill) {
            if (warp == 0) {
                double top = -INFINITY;
                
                for (int k = lane; k < a.K; k += 32) {
                    int64_t j = load_index(a.index, a.idx64, r * a.K + k);
                    if (j >= a.p.V) {
                        atomicOr(a.status, kDevErrTarget);
                        j = -1;
                    }
                    const int64_t w = r * a.K + k;
                    const float v = a.teacher_dtype == 0 ? Vec<float>::load1(a.teacher, w)
                                    : a.teacher_dtype == 1 ? Vec<__nv_bfloat16>::load1(a.teacher, w)
                                                           : Vec<__half>::load1(a.teacher, w);
                    ent[k].j = j;
                    ent[k].lq = j < 0 ? -INFINITY : v;
                    ent[k].x = j < 0 ? 0.f : VT::load1(x, j);
                    if (j >= 0) top = fmax(top, v * a.invT);
                }
                for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(~0u, top, o));
                double mass = 0.0;
                const double shift = a.teacher_lse ? static_cast<double>(a.teacher_lse[r]) : top;
                for (int k = lane; k < a.K; k += 32) {
                    const double lq = ent[k].j < 0 ? -INFINITY : ent[k].lq * a.invT - shift;
                    ent[k].lq = static_cast<float>(lq);
                    ent[k].q = exp_wide(lq);
                    mass += ent[k].q;
                }
                for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(~0u, mass, o);
                double rest = 0.0;
                if (a.teacher_lse) {
                    rest = fmax(0.0, 1.0 - mass);
                } else {
                    const float lm = logf(static_cast<float>(mass));
                    for (int k = lane; k < a.K; k += 32) {
                        ent[k].q = static_cast<float>(ent[k].q / mass);
                        ent[k].lq -= lm;
                    }
                    mass = 1.0;
                }
                __syncwarp();
                for (int k = lane; k < a.K; k += 32) {  // the first entry of each class
                    float qs = 0.f;
                    bool first = true;
                    for (int i = 0; i < a.K; ++i)
                        if (ent[i].j == ent[k].j) {
                            qs += ent[i].q;
                            first = first && i >= k;
                        }
                    ent[k].qs = first ? qs : -1.f;
                }
                __syncwarp();
                for (int k = lane; k < a.K; k += 32) {
                    if (ent[k].qs < 0.f) ent[k].j = -1;
                    if (ent[k].j >= 0 && tail_mode) atomicOr(&listed[ent[k].j >> 5], 1u << (ent[k].j & 31));
                }
                if (lane == 0) {
                    s_mass = mass;
                    s_rest = rest;
                }
            }
            __syncthreads();
        }
        // ---- statistics
        RowPart st = {-INFINITY, 0.f, 0.f};
        float top = -INFINITY;  // of all elements, the listed ones included
        auto add = [&](float f, float m) {
            const float d = f - (m == -INFINITY ? 0.f : m);
            const float arg = fmaf(d, a.c, d * a.c_low);
            const float e = ex2(arg);
            st.S += e;
            if (ENT) st.Q = fmaf(e, fmaxf(arg, -256.f), st.Q);
        };
        auto raise = [&](float m) {
            if (m > st.m) {
                RowPart b = {m, 0.f, 0.f};
                part_merge<ENT>(st, b, a.c);
            }
        };
        auto hidden = [&](int64_t j) { return (listed[j >> 5] >> (j & 31)) & 1u; };
        for (int v = tid; v < sp.nvec; v += kThreads) {
            const uint4 q = xv[v];
            float f[VE];
            VT::unpack(q, f);
            if (tail_mode) {
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (hidden(sp.head + static_cast<int64_t>(v) * VE + i)) f[i] = -INFINITY;
            }
            float m = f[0];
#pragma unroll
            for (int i = 1; i < VE; ++i) m = fmaxf(m, f[i]);
            raise(m);
#pragma unroll
            for (int i = 0; i < VE; ++i) add(f[i], st.m);
        }
        if (tid < edges) {
            float f = VT::load1(x, edge);
            if (tail_mode && hidden(edge)) f = -INFINITY;
            raise(f);
            add(f, st.m);
        }
        __syncwarp();
        part_warp_merge<ENT>(st, a.c);
        if (lane == 0) red[warp] = st;
        __syncthreads();
        st = lane < kWarps ? red[lane] : RowPart{-INFINITY, 0.f, 0.f};
        part_warp_merge<ENT>(st, a.c);
        const float weight = a.weight ? __ldg(a.weight + r) : 1.f;

        if (OP == kRowDistill) {
            // the listed classes' share, and the sums over all
            float left = st.S;
            if (tail_mode) {
                RowPart in = {-INFINITY, 0.f, 0.f};
                for (int k = lane; k < a.K; k += 32)
                    if (ent[k].j >= 0) in.m = fmaxf(in.m, ent[k].x);
                in.m = warp_max_f32(in.m);
                const float M = fmaxf(in.m, st.m);
                for (int k = lane; k < a.K; k += 32)
                    if (ent[k].j >= 0) in.S += ex2((ent[k].x - M) * a.c);
                in.S = warp_sum(in.S);
                RowPart zero = {M, 0.f, 0.f};
                part_merge<false>(st, zero, a.c);
                left = st.S;
                st.S += in.S;
            }
            const float logS = logf(st.S);
            if (warp == 0) {
                float l = 0.f;
                for (int k = lane; k < a.K; k += 32) {
                    const float lp = log_prob(ent[k].x, st.m, a.invT, logS);
                    if (ent[k].q != 0.f) l += ent[k].q * (ent[k].lq - lp);
                }
                l = warp_sum(l);
                const float rest = static_cast<float>(s_rest);
                if (rest > 0.f && left > 0.f) l += rest * (logf(rest) - (logf(left) - logS));
                if (lane == 0) {
                    if (a.reduction == kRedNone)
                        a.loss[r] = static_cast<float>(static_cast<double>(a.scale) * weight * l);
                    else
                        sum += static_cast<double>(weight) * l;
                }
            }
            if (dx) {
                const float s = row_scale(a, weight * a.invT);
                const float mass = static_cast<float>(s_mass + s_rest);
                const float cut = left > 0.f ? static_cast<float>(s_rest) * (st.S / left) : 0.f;
                const float u = s * (mass - (tail_mode ? cut : 0.f)) / st.S;
                for (int v = tid; v < sp.nvec; v += kThreads) {
                    float f[VE];
                    VT::unpack(xv[v], f);
#pragma unroll
                    for (int i = 0; i < VE; ++i) f[i] = u * ex2((f[i] - st.m) * a.c);
                    dv[v] = VT::pack(f);
                }
                if (tid < edges) VT::store1(dx, edge, u * ex2((VT::load1(x, edge) - st.m) * a.c));
                __syncthreads();
                for (int k = tid; k < a.K; k += kThreads)
                    if (ent[k].j >= 0)
                        VT::store1(dx, ent[k].j,
                                   s * (mass * (ex2((ent[k].x - st.m) * a.c) / st.S) - ent[k].qs));
            }
            __syncthreads();
            if (tail_mode)
                for (int k = tid; k < a.K; k += kThreads)
                    if (ent[k].j >= 0) listed[ent[k].j >> 5] = 0u;
            __syncthreads();
            continue;
        }

        const float logS = logf(st.S);
        const float xt = VT::load1(x, t);
        const float lp = log_prob(xt, st.m, a.invT, logS);
        const float H = ENT ? logS - kLn2 * (st.Q / st.S) : 0.f;
        if (tid == 0) {
            if (a.logp) a.logp[r] = lp;
            if (a.entropy) a.entropy[r] = H;
            if (a.kept) a.kept[r] = RowKept{st.m, st.S, H, lp};
        }
        if (OP == kRowPolicy) {
            const PolicyRow pr = policy_row(a, lp, __ldg(a.adv + r / a.adv_rows),
                                            a.old ? __ldg(a.old + r) : 0.f,
                                            a.ref ? __ldg(a.ref + r) : 0.f);
            if (tid == 0) {
                const float l = ENT ? fmaf(-a.ent, H, pr.loss) : pr.loss;
                if (a.reduction == kRedNone)
                    a.loss[r] = static_cast<float>(static_cast<double>(a.scale) * weight * l);
                else
                    sum += static_cast<double>(weight) * l;
                if (a.kl_out) a.kl_out[r] = pr.kl;
                if (a.clipped) a.clipped[r] = pr.clipped ? 1 : 0;
            }
            if (dx) {
                __syncthreads();  // every thread has read the token's logit (dx may be x)
                // g_j = e_j (u0 + u1 a_j), plus the slope at the token
                const float s = row_scale(a, weight * a.invT);
                const float k0 = pr.slope * s, k1 = a.ent * s;
                const float u0 = (ENT ? fmaf(k1, H - logS, -k0) : -k0) / st.S;
                const float u1 = ENT ? k1 * kLn2 / st.S : 0.f;
                auto grad = [&](float f) {
                    const float arg = (f - st.m) * a.c;
                    const float e = ex2(arg);
                    return e * (ENT ? fmaf(u1, fmaxf(arg, -256.f), u0) : u0);
                };
                for (int v = tid; v < sp.nvec; v += kThreads) {
                    float f[VE];
                    VT::unpack(xv[v], f);
#pragma unroll
                    for (int i = 0; i < VE; ++i) f[i] = grad(f[i]);
                    dv[v] = VT::pack(f);
                }
                if (tid < edges) VT::store1(dx, edge, grad(VT::load1(x, edge)));
                // the token's element, after every thread's stores
                const float gt = grad(xt) + k0;
                __syncthreads();
                if (tid == 0) VT::store1(dx, t, gt);
            }
        }
        __syncthreads();  // `red`, and x where dx is x
    }
    if (OP != kRowLogp && a.reduction != kRedNone)
        rows_finish(a, sum, gridDim.x, blockIdx.x, red_d, &s_flag);
}

template <typename T, int OP>
const void* pick_ent(bool ent) {
    return ent ? (const void*)&rows_kernel<T, OP, true> : (const void*)&rows_kernel<T, OP, false>;
}

template <typename T>
const void* pick(int op, bool ent) {
    return op == kRowLogp     ? pick_ent<T, kRowLogp>(ent)
           : op == kRowPolicy ? pick_ent<T, kRowPolicy>(ent)
                              : (const void*)&rows_kernel<T, kRowDistill, false>;
}

}  // namespace

// Launches the forward of `op`; ent: entropies are formed.
ce_status rows_launch(int op, bool ent, int dtype, const RowArgs& args, int sms, cudaStream_t st) {
    RowArgs a = args;
    const void* fn = dtype == CE_F32    ? pick<float>(op, ent)
                     : dtype == CE_BF16 ? pick<__nv_bfloat16>(op, ent)
                                        : pick<__half>(op, ent);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(a.p.rows, 8L * sms));
    const size_t smem = a.teacher_lse ? static_cast<size_t>((a.p.V + 31) / 32 * 4) : 0;
    void* kargs[] = {&a};
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e == cudaSuccess)
        e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kargs, smem, st);
    return e == cudaSuccess ? CE_OK : record_cuda_failure(e, "token loss launch");
}

}  // namespace gbce
