// route.hip — the router of the MoE chain: top-k experts of every token with
// their softmax weights, per-expert counts and the balance loss; and the
// gradient of the weights and of the loss through the logits.
//
//   p_t = softmax(z_t);  ids = the topk largest logits (ties: lowest index)
//   w_k = p at ids, or those divided by their sum (renormalized)
//   loss = E sum_e (c_e / C) (1 / Tv) sum_t p_te,  c counts, C their sum, Tv tokens
//
//   dz_te = sum_{k: id = e} w_k (dw_k - sum_j w_j dw_j)            (renormalized)
//         + p_te (h_te - sum_j p_tj h_tj),
//   h_te  = dloss (E c_e - C) / (C Tv) + sum_{k: id = e} dw_k      (not renormalized)
// The loss's part of h is E c_e / (C Tv) less a constant, which a softmax's
// gradient ignores: E c_e - C is an integer, so no digits cancel.
//
// A group of LPT lanes owns a token; lane `sub` holds experts sub, sub + LPT, ...
#include "common.hpp"
#include "launch.hpp"

namespace w4 {

enum { DT_F32 = 2 };

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (DT == DT_F32) return static_cast<const float *>(p)[i];
    else return h2f<DT>(static_cast<const uint16_t *>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float v) {
    if constexpr (DT == DT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<uint16_t *>(p)[i] = f2h<DT>(v);
}

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

// What a token's logits are good for: a distribution, nothing (every logit
// -inf), or NaN (a NaN or +inf among them).
enum { ROW_OK = 0, ROW_EMPTY = 1, ROW_NAN = 2 };

// exp(z - max) in place of z, their sum, and the row's kind.
template <int LPT, int EPL>
__device__ __forceinline__ int row_softmax(float (&z)[EPL], float (&p)[EPL], float &top, float &sum) {
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        m = fmaxf(m, z[i]);
        nan |= z[i] != z[i];
    }
    top = group_max<LPT>(m);
    const bool any_nan = group_max<LPT>(nan ? 1.0f : 0.0f) > 0.0f;
    const int kind = any_nan || top == INFINITY ? ROW_NAN : top == -INFINITY ? ROW_EMPTY : ROW_OK;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = kind == ROW_OK ? expf(z[i] - top) : kind == ROW_NAN ? __builtin_nanf("") : 0.0f;
        s += p[i];
    }
    sum = group_sum<LPT>(s);
    return kind;
}

constexpr int kRouteThreads = 256;

template <int DT, int LPT, int EPL>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(RouteArgs p, float *__restrict__ part_p, int32_t *__restrict__ part_c) {
    constexpr int TPB = kRouteThreads / LPT;
    __shared__ int cnt[kMoeMaxExperts + 1];
    __shared__ float psum[kRouteThreads / 64][kMoeMaxExperts];
    const int E = p.E, tid = threadIdx.x, sub = tid % LPT;
    if (part_c) {
        for (int e = tid; e <= E; e += kRouteThreads) cnt[e] = 0;
        __syncthreads();
    }
    float pacc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) pacc[i] = 0.0f;

    for (int64_t t = (int64_t)blockIdx.x * TPB + tid / LPT; t < p.T; t += (int64_t)gridDim.x * TPB) {
        int32_t *ids = p.ids + t * p.topk;
        float *w = p.w + t * p.topk;
        const bool live = !p.mask || p.mask[t] != 0;
        float z[EPL], pe[EPL], top = 0.0f, sum = 1.0f;
        int kind = ROW_EMPTY;
        if (live) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * LPT + sub;
                z[i] = e < E ? load_logit<DT>(p.logits, t * p.ld + e) : -INFINITY;
            }
            kind = row_softmax<LPT, EPL>(z, pe, top, sum);
        }
        if (kind != ROW_OK) {
            const float fill = kind == ROW_NAN ? __builtin_nanf("") : 0.0f;
            for (int k = sub; k < p.topk; k += LPT) {
                ids[k] = -1;
                w[k] = fill;
            }
            if (kind == ROW_NAN && part_c) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) pacc[i] = __builtin_nanf("");
                if (sub == 0) atomicAdd(&cnt[E], 1);
            }
            continue;
        }
        const float inv = 1.0f / sum;
        if (part_c) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) pacc[i] += pe[i] * inv;
            if (sub == 0) atomicAdd(&cnt[E], 1);
        }
        // the largest that is left, topk times
        float chosen = 0.0f;
        for (int k = 0; k < p.topk; ++k) {
            float bv = -INFINITY;
            int be = 1 << 30;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (z[i] > bv) {
                    bv = z[i];
                    be = i * LPT + sub;
                }
#pragma unroll
            for (int off = LPT / 2; off > 0; off >>= 1) {
                const float ov = __shfl_xor(bv, off);
                const int oe = __shfl_xor(be, off);
                if (ov > bv || (ov == bv && oe < be)) {
                    bv = ov;
                    be = oe;
                }
            }
            const bool none = bv == -INFINITY;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (be == i * LPT + sub) z[i] = -INFINITY;
            const float ex = none ? 0.0f : expf(bv - top);
            chosen += ex;
            if (sub == k % LPT) {
                ids[k] = none ? -1 : be;
                w[k] = p.renorm ? ex : ex * inv;
                if (part_c && !none) atomicAdd(&cnt[be], 1);
            }
        }
        if (p.renorm) {
            for (int k = sub; k < p.topk; k += LPT) w[k] = w[k] / chosen;      // each lane its own values
        }
    }
    if (!part_c) return;
    // sum over the token groups of a wave, then over the waves
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        float v = pacc[i];
#pragma unroll
        for (int off = LPT; off < 64; off <<= 1) v += __shfl_xor(v, off);
        const int e = i * LPT + sub;
        if ((tid & 63) < LPT && e < E) psum[tid >> 6][e] = v;
    }
    __syncthreads();
    for (int e = tid; e <= E; e += kRouteThreads) {
        part_c[(int64_t)blockIdx.x * (E + 1) + e] = cnt[e];
        if (e < E) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kRouteThreads / 64; ++w) v += psum[w][e];
            part_p[(int64_t)blockIdx.x * E + e] = v;
        }
    }
}

// Counts and loss from the blocks' partial sums, in a fixed order.
__global__ void __launch_bounds__(1024)
route_join_kernel(const float *__restrict__ part_p, const int32_t *__restrict__ part_c, int blocks, int E,
                  int32_t *__restrict__ counts, float *__restrict__ loss) {
    const int e = threadIdx.x;
    __shared__ double num[16];
    __shared__ long long den[16];
    __shared__ int tokens;
    int c = 0;
    double ps = 0.0;
    for (int b = 0; b < blocks && e < E; ++b) {
        c += part_c[(int64_t)b * (E + 1) + e];
        ps += part_p[(int64_t)b * E + e];
    }
    if (e < E) counts[e] = c;
    if (e == 0) {
        int tv = 0;
        for (int b = 0; b < blocks; ++b) tv += part_c[(int64_t)b * (E + 1) + E];
        counts[E] = tv;
        tokens = tv;
    }
    double x = c * ps;
    long long n = c;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        x += __shfl_xor(x, off);
        n += __shfl_xor(n, off);
    }
    if ((e & 63) == 0) {
        num[e >> 6] = x;
        den[e >> 6] = n;
    }
    __syncthreads();
    if (e == 0 && loss) {
        x = 0.0;
        n = 0;
        for (int w = 0; w < 16; ++w) {
            x += num[w];
            n += den[w];
        }
        const double tv = tokens > 0 ? tokens : 1, cc = n > 0 ? (double)n : 1.0;
        *loss = (float)(E * x / (cc * tv));
    }
}

template <int DT, int LPT, int EPL>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteArgs p) {
    constexpr int TPB = kRouteThreads / LPT;
    const int E = p.E, tid = threadIdx.x, sub = tid % LPT;
    // the loss's part of h
    float h0[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) h0[i] = 0.0f;
    if (p.dloss) {
        long long C = 0;
        for (int e = tid & 63; e < E; e += 64) C += p.counts[e];
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) C += __shfl_xor(C, off);
        const int tv = p.counts[E];
        const float f = C > 0 && tv > 0 ? (float)((double)*p.dloss / ((double)C * tv)) : 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * LPT + sub;
            if (e < E) h0[i] = f * (float)((long long)E * p.counts[e] - C);
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * TPB + tid / LPT; t < p.T; t += (int64_t)gridDim.x * TPB) {
        const bool live = !p.mask || p.mask[t] != 0;
        float z[EPL], pe[EPL], sel[EPL], top = 0.0f, sum = 1.0f;
        int kind = ROW_EMPTY;
        if (live) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * LPT + sub;
                z[i] = e < E ? load_logit<DT>(p.logits, t * p.ld + e) : -INFINITY;
            }
            kind = row_softmax<LPT, EPL>(z, pe, top, sum);
        }
        if (kind != ROW_OK) {
            const float fill = kind == ROW_NAN ? __builtin_nanf("") : 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * LPT + sub;
                if (e < E) store_logit<DT>(p.dlogits, t * p.ldd + e, fill);
            }
            continue;
        }
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sel[i] = 0.0f;
        if (p.dw) {
            const int32_t *ids = p.ids + t * p.topk;
            const float *w = p.w + t * p.topk, *dw = p.dw + t * p.topk;
            float mean = 0.0f;
            if (p.renorm)
                for (int k = 0; k < p.topk; ++k) mean += ids[k] >= 0 ? w[k] * dw[k] : 0.0f;
            for (int k = 0; k < p.topk; ++k) {
                const int id = ids[k];
                const float v = p.renorm ? w[k] * (dw[k] - mean) : dw[k];
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (id == i * LPT + sub) sel[i] += v;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            pe[i] *= inv;
            z[i] = h0[i] + (p.renorm ? 0.0f : sel[i]);
            dot += pe[i] * z[i];
        }
        dot = group_sum<LPT>(dot);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * LPT + sub;
            const float v = pe[i] * (z[i] - dot) + (p.renorm ? sel[i] : 0.0f);
            if (e < E) store_logit<DT>(p.dlogits, t * p.ldd + e, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
static int64_t route_blocks(int64_t T, int) {
    const int64_t b = (T + 3) / 4;
    return b < 256 ? b : 256;
}

size_t route_workspace_bytes(int64_t T, int64_t E) {
    return (size_t)route_blocks(T, (int)E) * (size_t)(2 * E + 1) * 4;
}

template <int DT, int EPL>
static hipError_t route_launch(const RouteArgs &p, void *workspace, hipStream_t stream) {
    const int64_t nb = route_blocks(p.T, p.E);
    float *pp = p.counts ? (float *)workspace : nullptr;
    int32_t *pc = p.counts ? (int32_t *)workspace + nb * p.E : nullptr;
    if (nb > 0)
        hipLaunchKernelGGL((route_kernel<DT, 64, EPL>), dim3((unsigned)nb), dim3(kRouteThreads), 0, stream, p, pp, pc);
    if (p.counts)
        hipLaunchKernelGGL(route_join_kernel, dim3(1), dim3(1024), 0, stream, pp, pc, (int)nb, p.E, p.counts, p.loss);
    return hipGetLastError();
}

template <int DT, int EPL>
static hipError_t route_backward_launch(const RouteArgs &p, hipStream_t stream) {
    const int64_t b = (p.T + 3) / 4;
    hipLaunchKernelGGL((route_backward_kernel<DT, 64, EPL>), dim3((unsigned)(b < 4096 ? b : 4096)), dim3(kRouteThreads),
                       0, stream, p);
    return hipGetLastError();
}

#define W4_ROUTE_EPL(F, ...)                    \
    (p.E <= 64    ? F<DT, 1>(__VA_ARGS__)       \
     : p.E <= 128 ? F<DT, 2>(__VA_ARGS__)       \
     : p.E <= 256 ? F<DT, 4>(__VA_ARGS__)       \
     : p.E <= 512 ? F<DT, 8>(__VA_ARGS__)       \
                  : F<DT, 16>(__VA_ARGS__))

template <int DT>
static hipError_t route_dt(const RouteArgs &p, void *workspace, hipStream_t stream) {
    return W4_ROUTE_EPL(route_launch, p, workspace, stream);
}
template <int DT>
static hipError_t route_backward_dt(const RouteArgs &p, hipStream_t stream) {
    return W4_ROUTE_EPL(route_backward_launch, p, stream);
}

hipError_t launch_route(const RouteArgs &p, int dt, void *workspace, hipStream_t stream) {
    if (dt == DT_F32) return route_dt<DT_F32>(p, workspace, stream);
    return dt == DT_BF16 ? route_dt<DT_BF16>(p, workspace, stream) : route_dt<DT_F16>(p, workspace, stream);
}

hipError_t launch_route_backward(const RouteArgs &p, int dt, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    if (dt == DT_F32) return route_backward_dt<DT_F32>(p, stream);
    return dt == DT_BF16 ? route_backward_dt<DT_BF16>(p, stream) : route_backward_dt<DT_F16>(p, stream);
}

}  // namespace w4
