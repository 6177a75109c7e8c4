// act.hpp — activations of the fused linear operators and what their kernels
// share: the finishing step (bias, activation, gated product, residual) applied
// to fp32 sums before the one rounding to the activation dtype, and LDS helpers.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace w4 {

// Two of the four codes (one per byte, 0..15) of m in fp32: bytes 0, 1 or 2, 3.  As an
// 8-bit float (4 exponent bits, 3 of mantissa) a byte u < 16 is u 2^-9 exactly, so
// one conversion with the factor 2^9 gives two codes (a byte conversion each:
// 2% more time of every bf16 tile product, 819 against 804 us for gated 4096 x 4096
// x 28672).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
// The factor may hold another power of two on top.
template <int HALF>
__device__ __forceinline__ f32x2_t codes_f32(uint32_t m, float f = 512.0f) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(m, f, HALF != 0);
}

// e^x by the hardware's base-2 exponential.  The argument's rounding costs
// |x| 2^-24 relative, far below the 16-bit rounding of every result.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// 1 / (1 + e^-x); e^-x = inf gives exactly 0.
__device__ __forceinline__ float sigmoid_fast(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x)); }

// The normal distribution's cumulative function (1 + erf(v / sqrt 2)) / 2, relative to its
// own size in the lower tail too, where GELU's result and a gated product live on it.
// erfc(x) = P(t) e^(-x^2), t = 1 / (1 + 3 x / 8): P is the polynomial of degree 7 without a
// constant term whose largest relative error from erfcx(x) = erfc(x) e^(x^2) on 0 <= x <= 9.4 is
// the smallest (a linear programme over 1500 points), 6.3e-7.  With fp32 steps and the
// exponent's rounding the result is off by 1e-6 at most around 0, 5e-6 down to v = -6
// and 2e-5 at -13, far below half a unit of 16 bits.  Free of branches (the library
// erff's two ranges diverge: it added 7 to 16 us to a 333 x 2816 epilogue).
__device__ __forceinline__ float normal_cdf(float v) {
    const float x = __builtin_fabsf(v) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.375f, x, 1.0f));
    float q = __builtin_fmaf(-0.13506828f, t, 0.38783652f);
    q = __builtin_fmaf(q, t, -0.12944822f);
    q = __builtin_fmaf(q, t, 0.2829496f);
    q = __builtin_fmaf(q, t, 0.1667095f);
    q = __builtin_fmaf(q, t, 0.2156801f);
    q = __builtin_fmaf(q, t, 0.21134017f);
    q = 0.5f * q * t * exp_fast(-x * x);
    return v < 0.f ? q : 1.0f - q;
}

constexpr float kGeluC0 = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluC1 = 0.044715f;

// act(v).  GELU_TANH uses (1 + tanh(y)) / 2 = sigmoid(2 y).
template <int V>
__device__ __forceinline__ void act_fwd(float (&v)[V], int act) {
    if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];     // keeps NaN
    } else if (act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid_fast(v[i]);
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= normal_cdf(v[i]);
    } else if (act == ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] *= sigmoid_fast(2.0f * kGeluC0 * (v[i] + kGeluC1 * v[i] * v[i] * v[i]));
    }
}

// f = act(v), d = act'(v) (0 at v = 0 for RELU).
__device__ __forceinline__ void act_both(float v, int act, float &f, float &d) {
    f = v;
    d = 1.f;
    if (act == ACT_RELU) {
        f = v < 0.f ? 0.f : v;
        d = v > 0.f ? 1.f : (v <= 0.f ? 0.f : v);                       // NaN stays NaN
    } else if (act == ACT_SILU) {
        const float s = sigmoid_fast(v);
        f = v * s;
        d = s * (1.0f + v * (1.0f - s));
    } else if (act == ACT_GELU) {
        const float cdf = normal_cdf(v);
        f = v * cdf;
        d = cdf + v * exp_fast(-0.5f * v * v) * 0.39894228040143268f;      // 1 / sqrt(2 pi)
    } else if (act == ACT_GELU_TANH) {
        // |v| > 30: the sigmoid is exactly 0 or 1 long before, and the
        // clamped polynomial cannot overflow (NaN passes both comparisons)
        const float c = v > 30.f ? 30.f : (v < -30.f ? -30.f : v);
        const float s = sigmoid_fast(2.0f * kGeluC0 * (c + kGeluC1 * c * c * c));
        f = v * s;
        d = s + c * s * (1.0f - s) * 2.0f * kGeluC0 * (1.0f + 3.0f * kGeluC1 * c * c);
    }
}

// V consecutive 16-bit values to and from fp32.  V = 8 is one 16-byte access.
template <int DT, int V>
__device__ __forceinline__ void load_vec(const uint16_t *p, float (&v)[V]) {
    if constexpr (V == 8) {
        const u32x4_t w = ld128(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t word = w[q];
            v[2 * q] = h2f<DT>((uint16_t)(word & 0xFFFFu));
            v[2 * q + 1] = h2f<DT>((uint16_t)(word >> 16));
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = h2f<DT>(p[i]);
    }
}
template <int DT, int V>
__device__ __forceinline__ void store_vec(uint16_t *p, const float (&v)[V]) {
    if constexpr (V == 8) {
        u32x4_t w;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = (uint32_t)f2h<DT>(v[2 * q]) | (uint32_t)f2h<DT>(v[2 * q + 1]) << 16;
        *reinterpret_cast<u32x4_t *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = f2h<DT>(v[i]);
    }
}

// y = act(v + bias) + residual for V columns of one row; pre gets v + bias.
template <int DT, int V>
__device__ __forceinline__ void finish_ep(const LinArgs &p, float (&v)[V], int64_t row, int64_t col) {
    if (p.bias) {
        float b[V];
        load_vec<DT, V>(p.bias + col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b[i];
    }
    if (p.pre) store_vec<DT, V>(p.pre + row * p.cols + col, v);
    act_fwd<V>(v, p.act);
    if (p.res) {
        float r[V];
        load_vec<DT, V>(p.res + row * p.ldr + col, r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += r[i];
    }
    store_vec<DT, V>(p.y + row * p.ldy + col, v);
}

// a = act(g + bias_g) * (u + bias_u) for V of the I = cols / 2 columns of one
// row; pre gets both biased sums (the gate half first).
template <int DT, int V>
__device__ __forceinline__ void finish_glu(const LinArgs &p, float (&g)[V], float (&u)[V], int64_t row, int64_t col) {
    const int64_t I = p.cols / 2;
    if (p.bias) {
        float b[V];
        load_vec<DT, V>(p.bias + col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += b[i];
        load_vec<DT, V>(p.bias + I + col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] += b[i];
    }
    if (p.pre) {
        store_vec<DT, V>(p.pre + row * p.cols + col, g);
        store_vec<DT, V>(p.pre + row * p.cols + I + col, u);
    }
    act_fwd<V>(g, p.act);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] *= u[i];
    store_vec<DT, V>(p.y + row * p.ldy + col, g);
}

typedef short v4s_t __attribute__((__vector_size__(8)));
typedef v4s_t __attribute__((address_space(3))) *lds_v4s_ptr;

// Four 16-bit elements of one column from four LDS rows: the 16 lanes of a
// group read 4 rows x 16 columns (lane 4 r + c addresses row r, columns 4 c ..)
// and lane i gets column i.
__device__ __forceinline__ u32x2_t lds_tr16(const uint8_t *p) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_ptr)(v4s_t *)(uint8_t *)p));
}

// Orders LDS accesses of one wave for the compiler (the hardware keeps a wave's
// LDS operations in order): lanes exchange values through wave-private LDS.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// colsum[c] = sum over the row blocks' partial sums of 64 columns: each wave of
// the workgroup takes a contiguous share of the blocks, and the waves' sums meet
// in LDS (64 floats per wave) in order.
__device__ __forceinline__ void colsum_body(const float *part, float *colsum, int64_t N, int blocks, int64_t c0,
                                            float *red) {
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, nw = blockDim.x >> 6;
    const int64_t c = c0 + tx;                         // N is a multiple of 64
    const int per = (blocks + nw - 1) / nw, b0 = ty * per, b1 = b0 + per < blocks ? b0 + per : blocks;
    float s = 0.f;
    for (int b = b0; b < b1; ++b) s += part[(int64_t)b * N + c];
    red[ty * 64 + tx] = s;
    __syncthreads();
    if (ty == 0) {
        for (int y = 1; y < nw; ++y) s += red[y * 64 + tx];
        colsum[c] = s;
    }
}

}  // namespace w4
