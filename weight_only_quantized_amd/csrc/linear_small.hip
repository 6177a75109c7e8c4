// linear_small.hip — decode-sized products of the fused linear operators:
// y = act(x . W + bias) + residual and a = act(g) * u for a few rows.
//
// A workgroup owns NB 16-column blocks (GLU: NB / 2 gate blocks and the up
// blocks of the same columns) and all of K; its waves take the 128-row groups
// in turn (wave w: groups w, w + W, ...), so that at any moment they read
// consecutive kilobytes of each column block.
#include "act.hpp"

namespace w4 {

constexpr int small_waves(int mt) { return mt == 1 ? 16 : 8; }

template <int DT, bool GLU, int NB, int MT>
__global__ void __launch_bounds__(small_waves(MT) * 64) lin_small_kernel(const LinArgs p) {
    static_assert(!GLU || NB % 2 == 0, "gate and up blocks in pairs");
    constexpr int D = 2;                              // groups in flight per wave
    constexpr int WMAX = small_waves(MT);
    const int G = (int)(p.K / kGroup);
    const int W = blockDim.x >> 6;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, kc = lane >> 4;
    const int64_t half = p.cols / 2;
    const int64_t m0 = (int64_t)blockIdx.y * 16 * MT;
    // first column of block b
    auto col_of = [&](int b) -> int64_t {
        if constexpr (GLU) {
            const int64_t c = (int64_t)blockIdx.x * (8 * NB) + (b % (NB / 2)) * 16;
            return b < NB / 2 ? c : half + c;
        }
        return (int64_t)blockIdx.x * (16 * NB) + b * 16;
    };

    // rows past M read row M - 1; their results are not stored
    const uint16_t *xrow[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t r = m0 + 16 * mt + j < p.M ? m0 + 16 * mt + j : p.M - 1;
        xrow[mt] = p.a + r * p.lda + 32 * kc;
    }
    const uint8_t *wb[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wb[b] = p.wp + col_of(b) / 16 * G * kTileBytes + lane * 16;
    // lane l fetches the scale and zero point of column l % (16 NB); without
    // zero points the scale's own bytes are read and ignored
    const int64_t scol = col_of((lane & (16 * NB - 1)) >> 4) + j;
    const uint8_t *zp = p.zero ? p.zero : reinterpret_cast<const uint8_t *>(p.scale);

    u32x4_t xa[D][MT][4], wr[D][NB];
    uint32_t sr[D], zr[D];
    auto load = [&](int d, int g) {
        const int gc = g < G ? g : G - 1;
#pragma unroll
        for (int b = 0; b < NB; ++b) wr[d][b] = ld128(wb[b] + (int64_t)gc * kTileBytes);
        const int64_t so = (int64_t)(gc / p.gm) * p.N + scol;
        sr[d] = p.scale[so];
        zr[d] = zp[so >> 1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < 4; ++t) xa[d][mt][t] = ld128(xrow[mt] + (int64_t)gc * kGroup + 8 * t);
    };

    float yacc[NB][MT][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) yacc[b][mt][r] = 0.f;

    auto compute = [&](int d) {
        const uint32_t z = p.zero ? __builtin_amdgcn_ubfe(zr[d], (uint32_t)(j & 1) * 4u, 4) : 8u;
        const uint32_t sz = sr[d] | z << 16;
        // bf16: the operand is 128 + v; S = row sums of x take (128 + z) S out
        f32x4_t S[MT];
        if constexpr (DT == DT_BF16) {
            const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                S[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 4; ++t) S[mt] = mfma16x16x32<DT>(xa[d][mt][t], ones, S[mt]);
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * b + j) << 2, (int)sz);
            const uint32_t zb = v >> 16;
            f32x4_t acc[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const u32x4_t wq = dequant_word<DT>(wr[d][b][t], f16_negbias2(zb));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[mt] = mfma16x16x32<DT>(xa[d][mt][t], wq, acc[mt]);
            }
            const float s = h2f<DT>((uint16_t)(v & 0xFFFFu));
            const float nbias = -(128.f + (float)zb);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float a = acc[mt][r];
                    if constexpr (DT == DT_BF16) a = __builtin_fmaf(nbias, S[mt][r], a);
                    yacc[b][mt][r] = __builtin_fmaf(s, a, yacc[b][mt][r]);
                }
        }
    };

#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + d * W);
    for (int g = wave; g < G; g += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (g + d * W < G) compute(d);
            load(d, g + (d + D) * W);
        }
    }

    // ---- sums of the waves, in wave order, then the finishing step ----------------
    __shared__ float red[WMAX][NB][16 * MT][17];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][b][16 * mt + 4 * kc + r][j] = yacc[b][mt][r];
    __syncthreads();
    constexpr int OB = GLU ? NB / 2 : NB;
    for (int i = threadIdx.x; i < OB * 256 * MT; i += blockDim.x) {
        const int b = i / (256 * MT), r = (i >> 4) % (16 * MT), c = i & 15;
        const int64_t row = m0 + r;
        if (row >= p.M) continue;
        float v[1] = {0.f}, u[1] = {0.f};
        for (int w = 0; w < W; ++w) {
            v[0] += red[w][b][r][c];
            if constexpr (GLU) u[0] += red[w][b + NB / 2][r][c];
        }
        if constexpr (GLU) finish_glu<DT, 1>(p, v, u, row, col_of(b) + c);
        else finish_ep<DT, 1>(p, v, row, col_of(b) + c);
    }
}

bool lin_small_ok(int mode, int64_t M, int64_t K, int64_t N) {
    (void)K;
    (void)N;
    return mode != LIN_T && M <= 64;
}

template <int DT, bool GLU, int NB>
static hipError_t small_go(const LinArgs &p, hipStream_t stream) {
    const int mt = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
    const int64_t G = p.K / kGroup;
    const int waves = (int)(G < 8 ? G : 8);
    const dim3 grid((unsigned)(p.cols / (16 * NB)), (unsigned)((p.M + 16 * mt - 1) / (16 * mt))), block(waves * 64);
    if (mt == 1) {
        hipLaunchKernelGGL((lin_small_kernel<DT, GLU, NB, 1>), grid, block, 0, stream, p);
    } else if (mt == 2) {
        hipLaunchKernelGGL((lin_small_kernel<DT, GLU, NB, 2>), grid, block, 0, stream, p);
    } else {
        if constexpr (NB <= 2) hipLaunchKernelGGL((lin_small_kernel<DT, GLU, NB, 4>), grid, block, 0, stream, p);
        else return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT>
static hipError_t small_dt(int mode, const LinArgs &p, hipStream_t stream) {
    // fewer column blocks per workgroup where NB = 4 would leave compute units
    // without one
    const bool narrow = p.cols / 64 < 256 || p.M > 32;      // four 16-row tiles: NB = 4 does not fit in registers
    if (mode == LIN_GLU) return narrow ? small_go<DT, true, 2>(p, stream) : small_go<DT, true, 4>(p, stream);
    if (narrow) return p.cols / 32 < 256 ? small_go<DT, false, 1>(p, stream) : small_go<DT, false, 2>(p, stream);
    return small_go<DT, false, 4>(p, stream);
}

hipError_t launch_lin_small(int mode, const LinArgs &p, int dt, hipStream_t stream) {
    return dt == DT_BF16 ? small_dt<DT_BF16>(mode, p, stream) : small_dt<DT_F16>(mode, p, stream);
}

}  // namespace w4
