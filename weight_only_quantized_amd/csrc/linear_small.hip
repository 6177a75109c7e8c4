// linear_small.hip — decode kernel of the fused linear operators: up to 32 rows
// of y = act(x . W + bias) + residual or a = act(g) * u.
//
// A workgroup owns NB 16-column blocks (GLU: NB / 2 gate blocks and the up
// blocks of the same columns) and all of K or a slice of it; its waves take the
// 128-row groups in turn (wave w: groups w, w + W, ...), so that at any moment
// they read consecutive kilobytes of each column block.  Two groups are on the
// way per wave: NB 16-byte slots of W per lane, x straight in operand order,
// one scale and one zero point per lane (lane l those of column l % (16 NB),
// handed to the lane that needs them by a lane permute).  The waves' sums meet in
// LDS in wave order and every output is finished and rounded once.
//
// Codes enter the matrix core (16 x 16 x 32 steps, rows padded to 16 MT) as
// exact integers: fp16 as u - z, bf16 as 128 + u, the pattern that one byte
// permute makes; four more steps with ones give the row sums of x, and
// (128 + z) times them is subtracted in fp32.  The group's scale multiplies the
// fp32 sum.  An infinite x therefore gives NaN in its row.
//
// Bound: the weight stream at the start (latency) and through the launch.
// Measured (bf16, zero points): gated 4096 x 28672, one row 12.8 us (61 MB, 4.8
// TB/s, the rate of a large copy), 16 rows 14.7 us; 14336 x 4096, one row 8.1 us
// (3.8 TB/s).  More groups on the way and bounded buffer loads measured slower
// (8.7 -> 9.9 us and more for 14336 x 4096).
#include "act.hpp"

namespace w4 {

constexpr int kSmallWaves = 8;       // most waves per workgroup
constexpr int64_t kSmallMaxM = 32;   // rows of the decode kernel

template <int DT, bool GLU, int NB, int MT>
__global__ void __launch_bounds__(kSmallWaves * 64) lin_small_kernel(const LinArgs p) {
    static_assert(!GLU || NB % 2 == 0, "gate and up blocks in pairs");
    constexpr int D = 2;                              // groups in flight per wave
    const int W = blockDim.x >> 6;
    // this workgroup's groups: [g0, G)
    const int g0 = (int)blockIdx.y * p.stages, Gall = (int)(p.K / kGroup);
    const int G = g0 + p.stages < Gall ? g0 + p.stages : Gall;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, kc = lane >> 4;
    const int64_t half = p.cols / 2;
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
        const int64_t r = 16 * mt + j < p.M ? 16 * mt + j : p.M - 1;
        xrow[mt] = p.a + r * p.lda + 32 * kc;
    }
    const uint8_t *wb[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wb[b] = p.wp + col_of(b) / 16 * Gall * kTileBytes + lane * 16;
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
    for (int d = 0; d < D; ++d) load(d, g0 + wave + d * W);
    for (int g = g0 + wave; g < G; g += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (g + d * W < G) compute(d);
            load(d, g + (d + D) * W);
        }
    }

    // ---- sums of the waves, in wave order, then the finishing step ----------------
    __shared__ float red[kSmallWaves][NB][16 * MT][17];
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
        const int64_t row = r;
        if (row >= p.M) continue;
        float v[1] = {0.f}, u[1] = {0.f};
        for (int w = 0; w < W; ++w) {
            v[0] += red[w][b][r][c];
            if constexpr (GLU) u[0] += red[w][b + NB / 2][r][c];
        }
        if (p.slices > 1) {
            float *o = p.part + ((int64_t)blockIdx.y * p.M + row) * p.cols + col_of(b) + c;
            o[0] = v[0];
            if constexpr (GLU) o[half] = u[0];
            continue;
        }
        if constexpr (GLU) finish_glu<DT, 1>(p, v, u, row, col_of(b) + c);
        else finish_ep<DT, 1>(p, v, row, col_of(b) + c);
    }
}

// Column blocks per workgroup, waves, 16-row tiles and K slices of a call.
struct SmallPlan { int nb, waves, mt, slices, groups; };

// Widest workgroups that still give about one per compute unit.  Every
// workgroup reads all of x (16 mt rows), N K 2 mt / nb bytes in all through L2 at
// about 10 TB/s: beyond four rows it pays to take four column blocks and cut K
// into slices instead once that saves more than the join's 4 us (40 MB).
// Measured, M = 16: K 14336 x N 4096 17.9 -> 13.3 us, while 8192^2 would go from 12.2
// to 13.2 and 4096^2 from 6.9 to 8.1.  Four waves per workgroup once there are more
// workgroups than compute units and x is not a single tile's few rows (K 4096
// x N 28672, M = 32: 26.9 -> 23.9 us), else eight (M = 1: 13.2 against 13.7 us).
static SmallPlan small_plan(int mode, int64_t M, int64_t K, int64_t N) {
    SmallPlan s{};
    const int G = (int)(K / kGroup);
    s.mt = M <= 16 ? 1 : 2;
    s.nb = N / 64 >= 224 ? 4 : N / 32 >= 224 || mode == LIN_GLU ? 2 : 1;
    int64_t slices = 1;
    if (M > 4 && s.nb < 4 && 2 * s.mt * N * K / s.nb - 2 * s.mt * N * K / 4 > 40000000) {
        s.nb = 4;
        slices = 256 / (N / 64) < 1 ? 1 : 256 / (N / 64);
        if (slices > 8) slices = 8;
    }
    s.groups = (int)((G + slices - 1) / slices);
    s.slices = (G + s.groups - 1) / s.groups;
    s.waves = M <= 4 || N / (16 * s.nb) * s.slices <= 256 ? kSmallWaves : 4;
    if (s.waves > s.groups) s.waves = s.groups;
    return s;
}

bool lin_small_ok(int mode, int64_t M) { return mode != LIN_T && M <= kSmallMaxM; }

size_t lin_small_workspace_bytes(int mode, int64_t M, int64_t K, int64_t N) {
    const SmallPlan s = small_plan(mode, M, K, N);
    return s.slices > 1 ? (size_t)s.slices * (size_t)M * (size_t)N * sizeof(float) : 0;
}

template <int DT, bool GLU, int NB, int MT>
static hipError_t small_go(const LinArgs &p, const SmallPlan &s, hipStream_t stream) {
    const dim3 grid((unsigned)(p.cols / (16 * NB)), (unsigned)s.slices);
    hipLaunchKernelGGL((lin_small_kernel<DT, GLU, NB, MT>), grid, dim3((unsigned)s.waves * 64), 0, stream, p);
    return hipGetLastError();
}

template <int DT, bool GLU, int NB>
static hipError_t small_mt(const LinArgs &p, const SmallPlan &s, hipStream_t stream) {
    if (s.mt == 1) return small_go<DT, GLU, NB, 1>(p, s, stream);
    return small_go<DT, GLU, NB, 2>(p, s, stream);
}

template <int DT>
static hipError_t small_dt(int mode, const LinArgs &p, const SmallPlan &s, hipStream_t stream) {
    if (mode == LIN_GLU) {
        if (s.nb == 2) return small_mt<DT, true, 2>(p, s, stream);
        if (s.nb == 4) return small_mt<DT, true, 4>(p, s, stream);
    } else {
        if (s.nb == 1) return small_mt<DT, false, 1>(p, s, stream);
        if (s.nb == 2) return small_mt<DT, false, 2>(p, s, stream);
        if (s.nb == 4) return small_mt<DT, false, 4>(p, s, stream);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_lin_small(int mode, LinArgs p, int dt, void *workspace, hipStream_t stream) {
    const SmallPlan s = small_plan(mode, p.M, p.K, p.N);
    p.slices = s.slices;
    p.stages = s.groups;
    p.part = (float *)workspace;
    hipError_t err = dt == DT_BF16 ? small_dt<DT_BF16>(mode, p, s, stream) : small_dt<DT_F16>(mode, p, s, stream);
    return err == hipSuccess && p.slices > 1 ? launch_lin_join(mode, p, dt, stream) : err;
}

}  // namespace w4
