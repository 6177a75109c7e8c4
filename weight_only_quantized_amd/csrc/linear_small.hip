// linear_small.hip — decode kernels of the fused linear operators: up to 32 rows
// of y = act(x . W + bias) + residual or a = act(g) * u, and of d . W^T.
//
// Forward (lin_small_kernel): a workgroup owns NB 16-column blocks (GLU: NB / 2 gate blocks and the up
// blocks of the same columns) and all of K or a slice of it; its waves take the
// 128-row groups in turn (wave w: groups w, w + W, ...), so that at any moment
// they read consecutive kilobytes of each column block.  Two groups are on the
// way per wave: NB 16-byte slots of W per lane, x straight in operand order,
// one scale and one zero point per lane (lane l those of column l % (16 NB),
// handed to the lane that needs them by a lane permute).  The waves' sums meet in
// LDS in wave order and every output is finished and rounded once.  More than 16
// MT rows of a small matrix lie as further row groups on the grid.
//
// Codes enter the matrix core (16 x 16 x 32 steps, rows padded to 16 MT) exactly:
// fp16 as u - z, bf16 as (128 + u) 2^-16, a pattern that one byte permute makes; four
// more steps with 2^-16 give the row sums of x, and (128 + z) times them is
// subtracted in fp32.  That small, both sums stay finite for any finite x (with 128 + u
// itself they passed fp32's range from x = 2e34 on, and their difference was NaN).
// The group's scale multiplies the difference; 2^8 of the factor comes back with
// it and 2^8 with the result, so that neither a scale below 2^120 nor a normal result
// leaves the range.  An infinite x gives NaN in its row.
//
// Bound: the weight stream at the start (latency) and through the launch.
// Measured (bf16, zero points): gated 4096 x 28672, one row 12.8 us (61 MB, 4.8
// TB/s, the rate of a large copy), 16 rows 14.7 us; 14336 x 4096, one row 8.3 us
// (3.7 TB/s).  More groups on the way and bounded buffer loads measured slower
// (8.7 -> 9.9 us and more for 14336 x 4096).
#include "act.hpp"

namespace w4 {

constexpr int kSmallWaves = 8;       // most waves per workgroup
// Rows up to which the forward decode kernel always runs: within 3% of the tile kernel or
// faster on nine matrices (32 rows: 4096^2 11.3 against 11.8 us, 1024^2 5.5 against 7.7, gated 4096 x
// 28672 23.8 against 23.1).
constexpr int64_t kSmallMaxM = 32;
constexpr int64_t kSmallGroupsM = 512;

// A byte offset past the end of every buffer (at most 2^31 bytes).
constexpr uint32_t kPast = 0xFFFFFF00u;
__device__ __forceinline__ u32x4_t buffer_ld128(__amdgpu_buffer_rsrc_t buf, uint32_t off) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(buf, (int)off, 0, 0));
}

// The 8 codes of a prepacked word as the kernel's operand: u - z, or (128 + u) 2^-16 (see
// dequant_word, whose bf16 pattern this is under another exponent byte).
template <int DT>
__device__ __forceinline__ u32x4_t small_operand(uint32_t w, uint32_t z) {
    if constexpr (DT == DT_F16) return dequant_word<DT>(w, f16_negbias2(z));
    constexpr uint32_t expb = 0x3B3B3B3Bu;
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    return u32x4_t{__builtin_amdgcn_perm(expb, lo, 0x04020400u), __builtin_amdgcn_perm(expb, hi, 0x04020400u),
                   __builtin_amdgcn_perm(expb, lo, 0x04030401u), __builtin_amdgcn_perm(expb, hi, 0x04030401u)};
}

template <int DT, bool GLU, int NB, int MT>
__global__ void __launch_bounds__(kSmallWaves * 64) lin_small_kernel(const LinArgs p) {
    static_assert(!GLU || NB % 2 == 0, "gate and up blocks in pairs");
    constexpr int D = 2;                              // groups in flight per wave
    constexpr float back = DT == DT_BF16 ? 256.f : 1.f;       // half of the operand's 2^-16
    const int W = blockDim.x >> 6;
    // this workgroup's groups: [g0, G)
    const int g0 = (int)blockIdx.y * p.stages, Gall = (int)(p.K / kGroup);
    const int G = g0 + p.stages < Gall ? g0 + p.stages : Gall;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, kc = lane >> 4;
    const int64_t half = p.cols / 2;
    const int64_t m0 = (int64_t)blockIdx.z * (16 * MT), rows = p.M - m0;       // this workgroup's rows
    const uint16_t *const a = p.a + m0 * p.lda;
    // first column of block b
    auto col_of = [&](int b) -> int64_t {
        if constexpr (GLU) {
            const int64_t c = (int64_t)blockIdx.x * (8 * NB) + (b % (NB / 2)) * 16;
            return b < NB / 2 ? c : half + c;
        }
        return (int64_t)blockIdx.x * (16 * NB) + b * 16;
    };

    // Rows past M and groups past the end: with one row tile they read row M - 1
    // and the last group again (few lines, in L2); with two, where that would be
    // many lines, they are requested past the end of x's buffer, which gives zeros
    // without a memory access (M = 32: 1024^2 7.4 -> 5.5 us, 4096^2 12.6 -> 11.6;
    // one row 8.7 -> 10.1 us for 14336 x 4096 if x and W did so).
    const __amdgpu_buffer_rsrc_t xbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(a), (short)0, (int)((((rows < 16 * MT ? rows : 16 * MT) - 1) * p.lda + p.K) * 2), 0x00020000);
    uint32_t xoff[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        xoff[mt] = 16 * mt + j < rows ? (uint32_t)((16 * mt + j) * p.lda + 32 * kc) * 2u : kPast;
    const uint16_t *const xrow = a + (j < rows ? j : rows - 1) * p.lda + 32 * kc;
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
        if constexpr (MT == 1) {
#pragma unroll
            for (int t = 0; t < 4; ++t) xa[d][0][t] = ld128(xrow + (int64_t)gc * kGroup + 8 * t);
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint32_t xo = g < G && xoff[mt] != kPast ? xoff[mt] + g * (kGroup * 2) : kPast;
#pragma unroll
                for (int t = 0; t < 4; ++t) xa[d][mt][t] = buffer_ld128(xbuf, xo + 16 * t);
            }
        }
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
        // bf16: S = 2^-16 of the row sums of x take (128 + z) S out
        f32x4_t S[MT];
        if constexpr (DT == DT_BF16) {
            const u32x4_t part = {0x37803780u, 0x37803780u, 0x37803780u, 0x37803780u};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                S[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 4; ++t) S[mt] = mfma16x16x32<DT>(xa[d][mt][t], part, S[mt]);
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
                const u32x4_t wq = small_operand<DT>(wr[d][b][t], zb);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[mt] = mfma16x16x32<DT>(xa[d][mt][t], wq, acc[mt]);
            }
            const float s = h2f<DT>((uint16_t)(v & 0xFFFFu)) * back;
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
        if (r >= rows) continue;
        const int64_t row = m0 + r;
        float v[1] = {0.f}, u[1] = {0.f};
        for (int w = 0; w < W; ++w) {
            v[0] += red[w][b][r][c];
            if constexpr (GLU) u[0] += red[w][b + NB / 2][r][c];
        }
        v[0] *= back;
        u[0] *= back;
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

// Transposed product for a few rows: y [M][K] = d . W^T (+ addend), 32 rows per
// workgroup.
//
// A workgroup owns 32 output columns (one 32-row chunk of a 128-row group) and all
// of N or a slice of it; its waves take blocks of 64 columns of W in turn.  Per
// block a lane dequantizes 32 codes of one column to (u - z) s in the activation
// dtype, the wave writes them as rows [n][32 k] of its own 4 KB of LDS and reads
// them back transposed as the matrix-core operand (32 x 32 x 16 steps, rows of d
// padded to 32); no barrier until the waves' sums meet in LDS in wave order.
// 16-byte chunk c of row n sits at chunk c ^ (n / 2 % 4): writes of 8 rows at one
// chunk and reads of 4 whole rows both touch different banks.
//
// Every workgroup reads all of d: K / 32 times M N 2 bytes, which bounds it for
// many rows of large matrices; the weights' stream and the launch otherwise.
// Measured (bf16, graph replay; the tile kernel with its best slices behind it): one row of
// 1024^2 5.9 (7.9) us, of 4096^2 8.5 (11.2), of 14336 x 1024 10.8 (9.4), of 4096 x 28672 28.5
// (28.7); 32 rows 7.2 (8.6), 13.7 (12.5), 14.0 (10.1), 60 (30).
constexpr int kSmallTWaves = 16;

template <int DT>
__global__ void __launch_bounds__(kSmallTWaves * 64) lin_small_t_kernel(const LinArgs p) {
    constexpr int D = 3;                              // blocks of 64 columns in flight per wave
    const int W = blockDim.x >> 6;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, qq = lane >> 4;
    // 4 KB per wave for the operand; the sums use the same memory at the end
    __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallTWaves * 32 * 33 * 4];
    static_assert(32 * 33 * 4 >= 4096, "operand fits in a wave's share");
    if (blockIdx.x >= p.K / 32) {
        // workgroups past the product's: the bias gradient, 64 columns each
        if (blockIdx.y == 0 && blockIdx.z == 0)
            colsum_body(p.cpart, p.colsum, p.N, p.cblocks, (int64_t)(blockIdx.x - p.K / 32) * 64,
                        reinterpret_cast<float *>(lds));
        return;
    }
    const int64_t G = p.K / kGroup, g = blockIdx.x >> 2;
    const int c = blockIdx.x & 3;
    const int64_t m0 = (int64_t)blockIdx.z * 32, rows = p.M - m0 < 32 ? p.M - m0 : 32;   // this workgroup's rows
    // this workgroup's blocks: [b0, b1)
    const int b0 = (int)blockIdx.y * p.stages, nblk = (int)(p.N / 64);
    const int b1 = b0 + p.stages < nblk ? b0 + p.stages : nblk;

    // Rows of d past M and blocks past the end are requested past the end of its
    // buffer: zeros, without a memory access or a branch around the load (M = 32,
    // 1024^2: 11.9 us with clamped loads, 7.2 so)
    const __amdgpu_buffer_rsrc_t abuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(p.a + m0 * p.lda), (short)0, (int)(((rows - 1) * p.lda + p.N) * 2), 0x00020000);
    const uint32_t aoff = (lane & 31) < rows ? (uint32_t)((lane & 31) * p.lda + 8 * (lane >> 5)) * 2u : kPast;
    const uint8_t *const wbase = p.wp + (qq * G + g) * kTileBytes + c * 256 + j * 16;
    const int64_t srow = g / p.gm * p.N + qq * 16 + j;
    const uint8_t *const zbase = p.zero ? p.zero : reinterpret_cast<const uint8_t *>(p.scale);

    u32x4_t wr[D], ar[D][4];
    uint32_t sr[D], zr[D];
    auto load = [&](int d, int b) {
        const bool in = b < b1;
        const int64_t bc = in ? b : b1 - 1;
        wr[d] = ld128(wbase + bc * (4 * G * kTileBytes));
        const int64_t so = srow + bc * 64;
        sr[d] = p.scale[so];
        zr[d] = zbase[so >> 1];
        const uint32_t ao = in && aoff != kPast ? aoff + b * 128 : kPast;
#pragma unroll
        for (int t = 0; t < 4; ++t) ar[d][t] = buffer_ld128(abuf, ao + 32 * t);
    };

    uint8_t *const mine = lds + wave * (32 * 33 * 4);
    const int n = 16 * qq + j;                        // this lane's column of the block
    uint8_t *const dst = mine + n * 64;
    const int wkey = (n >> 1) & 3;
    // transposing reads: rows 8 (lane / 32) + 4 h + lane % 16 / 4 of step t
    const int tr = (lane & 15) >> 2, tc = lane & 3, ch = 2 * (qq & 1) + (tc >> 1);
    const uint8_t *src[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 8 * (qq >> 1) + 4 * h + tr;
        src[h] = mine + row * 64 + ((ch ^ ((row >> 1) & 3)) << 4) + (tc & 1) * 8;
    }

    f32x16_t acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    auto compute = [&](int d) {
        const uint32_t z = p.zero ? __builtin_amdgcn_ubfe(zr[d], (uint32_t)(j & 1) * 4u, 4) : 8u;
        const float s = h2f<DT>((uint16_t)sr[d]), zs = -(float)z * s;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u32x4_t o;
            if constexpr (DT == DT_BF16) {
                const uint32_t w = wr[d][t];
                const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
                const f32x2_t c04 = codes_f32<0>(lo), c15 = codes_f32<1>(lo), c26 = codes_f32<0>(hi), c37 = codes_f32<1>(hi);
                float v[8] = {c04[0], c15[0], c26[0], c37[0], c04[1], c15[1], c26[1], c37[1]};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], s, zs);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bf16x2_t b = {(__bf16)v[2 * q], (__bf16)v[2 * q + 1]};
                    o[q] = __builtin_bit_cast(uint32_t, b);
                }
            } else {
                o = dequant_word<DT>(wr[d][t], f16_negbias2(z));
                const _Float16 m = (_Float16)s;
                const f16x2_t m2 = {m, m};
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, as<f16x2_t>(o[i]) * m2);
            }
            *reinterpret_cast<u32x4_t *>(dst + ((t ^ wkey) << 4)) = o;
        }
        wave_lds_sync();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const u32x2_t x0 = lds_tr16(src[0] + t * 16 * 64), x1 = lds_tr16(src[1] + t * 16 * 64);
            acc = mfma32x32x16<DT>(ar[d][t], u32x4_t{x0[0], x0[1], x1[0], x1[1]}, acc);
        }
        wave_lds_sync();
    };

#pragma unroll
    for (int d = 0; d < D; ++d) load(d, b0 + wave + d * W);
    for (int b = b0 + wave; b < b1; b += D * W) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (b + d * W < b1) compute(d);
            load(d, b + (d + D) * W);
        }
    }

    // ---- sums of the waves, in wave order, then the finishing step ----------------
    float *const red = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int i = 0; i < 16; ++i) red[(8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)) * 33 + (lane & 31)] = acc[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 1024; i += blockDim.x) {
        const int rr = i >> 5, cc = i & 31;
        if (rr >= rows) break;
        float v[1] = {0.f};
        for (int w = 0; w < W; ++w) v[0] += reinterpret_cast<const float *>(lds)[w * (32 * 33) + rr * 33 + cc];
        const int64_t col = (int64_t)blockIdx.x * 32 + cc;
        if (p.slices > 1) p.part[((int64_t)blockIdx.y * p.M + m0 + rr) * p.cols + col] = v[0];
        else finish_ep<DT, 1>(p, v, m0 + rr, col);
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
    // waves that finish the outputs, also where fewer have a share of the contraction
    // (100 rows of 128 x 1024 4.6 -> 3.2 us; one row 2.6 us, 2.7 with four)
    const int finish = M > 16 ? 8 : M > 8 ? 4 : 1;
    if (lin_transposed(mode)) {
        // slices of at least 32 blocks where K gives fewer than 128 workgroups
        // (256 x 14336: 9.5 us in eight)
        const int nblk = (int)(N / 64);
        int64_t slices = 128 / (K / 32);
        if (slices > nblk / 32) slices = nblk / 32;
        if (slices > 8) slices = 8;
        if (slices < 1) slices = 1;
        s.groups = (int)((nblk + slices - 1) / slices);
        s.slices = (nblk + s.groups - 1) / s.groups;
        s.waves = s.groups < finish ? finish : s.groups < kSmallTWaves ? s.groups : kSmallTWaves;
        return s;
    }
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
    if (s.waves > s.groups) s.waves = s.groups < finish ? finish : s.groups;
    return s;
}

// Where the decode kernels always run.  Beyond (forward up to kSmallGroupsM rows in
// row groups on the grid, transposed from one row on) they compete with the tile
// kernel by estimated time: small matrices leave most of the machine idle there.
bool lin_small_ok(int mode, int64_t M) { return M <= kSmallMaxM && !lin_transposed(mode); }

// Estimated us of a transposed call or one with several 32-row groups (forward: whole K,
// no slices; a large value where it may not run), launch included: rounds of 256 workgroups,
// each as long as its share of the contraction and 0.9 us for its ends.  Fits to
// M = 33..400 on matrices from 256^2 to 4096^2 (1024^2, M = 100: 6.2 against 9.0 us on
// tiles, transposed 8.2 against 10.0; 1408 x 2816 gated, M = 64: 7.6 against 10.7).
// Transposed, up to 32 rows: what a block costs grows with the rows of d, and a second
// round starts cold.  On 24 random matrices and six row counts up to 32 each the choice was
// within 5% of the better kernel in 141 of 144 (14, 18 and 21% off for nine rows of large ones).
double lin_small_us(int mode, int64_t M, int64_t K, int64_t N) {
    const SmallPlan s = small_plan(mode, M, K, N);
    if (M > kSmallGroupsM || (s.slices > 1 && !lin_transposed(mode))) return 1e9;
    const int64_t groups = (M + 31) / 32;
    if (lin_transposed(mode)) {
        const int64_t wgs = K / 32 * groups * s.slices;
        if (M <= kSmallMaxM) {
            // (two workgroups of up to eight waves share a compute unit)
            const int64_t once = s.waves > 8 ? 256 : 512;
            const double rounds = (double)((wgs + once - 1) / once);
            return 2.6 + (rounds > 1 ? 1.3 * rounds : 1.0) * (2.0 + (0.9 + 1.1 / 32 * (double)M) / 1024 * (double)N / s.slices) +
                   (s.slices > 1 ? 3.0 : 0.0);
        }
        const double rounds = (double)((wgs + 255) / 256);
        return 3.6 + rounds * (rounds > 1 ? 1.3 : 1.0) * (1.0 + 2.3 / 1024 * (double)N / s.slices) +
               (s.slices > 1 ? 3.0 : 0.0);
    }
    const double rounds = (double)((N / (16 * s.nb) * groups + 255) / 256);
    return 3.2 + (s.nb == 1 ? 2.4 : 3.1) / 1024 * (double)K * rounds + 0.9 * (rounds - 1);
}

size_t lin_small_workspace_bytes(int mode, int64_t M, int64_t K, int64_t N) {
    const SmallPlan s = small_plan(mode, M, K, N);
    return s.slices > 1 ? (size_t)s.slices * (size_t)M * (size_t)(lin_transposed(mode) ? K : N) * sizeof(float) : 0;
}

template <int DT, bool GLU, int NB, int MT>
static hipError_t small_go(const LinArgs &p, const SmallPlan &s, hipStream_t stream) {
    const dim3 grid((unsigned)(p.cols / (16 * NB)), (unsigned)s.slices, (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
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
    if (lin_transposed(mode)) {
        const dim3 grid((unsigned)(p.cols / 32 + (p.colsum ? p.N / 64 : 0)), (unsigned)s.slices, (unsigned)((p.M + 31) / 32));
        hipLaunchKernelGGL(lin_small_t_kernel<DT>, grid, dim3((unsigned)s.waves * 64), 0, stream, p);
        return hipGetLastError();
    }
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
