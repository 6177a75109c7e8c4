// w8a8.hip — products of 8-bit integers: activations quantized per row (token),
// int8 weights with one scale per column, dense and grouped (experts).
//
//   s_m = fl32(max_k |x[m][k]| / 127),  q[m][k] = rne(x[m][k] / s_m) in [-127, 127]
//   y[m][n] = round(s_m sw[n] sum_k q[m][k] W[k][n] + bias[n])
//
// The integer sum is exact (|q W| <= 2^14 and K < 2^17: below 2^31), so every
// kernel and every split of K gives the same bits.
//
// Bounds.  Few rows: the weights' bytes (one row of 4096 x 14336 with its quantization 12.5 us,
// 4.7 TB/s; a large copy reaches 4.93).  Many rows: the matrix core (8192^3 410 us, 2.67 POP/s,
// the matrix core busy in 75% of the clocks at the 1.7 GHz that its power leaves; zeros for data
// take 360 us).  In between, 40 to 3000 rows, 2 to 5 times the larger of the two: what 64-row tiles draw from L2
// into LDS, about 15 TB/s (351 x 4096 x 8192: 768 workgroups, 403 MB, 26 us); 128 x 256 tiles draw a third of it, with
// too few workgroups for the card.
//
// Weights: the 2048-byte tiles of w8.hip (16 columns x 128 rows, stored as
// q + 128; slot 16 c + j holds rows 32 c .. + 31 of column j).  Matrix-core
// mapping (v_mfma_i32_16x16x64_i8): W is the first operand and x the second,
// so lane l feeds weight column l % 16 and x row l % 16, both with rows
// 128 g + 32 (l / 16) + 16 h .. + 15 of step h; result register r of lane l is
// column 4 (l / 16) + r of x row l % 16: four neighbouring outputs per lane.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace w4 {

constexpr int kW8Tile = 2048;

// ---------------------------------------------------------------------------
// Quantization of rows
// ---------------------------------------------------------------------------

// Largest magnitude of 8 values as bits (magnitudes compare as integers, a NaN's
// above infinity's), joined with what came before: two 16-bit maxima.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void join_top(uint32_t &top, const u32x4_t &v) {
    u16x2_t t = as<u16x2_t>(top);
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, as<u16x2_t>(v[i] & 0x7FFF7FFFu));
    top = __builtin_bit_cast(uint32_t, t);
}
__device__ __forceinline__ uint32_t larger_half(uint32_t top) {
    const uint32_t a = top & 0xFFFFu, b = top >> 16;
    return a > b ? a : b;
}

// Scale of a row from the bits of its largest magnitude; NaN if the row holds a NaN or an
// infinity.
template <int DT>
__device__ __forceinline__ float row_scale(uint32_t top) {
    const float amax = h2f<DT>((uint16_t)top);
    return amax < INFINITY ? amax / 127.0f : __builtin_nanf("");
}

// rne(x / s) for x of a 16-bit type with |x| <= 127 s (1 + 2^-23), exactly.
//
// Nearly always: t = x (1 / s) is within 2^-17 of the quotient; adding 3 2^22 rounds it to
// an integer q, held in the sum's low bits, and t - q, below 1/2 - 2^-16, says that
// the quotient's nearest integer is the same.
// Next to a border k + 1/2 (exact()): the remainder x - q s is exact in fp32 wherever it
// is below s (x and s / 2 are multiples of one unit, at most 2^24 of which make s), so
// comparing it with s / 2 decides; ties go to the even code.  Rows of tiny
// values come here too and are scaled by 2^64 (both x and s, exactly), which keeps s, 1 / s and
// s / 2 normal numbers.
struct RowQuant {
    float scale, inv, limit;
    __device__ __forceinline__ explicit RowQuant(float s) : scale(s) {
        const bool plain = s >= 0x1p-60f;                     // not zero, tiny or NaN
        inv = plain ? 1.0f / s : 0.0f;
        limit = plain ? 0.5f - 0x1p-16f : -1.0f;
    }
    __device__ __forceinline__ int exact(float x) const {
        const float up = scale < 0x1p-60f ? 0x1p64f : 1.0f, s = scale * up;
        if (!(s > 0.0f)) return 0;
        const float half = 0.5f * s, v = x * up;
        float q = __builtin_rintf(v * (1.0f / s));
        const float r = __builtin_fmaf(-q, s, v);
        const bool odd = ((int)q & 1) != 0;
        if (r > half || (r == half && odd)) q += 1.0f;
        if (r < -half || (r == -half && odd)) q -= 1.0f;
        return q > 127.0f ? 127 : q < -127.0f ? -127 : (int)q;
    }
};

// Codes of 8 values.
template <int DT>
__device__ __forceinline__ u32x2_t codes_of(const u32x4_t &v, const RowQuant &rq) {
    constexpr float kRound = 12582912.0f;                    // 3 2^22
    uint32_t m[8];
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v[i >> 1];
        const float x = h2f<DT>((uint16_t)(w >> (16 * (i & 1))));
        const float sum = __builtin_fmaf(x, rq.inv, kRound);
        far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(x, rq.inv, kRound - sum)));
        m[i] = __float_as_uint(sum);
    }
    if (!(far <= rq.limit)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = v[i >> 1];
            m[i] = (uint32_t)rq.exact(h2f<DT>((uint16_t)(w >> (16 * (i & 1)))));
        }
    }
    u32x2_t out;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0C0C0400u);
        const uint32_t b = __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x0C0C0400u);
        out[i] = a | b << 16;
    }
    return out;
}

// Quantization kernel: NW waves per row (workgroups of at least four waves), C pieces of 8
// values per lane in registers between the maximum and the codes.  Bound by memory:
// 3 bytes per element (4096 x 4096: 13 us, 3.9 TB/s); small calls by a load, the maximum across
// waves and the conversions in turn (77 x 8192: 4 us).
// GATHER: row m is that of x row sorted[m] / topk (ids past the X rows take the last one).
template <int DT, int NW, int C, bool GATHER>
__global__ void __launch_bounds__(NW > 4 ? NW * 64 : 256)
w8a8_quantize_kernel(const uint16_t *__restrict__ x, int64_t ldx, const int32_t *__restrict__ row_count,
                     const int32_t *__restrict__ sorted, int topk, int64_t X, uint8_t *__restrict__ qx,
                     float *__restrict__ sx, int64_t M, int64_t K) {
    constexpr int RPB = NW >= 4 ? 1 : 4 / NW, NT = NW * 64;
    __shared__ uint32_t tops[2][NW >= 4 ? NW : 1];
    if (row_count) {
        const int64_t n = *row_count;
        M = n < M ? n : M;
    }
    const int wave = threadIdx.x >> 6, at = NW >= 4 ? threadIdx.x : lane_id();
    int turn = 0;
    for (int64_t m = (int64_t)blockIdx.x * RPB + (NW >= 4 ? 0 : wave); m < M; m += (int64_t)gridDim.x * RPB, turn ^= 1) {
        int64_t src = m;
        if constexpr (GATHER) {
            src = (int64_t)((uint32_t)sorted[m] / (uint32_t)topk);
            src = src < X ? src : X - 1;
        }
        const uint16_t *row = x + src * ldx;
        uint32_t top = 0;
        u32x4_t v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t k = ((int64_t)i * NT + at) * 8;
            v[i] = k < K ? ld128(row + k) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < C; ++i) join_top(top, v[i]);
        for (int64_t k = ((int64_t)C * NT + at) * 8; k < K; k += NT * 8) join_top(top, ld128(row + k));
        top = lane_umax<64>(larger_half(top));
        if constexpr (NW >= 4) {
            if (lane_id() == 0) tops[turn][wave] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < NW; ++w) top = tops[turn][w] > top ? tops[turn][w] : top;
        }
        const float scale = row_scale<DT>(top);
        const RowQuant rq(scale);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t k = ((int64_t)i * NT + at) * 8;
            if (k < K) *reinterpret_cast<u32x2_t *>(qx + m * K + k) = codes_of<DT>(v[i], rq);
        }
        for (int64_t k = ((int64_t)C * NT + at) * 8; k < K; k += NT * 8)
            *reinterpret_cast<u32x2_t *>(qx + m * K + k) = codes_of<DT>(ld128(row + k), rq);
        if (at == 0) sx[m] = scale;
    }
}

// ---------------------------------------------------------------------------
// Shared pieces of the products
// ---------------------------------------------------------------------------

// A scale as significand and exponent: s_m sw_n may leave fp32's range where
// their product with the sum does not.
struct Split {
    float m;
    int e;
    Split() = default;
    __device__ __forceinline__ explicit Split(float s)
        : m(__builtin_amdgcn_frexp_mantf(s)), e(__builtin_amdgcn_frexp_expf(s)) {}
};

__device__ __forceinline__ float finish(int acc, const Split &row, const Split &col, float bias) {
    return __builtin_ldexpf((float)acc * (row.m * col.m), row.e + col.e) + bias;
}

// Row tile `tile` of BM rows, the tiles numbered over all experts: its expert
// and rows; false past the last tile.  Every wave finds it by itself (64 experts
// per scan); rows never leave [0, R) whatever the offsets hold.
__device__ __forceinline__ bool expert_tile(const int32_t *__restrict__ offsets, int E, int64_t R, int BM,
                                            int64_t tile, int &e, int64_t &row0, int64_t &row_end) {
    const int lane = lane_id();
    int64_t before = 0;
    for (int base = 0; base < E; base += 64) {
        const int ee = base + lane;
        int o0 = ee < E ? offsets[ee] : 0, o1 = ee < E ? offsets[ee + 1] : 0;
        o0 = o0 < 0 ? 0 : o0;
        o1 = o1 > R ? (int)R : o1;
        const int rows = o1 - o0;
        const int tl = rows > 0 ? (rows + BM - 1) / BM : 0;
        const int incl = wave_incl_scan(tl);
        const int64_t at = tile - before;
        const uint64_t hit = __ballot(at >= incl - tl && at < incl);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            e = base + src;
            const int in = (int)at - __builtin_amdgcn_readlane(incl - tl, src);
            row0 = __builtin_amdgcn_readlane(o0, src) + (int64_t)in * BM;
            row_end = __builtin_amdgcn_readlane(o1, src);
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// ---------------------------------------------------------------------------
// Split-K kernel: a workgroup owns 16 MT rows x 16 NB columns, its waves split
// the 128-row groups of K and meet in LDS.  Each wave keeps the weights of D groups
// in flight in registers; W goes from memory into operands without LDS, since each byte is used by one
// wave only.  FUSED: x comes in 16 bits, and the workgroup quantizes its
// rows into LDS while the first weights are on their way.
// ---------------------------------------------------------------------------
constexpr int kHeld = 2;                         // pieces of 512 elements that a wave of a fused call quantizes
constexpr int kFusedBytes = 16 * (kHeld * 512 + 16);    // their codes, at most 16 rows of K + 16 bytes

template <int DT, int MT, int NB, int D, int WMAX, bool GROUPED, bool FUSED>
__global__ void __launch_bounds__(WMAX * 64)
w8a8_split_kernel(W8A8Args p, unsigned ncb) {
    static_assert(!GROUPED || !FUSED, "the grouped form reads quantized rows");
    constexpr int RED = WMAX * NB * MT * 1024, LDS = FUSED && kFusedBytes > RED ? kFusedBytes : RED;
    __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
    __shared__ uint32_t tops[FUSED ? 16 * MT : 1];
    i32x4_t *red = reinterpret_cast<i32x4_t *>(lds);          // [wave][MT * NB][64]
    const int64_t K = p.K, N = p.N;
    const int G = (int)(K / kGroup), W = blockDim.x >> 6;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, c = lane >> 4;
    const int64_t n0 = (int64_t)(blockIdx.x % ncb) * (16 * NB);
    const int64_t tile = blockIdx.x / ncb;
    int e = 0;
    int64_t row0 = tile * (16 * MT), row_end = p.M;
    if constexpr (GROUPED) {
        if (!expert_tile(p.offsets, p.E, p.M, 16 * MT, tile, e, row0, row_end)) return;
    }
    // x row of a tile's row; rows past the end take the last one and are not stored
    auto src_row = [&](int64_t r) -> int64_t {
        if (r >= row_end) r = row_end - 1;
        if constexpr (GROUPED) {
            if (p.sorted) {
                const int64_t t = (int64_t)((uint32_t)p.sorted[r] / (uint32_t)p.topk);
                return t < p.X ? t : p.X - 1;
            }
        }
        return r;
    };
    const int g0 = (int)((int64_t)G * wave / W), g1 = (int)((int64_t)G * (wave + 1) / W);
    const uint8_t *wb = p.wp + ((int64_t)e * (N / 16) + n0 / 16) * G * kW8Tile + lane * 32;
    u32x4_t wf[D][NB][2], xf[FUSED ? 1 : D][MT][2];
    // groups past the wave's share re-read its last one
    auto load_w = [&](int d, int g) {
        g = g < g1 ? g : g1 - 1;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) wf[d][b][h] = ld128(wb + ((int64_t)b * G + g) * kW8Tile + 16 * h);
    };
    const uint8_t *xp[MT];
    auto load_x = [&](int d, int g) {
        if constexpr (!FUSED) {
            g = g < g1 ? g : g1 - 1;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) xf[d][t][h] = ld128(xp[t] + (int64_t)g * kGroup + 16 * h);
        }
    };
    const int rows = (int)(row_end - row0 < 16 * MT ? row_end - row0 : 16 * MT);
    const int stride = (int)K + 16;
    if constexpr (FUSED) {
        // Pieces of 512 elements of a row, round robin over the waves, at most kHeld each.  They are
        // requested before the weights: loads return in order.
        const int pieces = (int)((K + 511) / 512), total = pieces * rows;
        u32x4_t held[kHeld];
        int pr[kHeld], pk[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            const int i = wave + u * W;
            pr[u] = i / pieces;
            pk[u] = (i - pr[u] * pieces) * 512 + lane * 8;
            if (i >= total || pk[u] >= K) pr[u] = -1;
            held[u] = pr[u] >= 0 ? ld128(p.x + (row0 + pr[u]) * p.ldx + pk[u]) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int d = 0; d < D; ++d) load_w(d, g0 + d);
        for (int r = threadIdx.x; r < rows; r += W * 64) tops[r] = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            if (wave + u * W >= total) break;
            uint32_t top = 0;
            join_top(top, held[u]);
            top = lane_umax<64>(larger_half(top));
            if (lane == 0) atomicMax(&tops[pr[u]], top);       // lane 0 of a piece is inside its row
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            if (pr[u] >= 0)
                *reinterpret_cast<u32x2_t *>(lds + pr[u] * stride + pk[u]) =
                    codes_of<DT>(held[u], RowQuant(row_scale<DT>(tops[pr[u]])));
        __syncthreads();
    } else {
#pragma unroll
        for (int d = 0; d < D; ++d) load_w(d, g0 + d);
#pragma unroll
        for (int t = 0; t < MT; ++t) xp[t] = p.qx + src_row(row0 + 16 * t + j) * K + 32 * c;
#pragma unroll
        for (int d = 0; d < D; ++d) load_x(d, g0 + d);
    }

    i32x4_t acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[b][t] = i32x4_t{0, 0, 0, 0};
    for (int g = g0; g < g1; g += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if constexpr (FUSED) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int r = 16 * t + j < rows ? 16 * t + j : rows - 1, gg = g + d < g1 ? g + d : g1 - 1;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        xf[0][t][h] = ld128(lds + r * stride + gg * kGroup + 32 * c + 16 * h);
                }
            }
            if (g + d < g1) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const u32x4_t q = wf[d][b][h] ^ 0x80808080u;
#pragma unroll
                        for (int t = 0; t < MT; ++t) acc[b][t] = mfma_i8_16x16x64(q, xf[FUSED ? 0 : d][t][h], acc[b][t]);
                    }
            }
            if (g + D < g1) {
                load_w(d, g + d + D);
                load_x(d, g + d + D);
            }
        }
    }
    if constexpr (FUSED) __syncthreads();            // the codes make room for the sums
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[(wave * NB * MT + b * MT + t) * 64 + lane] = acc[b][t];
    __syncthreads();

    for (int o = wave; o < NB * MT; o += W) {
        i32x4_t sum = red[o * 64 + lane];
        for (int w = 1; w < W; ++w) sum += red[(w * NB * MT + o) * 64 + lane];
        const int b = o / MT, t = o % MT;
        const int64_t r = row0 + 16 * t + j;
        if (r < row_end) {
            const Split rs(FUSED ? row_scale<DT>(tops[FUSED ? 16 * t + j : 0]) : p.sx[src_row(r)]);
            const int64_t n = n0 + 16 * b + 4 * c;
            uint16_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float bv = p.bias ? h2f<DT>(p.bias[n + i]) : 0.0f;
                h[i] = f2h<DT>(finish(sum[i], rs, Split(p.sw[(int64_t)e * N + n + i]), bv));
            }
            *reinterpret_cast<u32x2_t *>(p.y + r * p.ldy + n) =
                u32x2_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
        }
    }
}

// ---------------------------------------------------------------------------
// Tile kernel: BM x BN of y per workgroup, WM x WN waves, K in stages of 64 HALVES, NBUF
// stages in LDS.  Two halves: whole cache lines of x rows, where with stages of 64 every
// line comes twice (64 x 128 tiles, 4096 x 4096 x 14336: 517 -> 326 us); one half: more
// stages in flight, spread evenly (256 x 256 tiles, 8192^3: 410 us against 422).
// ---------------------------------------------------------------------------
constexpr int kXcd8 = 8;              // XCDs; workgroups go to them round-robin
constexpr unsigned kBand = 4;         // row tiles side by side on an XCD

// 16 bytes per lane from global memory (base + off) to LDS (lds_base + 16 lane), not
// waited for here.  In assembly, since the compiler follows its own form of this
// load with a wait for every outstanding load before any LDS read.  It names M0, which the compiler
// writes for loads and indexed registers of its own (and warns that it then does not keep M0's old
// value, which is meant).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds_base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Every DMA but the newest N of this wave and every LDS read have landed; then
// the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Matrix-core step whose sources stay live past it (the destination must not share their
// registers), without ordering it against memory operations.
__device__ __forceinline__ i32x4_t mfma_step(const u32x4_t &a, const u32x4_t &b, const i32x4_t &c) {
    i32x4_t r = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
    asm("" : "+v"(r) : "v"(a), "v"(b));
    return r;
}

// (Registers for as many workgroups per compute unit as LDS holds: 64 x 128 tiles three, which
// take 106 us instead of 118 for 512 tokens top-8 of 64 experts, 2048 x 2816.)
template <int DT, int BM, int BN, int WM, int WN, int HALVES, int NBUF, bool GROUPED>
__global__ void __launch_bounds__(WM * WN * 64, WM * WN == 8 ? 2 : (160 << 10) / (NBUF * (BM + BN) * 64 * HALVES))
w8a8_tile_kernel(W8A8Args p, unsigned mtiles, unsigned ncb, unsigned per_xcd) {
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, RT = TM / 16, CT = TN / 16;
    constexpr int SK = 64 * HALVES, ABYTES = BM * SK, SBYTES = ABYTES + BN * SK;
    constexpr int RPL = 16 / HALVES;                                    // x rows per DMA load
    constexpr int AL = BM / RPL / NW, BL = BN / RPL / NW, L = AL + BL;  // loads per wave and stage
    static_assert(HALVES == 1 || HALVES == 2, "stages of 64 or 128");
    static_assert(CT % 2 == 0 && BM % (RPL * NW) == 0 && BN % (RPL * NW) == 0, "whole loads and column pairs");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * SBYTES];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t K = p.K, N = p.N;
    // XCD x takes a contiguous range of the tiles, which run through bands of kBand row
    // tiles column by column: the tiles at work on an XCD share x and W in its L2.  The slices of a
    // tile follow each other on one XCD.
    const unsigned slot = (blockIdx.x % kXcd8) * per_xcd + blockIdx.x / kXcd8;
    const unsigned id = slot / p.slices, slice = slot % p.slices, bsize = kBand * ncb;
    const unsigned band = id / bsize, in = id % bsize;
    if (band * kBand >= mtiles) return;
    const unsigned high = mtiles - band * kBand < kBand ? mtiles - band * kBand : kBand;
    if (in >= high * ncb) return;             // behind the last tile
    const int64_t tile = band * kBand + in % high, n0 = (int64_t)(in / high) * BN;
    int e = 0;
    int64_t row0 = tile * BM, row_end = p.M;
    if constexpr (GROUPED) {
        if (!expert_tile(p.offsets, p.E, p.M, BM, tile, e, row0, row_end)) return;
    }
    // this slice's 128-row groups: at least one
    const int all = (int)(K / kGroup), first = (int)((int64_t)all * slice / p.slices);
    const int S = ((int)((int64_t)all * (slice + 1) / p.slices) - first) * (2 / HALVES);
    auto src_row = [&](int64_t r) -> int64_t {
        if (r >= row_end) r = row_end - 1;
        if constexpr (GROUPED) {
            if (p.sorted) {
                const int64_t t = (int64_t)((uint32_t)p.sorted[r] / (uint32_t)p.topk);
                return t < p.X ? t : p.X - 1;
            }
        }
        return r;
    };

    // DMA sources.  x: a load fills 16 rows of 64 bytes or 8 of 128, 16-byte chunk c of row r at
    // chunk c ^ fx(r) of its row, fx(r) = (-(r / 4) & 3) + 4 (r / 2 % 2) of the row's last four bits
    // (rows of 64 bytes: the first term); W: a load fills one 1024-byte half of a weight tile, piece p
    // at p ^ 8 (tile & 1).  LDS serves a
    // 128-bit read in four passes over the lanes' quads {0, 3, 5, 6}, {1, 2, 4, 7} and the
    // same plus 8 (measured with pairs of quads on the same banks), 256 bytes each: with these
    // orders the 16 lanes of a pass touch each bank once (4.06 clocks a read; orders for 8
    // neighbouring lanes 6.5 and 8.0).
    auto fx = [](int r) { return (-(r >> 2) & 3) | (HALVES == 2 ? ((r >> 1) & 1) << 2 : 0); };
    uint32_t aoffs[AL], boffs[BL];
    const bool gather = GROUPED && p.sorted;
    const uint8_t *abase = p.qx + (int64_t)first * kGroup;
    const uint8_t *bbase = p.wp + (((int64_t)e * (N / 16) + n0 / 16) * (K / kGroup) + first) * kW8Tile;
    if (!gather) abase += row0 * K;          // gathered rows: X K <= kW8A8GatherBytes
#pragma unroll
    for (int i = 0; i < AL; ++i) {
        const int r = (wave + NW * i) * RPL + lane / (4 * HALVES), c = (lane % (4 * HALVES)) ^ fx(r & 15);
        const int64_t m = src_row(row0 + r);
        aoffs[i] = (uint32_t)((gather ? m : m - row0) * K) + 16 * c;
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
        const int t = (wave + NW * i) / HALVES, half = (wave + NW * i) % HALVES, last = (int)((N - n0) / 16) - 1;
        const int piece = lane ^ ((t & 1) << 3);
        boffs[i] = (uint32_t)((t < last ? t : last) * (K * 16)) + 1024 * half + 16 * piece;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + wave * 1024;
    uint32_t place = 0;                      // of the next stage to fetch
    auto fetch = [&]() {
        const uint32_t base = lds0 + place;
#pragma unroll
        for (int i = 0; i < AL; ++i) dma16(abase, aoffs[i], base + NW * i * 1024);
#pragma unroll
        for (int i = 0; i < BL; ++i) dma16(bbase, boffs[i], base + ABYTES + NW * i * 1024);
        abase += SK;
        bbase += 1024 * HALVES;
        place = place + SBYTES == NBUF * SBYTES ? 0 : place + SBYTES;
    };
#pragma unroll
    for (int s = 0; s < (NW == 8 ? NBUF - 1 : NBUF); ++s)
        if (s < S) fetch();

    // LDS offsets of this lane's operands in the first half of a stage
    const int i16 = lane & 15, q = lane >> 4;
    const int aoff = (wm * TM + i16) * SK + 16 * (q ^ fx(i16));
    // W operand row i of column block ct is column 32 (ct / 2) + 8 (i / 4) + 4 (ct % 2) + i % 4
    // of the wave's tile: a lane then ends up with 8 neighbouring columns per pair of blocks
    const int piece = (q & 1) | (i16 & 3) << 1 | (i16 >> 3) << 3 | ((i16 >> 2) & 1) << 4 | (q >> 1) << 5;
    const int boff = ABYTES + (wn * CT + (i16 >> 3)) * 1024 * HALVES + 16 * piece;

    i32x4_t acc[RT][CT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = i32x4_t{0, 0, 0, 0};

    constexpr int SETS = NW == 8 ? 1 : 2 * HALVES;      // operands of half stages in registers
    u32x4_t xf[SETS][RT], wf[SETS][CT];
    uint32_t at = 0;                         // place of the next stage to read
    auto read = [&](auto set, int half) {
        constexpr int U = decltype(set)::value;
        const uint8_t *base = lds + at;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            wf[U][ct] = *reinterpret_cast<const u32x4_t *>(base + (boff ^ ((ct & 1) * 128)) + (ct >> 1) * 2048 * HALVES + half * 1024);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            xf[U][rt] = *reinterpret_cast<const u32x4_t *>(base + (aoff ^ (half * 64)) + rt * 16 * SK);
    };
    auto passed = [&]() { at = at + SBYTES == NBUF * SBYTES ? 0 : at + SBYTES; };
    auto to_signed = [&](auto set) {
        constexpr int U = decltype(set)::value;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            wf[U][ct] ^= 0x80808080u;                  // u = q + 128 to two's complement q
            asm volatile("" : "+v"(wf[U][ct]));
        }
    };
    auto multiply = [&](auto set) {
        constexpr int U = decltype(set)::value;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                acc[rt][ct] = mfma_step(wf[U][ct], xf[U][rt], acc[rt][ct]);
        __builtin_amdgcn_sched_barrier(0);
    };
    using std::integral_constant;
    using Zero = integral_constant<int, 0>;
    if constexpr (NW == 8) {
        // Two groups of waves, one wave of each on every SIMD, take turns: while one multiplies
        // a half stage, the other reads its operands.  A phase ends in a barrier; group 0 reads half
        // h of stage s in phase 2 (HALVES s + h) and multiplies it in the next, group 1 one phase
        // later.  The place of stage s - 1 is free when group 0 begins stage s (group 1 has read its last
        // half in the phase before) and is filled again from there on.  Every wave waits for its
        // loads of stage s + 1 (WAIT later loads may be outstanding) at the end of its last reads of
        // stage s, which is a barrier before group 0 reads stage s + 1.
        auto stage = [&](auto wait, auto refill) {
            constexpr int WAIT = decltype(wait)::value;
            if constexpr (decltype(refill)::value) fetch();
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                read(Zero{}, h);
                to_signed(Zero{});
                if (h == HALVES - 1) wait_and_meet<WAIT>();
                else wait_and_meet<63>();
                multiply(Zero{});
                wait_and_meet<63>();
            }
            passed();
        };
        if (S >= NBUF - 1) wait_and_meet<(NBUF - 2) * L>();
        else wait_and_meet<0>();
        if (wave >= 4) wait_and_meet<63>();
        int s = 0;
        for (; s + NBUF <= S; ++s) stage(integral_constant<int, (NBUF - 2) * L>{}, integral_constant<bool, true>{});
        for (; s < S; ++s) stage(Zero{}, integral_constant<bool, false>{});
        if (wave < 4) wait_and_meet<63>();
    } else {
        // The operands of stage s + 1 are on their way into registers while stage s is multiplied.
        // Behind the barrier stage s + 1 has landed and everybody has read stage s, whose place is
        // filled again.
        auto read_stage = [&](auto set) {
            constexpr int U = decltype(set)::value * HALVES;
            read(integral_constant<int, U>{}, 0);
            if constexpr (HALVES == 2) read(integral_constant<int, U + HALVES - 1>{}, 1);
            passed();
        };
        auto multiply_stage = [&](auto set) {
            constexpr int U = decltype(set)::value * HALVES;
            to_signed(integral_constant<int, U>{});
            multiply(integral_constant<int, U>{});
            if constexpr (HALVES == 2) {
                to_signed(integral_constant<int, U + HALVES - 1>{});
                multiply(integral_constant<int, U + HALVES - 1>{});
            }
        };
        auto step = [&](auto set) {
            wait_and_meet<(NBUF - 2) * L>();
            fetch();
            read_stage(integral_constant<int, 1 - decltype(set)::value>{});
            __builtin_amdgcn_sched_barrier(0);
            multiply_stage(set);
        };
        auto last_step = [&](auto set, int s) {
            if (s + 1 < S) {
                wait_and_meet<0>();
                if (s + NBUF < S) fetch();
                read_stage(integral_constant<int, 1 - decltype(set)::value>{});
                __builtin_amdgcn_sched_barrier(0);
            }
            multiply_stage(set);
        };
        using One = integral_constant<int, 1>;
        if (S >= NBUF) wait_and_meet<(NBUF - 1) * L>();
        else wait_and_meet<0>();
        read_stage(Zero{});
        int s = 0;
        for (; s + 1 + NBUF < S; s += 2) {
            step(Zero{});
            step(One{});
        }
        for (; s < S; s += 2) {
            last_step(Zero{}, s);
            if (s + 1 < S) last_step(One{}, s + 1);
        }
    }

    if (p.slices > 1) {
        // the slices' sums meet in w8a8_join_kernel
        int *part = p.part + (int64_t)slice * p.M * N;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int64_t r = row0 + wm * TM + rt * 16 + i16;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int64_t n = n0 + wn * TN + 32 * (ct >> 1) + 8 * q + 4 * (ct & 1);
                if (r < row_end && n < N) *reinterpret_cast<i32x4_t *>(part + r * N + n) = acc[rt][ct];
            }
        }
        return;
    }
    int64_t rows[RT];
    Split rs[RT] = {};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        rows[rt] = row0 + wm * TM + rt * 16 + i16;
        rs[rt] = Split(p.sx[src_row(rows[rt])]);
    }
#pragma unroll
    for (int cc = 0; cc < CT / 2; ++cc) {
        const int64_t n = n0 + wn * TN + 32 * cc + 8 * q;
        if (n >= N) continue;
        Split cs[8] = {};
        float bv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = Split(p.sw[(int64_t)e * N + n + i]);
            bv[i] = p.bias ? h2f<DT>(p.bias[n + i]) : 0.0f;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            uint16_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = f2h<DT>(finish(acc[rt][2 * cc + (i >> 2)][i & 3], rs[rt], cs[i], bv[i]));
            if (rows[rt] < row_end)
                *reinterpret_cast<u32x4_t *>(p.y + rows[rt] * p.ldy + n) =
                    u32x4_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                            h[6] | (uint32_t)h[7] << 16};
        }
    }
}

// y from the slices' sums; 4 columns per lane.
template <int DT>
__global__ void __launch_bounds__(256) w8a8_join_kernel(W8A8Args p) {
    const int64_t quads = p.N / 4, total = p.M * quads;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / quads, n = (i % quads) * 4;
        const int *part = p.part + r * p.N + n;
        i32x4_t sum = {0, 0, 0, 0}, next[4];
        for (int s0 = 0; s0 < p.slices; s0 += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                next[u] = *reinterpret_cast<const i32x4_t *>(part + (int64_t)(s0 + u < p.slices ? s0 + u : 0) * p.M * p.N);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (s0 + u < p.slices) sum += next[u];
        }
        const Split rs(p.sx[r]);
        uint16_t h[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float bv = p.bias ? h2f<DT>(p.bias[n + u]) : 0.0f;
            h[u] = f2h<DT>(finish(sum[u], rs, Split(p.sw[n + u]), bv));
        }
        *reinterpret_cast<u32x2_t *>(p.y + r * p.ldy + n) = u32x2_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
struct QuantizeArgs {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *row_count, *sorted;
    int topk;
    int64_t X;
    uint8_t *qx;
    float *sx;
    int64_t M, K;
};

template <int DT, int NW, int C, bool GATHER = false>
static hipError_t quantize_launch(const QuantizeArgs &a, hipStream_t stream) {
    constexpr int RPB = NW >= 4 ? 1 : 4 / NW;
    const int64_t blocks = (a.M + RPB - 1) / RPB;
    hipLaunchKernelGGL((w8a8_quantize_kernel<DT, NW, C, GATHER>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                       dim3(NW > 4 ? NW * 64 : 256), 0, stream, a.x, a.ldx, a.row_count, a.sorted, a.topk, a.X, a.qx, a.sx,
                       a.M, a.K);
    return hipGetLastError();
}

template <int DT, bool GATHER>
static hipError_t quantize_large(const QuantizeArgs &a, hipStream_t stream) {
    if (a.K <= 1024) return quantize_launch<DT, 1, 2, GATHER>(a, stream);
    if (a.K <= 2048) return quantize_launch<DT, 1, 4, GATHER>(a, stream);
    if (a.K <= 4096) return quantize_launch<DT, 4, 2, GATHER>(a, stream);
    if (a.K <= 8192) return quantize_launch<DT, 4, 4, GATHER>(a, stream);
    return quantize_launch<DT, 16, 2, GATHER>(a, stream);
}

template <int DT>
static hipError_t quantize_dispatch(const QuantizeArgs &a, hipStream_t stream) {
    if (a.sorted) return quantize_large<DT, true>(a, stream);
    // Small matrices: one piece per lane, for a short chain of loads and conversions (77 rows of 8192:
    // 3.9 us against 5.9); large ones: more per lane, fewer maxima across waves (4096 rows of
    // 4096: 13.3 us against 15.6; 1024 rows: 5.6 against 5.8).
    if (a.M * a.K <= int64_t(3) << 20) {
        if (a.K <= 512) return quantize_launch<DT, 1, 1>(a, stream);
        if (a.K <= 2048) return quantize_launch<DT, 4, 1>(a, stream);
        if (a.K <= 4096) return quantize_launch<DT, 8, 1>(a, stream);
        if (a.K <= 8192) return quantize_launch<DT, 16, 1>(a, stream);
        return quantize_launch<DT, 16, 2>(a, stream);
    }
    return quantize_large<DT, false>(a, stream);
}

hipError_t launch_w8a8_quantize(const void *x, int64_t ldx, const int32_t *row_count, void *qx, float *sx, int64_t M,
                                int64_t K, int dt, hipStream_t stream) {
    return launch_w8a8_quantize_routed(x, ldx, row_count, nullptr, 1, M, qx, sx, M, K, dt, stream);
}

hipError_t launch_w8a8_quantize_routed(const void *x, int64_t ldx, const int32_t *row_count, const int32_t *sorted,
                                       int topk, int64_t X, void *qx, float *sx, int64_t M, int64_t K, int dt,
                                       hipStream_t stream) {
    if (M == 0) return hipSuccess;
    const QuantizeArgs a{(const uint16_t *)x, ldx, row_count, sorted, topk, X, (uint8_t *)qx, sx, M, K};
    return dt == DT_BF16 ? quantize_dispatch<DT_BF16>(a, stream) : quantize_dispatch<DT_F16>(a, stream);
}

template <int DT, int MT, int NB, int D, int WMAX, bool GROUPED, bool FUSED>
static hipError_t split_launch(const W8A8Args &p, hipStream_t stream) {
    const int64_t G = p.K / kGroup;
    const int W = (int)(G < WMAX ? G : WMAX);
    const int64_t ncb = p.N / (16 * NB);
    const int64_t few = p.M < p.E ? p.M : p.E;                 // experts that can end in a partial tile
    const int64_t mtiles = GROUPED ? p.M / (16 * MT) + few : (p.M + 16 * MT - 1) / (16 * MT);
    if (p.N % (16 * NB) != 0 || mtiles * ncb * W * 64 > UINT32_MAX) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((w8a8_split_kernel<DT, MT, NB, D, WMAX, GROUPED, FUSED>), dim3((unsigned)(mtiles * ncb)),
                       dim3(W * 64), 0, stream, p, (unsigned)ncb);
    return hipGetLastError();
}

static bool slices_fit(const W8A8Args &p, int slices);

template <int DT, int BM, int BN, int WM, int WN, int HALVES, int NBUF, bool GROUPED>
static hipError_t tile8_launch(const W8A8Args &p, hipStream_t stream) {
    const int64_t ncb = (p.N + BN - 1) / BN;
    const int64_t few = p.M < p.E ? p.M : p.E;
    const int64_t mtiles = GROUPED ? p.M / BM + few : (p.M + BM - 1) / BM;
    const int64_t per_xcd = (mtiles * ncb * p.slices + kXcd8 - 1) / kXcd8;
    if (per_xcd * kXcd8 * WM * WN * 64 > UINT32_MAX || p.slices < 1 || p.K / kGroup < p.slices) return hipErrorInvalidConfiguration;
    if (p.slices > 1 && (GROUPED || !slices_fit(p, p.slices))) return hipErrorInvalidConfiguration;
    if (p.sorted && p.X * p.K > kW8A8GatherBytes) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((w8a8_tile_kernel<DT, BM, BN, WM, WN, HALVES, NBUF, GROUPED>), dim3((unsigned)(per_xcd * kXcd8)),
                       dim3(WM * WN * 64), 0, stream, p, (unsigned)mtiles, (unsigned)ncb, (unsigned)per_xcd);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.slices == 1) return err;
    const int64_t blocks = (p.M * (p.N / 4) + 255) / 256;
    hipLaunchKernelGGL(w8a8_join_kernel<DT>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// Column blocks of 16 per workgroup of the split-K kernel: as many as leave about a
// workgroup per compute unit.
static int split_columns(int64_t N, int64_t mtiles) {
    return N * mtiles >= 64 * 192 ? 4 : N * mtiles >= 32 * 192 ? 2 : 1;
}

// The kernels, by number.  0: split-K, 16 rows; 1, 2: split-K, 32 rows; 3 ..: tiles.  7 has kernel 3's tiles
// and more stages in flight, for a workgroup alone on its compute unit (77 x 8192 x 8192: 22.8 us against 26.4);
// three that share one are as fast with three stages each (1024 x 4096 x 4096: 35.0 us against 36.0).
struct W8A8Kernel {
    int bm, bn;
    int resident;              // workgroups on a compute unit
    int waves;                 // split-K: waves that share K (tiles: 0)
    double base, step, more, round;  // us: a launch, per step (a 128-row group per wave, or 64 of K), per further
                                     // resident workgroup, per round of resident workgroups
};
static constexpr W8A8Kernel kKernels[] = {{16, 16, 2, 16, 0.27, 1.22, 1.09, 3.25},  {32, 64, 2, 8, 2.46, 1.74, 2.11, 0.54},
                                          {32, 32, 2, 16, 1.72, 2.12, 2.64, 0},     {64, 64, 3, 0, 3.53, 0.144, 0.091, 0.055},
                                          {64, 128, 3, 0, 3.06, 0.309, 0.098, 0.29}, {128, 256, 1, 0, 3.15, 0.411, 0, 1.71},
                                          {256, 256, 1, 0, 3.25, 0.525, 0, 3.51},   {64, 64, 2, 0, 4.28, 0.129, 0.101, 0}};
constexpr int kKernelCount = sizeof(kKernels) / sizeof(kKernels[0]);
int w8a8_config_count() { return kKernelCount; }

// Estimated time in us of a kernel whose tiles cover `mtiles` row tiles of M rows, K
// cut into `slices`.  The constants of kKernels and of this formula are fitted to 5700 measured
// products (338 sizes of 17 to 4096 rows, K from 256 to 14336, N from 512 to 14336) such that the choice by
// it is near the best of these kernels: there 1.0% slower on average, 14% at most; on 90 other sizes of the same
// ranges 1.2% on average, more than 5% for 8 of them, 22% at most (284 x 2560 x 3584).
static double kernel_us(const W8A8Kernel &k, int64_t mtiles, int64_t M, int64_t K, int64_t N, int slices) {
    const int64_t wg = mtiles * ((N + k.bn - 1) / k.bn) * slices, G = K / kGroup;
    const double steps = k.waves ? (G >= k.waves ? (double)G / k.waves : 1.0) : (double)K / 64 / slices;
    const int64_t full = wg / (256 * k.resident), left = (wg - full * 256 * k.resident + 255) / 256;
    double us = k.base + steps * full * (k.step + k.more * (k.resident - 1)) + k.round * (double)(full + (left > 0));
    if (left > 0) us += steps * (k.step + k.more * (double)(left - 1));
    return slices > 1 ? us + 2.22 + 2.38e-6 * (double)(slices * M * N) : us;
}

// Test hook: the kernel of the next calls, plus 100 times its slices (-1: by size).
static std::atomic<int> g_w8a8_cfg{-1};
void set_w8a8_config(int idx) { g_w8a8_cfg.store(idx, std::memory_order_relaxed); }

static bool slices_fit(const W8A8Args &p, int slices) {
    return p.part && p.K / kGroup / slices >= 2 && (double)slices * (double)p.M * (double)p.N * 4 <= (double)kW8A8PartBytes;
}

// A launch has at most 2^32 - 1 threads.
static bool grid_fits(const W8A8Args &p, int kernel, int slices) {
    const W8A8Kernel &k = kKernels[kernel];
    const int64_t few = p.M < p.E ? p.M : p.E, G = p.K / kGroup;
    const int64_t mtiles = p.offsets ? p.M / k.bm + few : (p.M + k.bm - 1) / k.bm;
    const int64_t bn = kernel == 0 ? 16 * split_columns(p.N, p.offsets ? few : 1) : k.bn;
    const int64_t wgs = mtiles * ((p.N + bn - 1) / bn) * slices + kXcd8;
    const int64_t threads = k.waves ? 64 * (G < k.waves ? G : k.waves) : k.bm <= 64 ? 256 : 512;
    return wgs <= UINT32_MAX / threads;
}

static void pick_kernel(const W8A8Args &p, int &kernel, int &slices) {
    const int forced = g_w8a8_cfg.load(std::memory_order_relaxed);
    slices = 1;
    if (forced >= 0 && forced % 100 < kKernelCount) {
        kernel = forced % 100;
        if (kernel >= 3 && forced >= 200 && slices_fit(p, forced / 100)) slices = forced / 100;
        return;
    }
    // grouped: the experts' row counts are on the device.  With counts spread as skewed routing spreads
    // them (exponentially around their mean), an expert has 1 / (1 - exp(-bm / mean)) row tiles.
    const double held = (double)(p.M < p.E ? p.M : p.E), mean = p.offsets ? (double)p.M / held : 0;
    // At most 8 rows per expert on average: 16-row tiles (64 experts, 1408 x 2048, M / E = 0.5, 2, 4, 8: 15.5,
    // 27.5, 35.4, 42.4 us against 19, 34, 40, 46 us with the best others; M / E = 16: 51.5 against 49.9 us; 16 experts of
    // 4096 x 1024 and 2048 x 4096, M / E = 8: 18.9 and 30.9 us, the best; but 128 experts of 768 x 2048, M / E = 8: 56 against
    // 51 us, and 8 experts of 4096 x 14336, M / E = 4: 91 against 82 us).  Dense products of up to 16 rows: near the best where
    // the weights are most of the time (16 x 4096 x 14336), slower on small ones (20 sizes of 2 to 16 rows: 13% on average, at
    // most 57%, 15 x 1280 x 5184 11.9 against 7.6 us).
    kernel = 0;
    if ((p.offsets ? p.M <= 8 * (int64_t)p.E : p.M <= 16) && grid_fits(p, 0, 1)) return;
    double best = 1e30;
    for (int i = 0; i < kKernelCount; ++i) {
        const W8A8Kernel &k = kKernels[i];
        if (i == 0 && split_columns(p.N, 1) != 1) continue;
        const int64_t mtiles = p.offsets ? (int64_t)std::ceil(held / (1 - std::exp(-k.bm / mean))) : (p.M + k.bm - 1) / k.bm;
        for (int n = 1; n <= 8; n *= 2) {
            if ((n > 1 && (k.waves != 0 || !slices_fit(p, n))) || !grid_fits(p, i, n)) break;
            const double us = kernel_us(k, mtiles, p.M, p.K, p.N, n);
            if (us < best) {
                best = us;
                kernel = i;
                slices = n;
            }
        }
    }
}

int w8a8_plan(int64_t M, int64_t K, int64_t N, int E) {
    static const int32_t offsets = 0;
    static int32_t room = 0;
    W8A8Args p{};
    p.M = p.X = M;
    p.K = K;
    p.N = N;
    p.E = E > 0 ? E : 1;
    p.offsets = E > 0 ? &offsets : nullptr;
    p.part = E == 0 && M <= kW8A8SliceRows ? &room : nullptr;
    int kernel = 0, slices = 1;
    pick_kernel(p, kernel, slices);
    return grid_fits(p, kernel, slices) ? kernel + 100 * slices : -1;
}

template <int DT, bool GROUPED>
static hipError_t w8a8_dispatch(const W8A8Args &args, hipStream_t stream) {
    W8A8Args p = args;
    int kernel = 0;
    pick_kernel(p, kernel, p.slices);
    switch (kernel) {
        case 0:
            // grouped: one group of weights in flight leaves room for two workgroups on a compute unit
            // (M / E = 0.5 as above: 15.5 us against 18.6)
            switch (split_columns(p.N, GROUPED ? (p.M < p.E ? p.M : p.E) : 1)) {
                case 4: return split_launch<DT, 1, 4, GROUPED ? 1 : 2, 16, GROUPED, false>(p, stream);
                case 2: return split_launch<DT, 1, 2, 2, 16, GROUPED, false>(p, stream);
                default: return split_launch<DT, 1, 1, 4, 16, GROUPED, false>(p, stream);
            }
        case 1: return split_launch<DT, 2, 4, 2, 8, GROUPED, false>(p, stream);
        case 2: return split_launch<DT, 2, 2, 1, 16, GROUPED, false>(p, stream);
        case 3: return tile8_launch<DT, 64, 64, 2, 2, 2, 3, GROUPED>(p, stream);
        case 4: return tile8_launch<DT, 64, 128, 2, 2, 2, 2, GROUPED>(p, stream);
        case 5: return tile8_launch<DT, 128, 256, 2, 4, 2, 3, GROUPED>(p, stream);
        case 6: return tile8_launch<DT, 256, 256, 2, 4, 1, 4, GROUPED>(p, stream);
        default: return tile8_launch<DT, 64, 64, 2, 2, 2, 5, GROUPED>(p, stream);
    }
}

bool w8a8_fused_ok(int64_t M, int64_t K) {
    const int64_t W = K / kGroup < 16 ? K / kGroup : 16;
    return M <= 16 && M * ((K + 511) / 512) <= kHeld * W;
}

template <int DT>
static hipError_t w8a8_fused_dispatch(const W8A8Args &p, hipStream_t stream) {
    switch (split_columns(p.N, 1)) {
        case 4: return split_launch<DT, 1, 4, 2, 16, false, true>(p, stream);
        case 2: return split_launch<DT, 1, 2, 2, 16, false, true>(p, stream);
        default: return split_launch<DT, 1, 1, 4, 16, false, true>(p, stream);
    }
}

hipError_t launch_w8a8_fused(const W8A8Args &p, int dt, hipStream_t stream) {
    return dt == DT_BF16 ? w8a8_fused_dispatch<DT_BF16>(p, stream) : w8a8_fused_dispatch<DT_F16>(p, stream);
}

hipError_t launch_w8a8(const W8A8Args &p, int dt, hipStream_t stream) {
    if (p.M == 0) return hipSuccess;
    if (dt == DT_BF16) return p.offsets ? w8a8_dispatch<DT_BF16, true>(p, stream) : w8a8_dispatch<DT_BF16, false>(p, stream);
    return p.offsets ? w8a8_dispatch<DT_F16, true>(p, stream) : w8a8_dispatch<DT_F16, false>(p, stream);
}

}  // namespace w4
