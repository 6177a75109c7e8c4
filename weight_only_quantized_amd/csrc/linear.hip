// linear.hip — tile kernel of the fused linear operators: the forward products
// x . W (with bias, activation and residual, or gated) for more than 32 rows, and
// the transposed product d . W^T of their backward passes; the activation
// gradient d with its column sums; the sum of sliced products.
//
// Forward tiles of 64 or 128 rows by 128 columns: lin_mid_kernel, below.
//
// Tile kernel (lin_wide_kernel): a workgroup owns a BM x BN tile; 2 x BN / 64 waves
// run over the contraction in stages of 64 elements, each with (BM / 2) x 64 of
// the tile in 32 x 32 x 16 matrix-core steps.  Tiles of 128 columns (transposed) have
// two such groups of waves, each with half of the contraction and LDS of its
// own: two waves per SIMD, one's vector work beside the other's products (64 x 128,
// M = 128, 4096^2 unsliced 33.9 -> 26.7 us).  Both operands of a stage lie in LDS, double buffered.  W is dequantized once per workgroup on its way
// there (32 codes of one column per thread and stage), so one conversion serves
// BM rows: with 256 rows 3 vector instructions per matrix-core step, where a
// wave that dequantizes its own columns for 64 rows needs 7.
//
// Forward (contraction over K): codes enter the matrix core as exact integers
// u - z (bf16: times the scale's power of two) and the scale acts on fp32 sums.  The
// sums are kept in units of the current group's scale (bf16: of its significand):
// entering group g they are multiplied by s[g-1] / s[g] in place (Horner's scheme
// for sum_g s_g P_g), and by the last scale at the end.  So no second set of
// accumulators is needed, and nothing but the result is rounded to 16 bits.  A
// group multiplies every sum once: 2 vector instructions per matrix-core step.
//
// Transposed (contraction over N): column n of W contributes to all outputs of
// its group with one scale s[g][n], which varies along the contraction; it must
// sit on an operand.  W is therefore rounded to the activation dtype as
// (u - z) s, and d enters as it is stored; both are the 16-bit operands the matrix
// core needs.  That costs accuracy: against 64 bits dx is 1.3 times as far off as one rounding
// of the result, 1.6 times where d was rounded too (plain fp32: once).  A second
// product with the remainder of W would bring those to 1 and 1.4, and
// its matrix instructions alone take gated 4096 x 4096 x 28672 from 875 to 1390 us.
// The codes of one lane belong to one column n and 32 rows k, while the operand
// wants 8 columns n of one k: the tile is written as [n][k] rows and read with
// the transposing LDS read.
//
// Matrix-core mapping (32 x 32 x 16): lane l feeds row / column l % 32 and
// contraction elements 8 (l / 32) .. + 7; result register r of lane l is row
// 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
//
// Bound: large products by the matrix core, at the clock that it leaves under full load.  Measured
// (bf16, graph replay): gated 4096 x 4096 x 28672 with h saved 804 to 821 us on
// different cards (1.2 PFLOP/s; a library product of unquantized bf16 operands of that size takes
// 731 us here), transposed 4096 x 28672 x 4096 750 us (1.28 PFLOP/s; library 681 us),
// 4096^3 124 to 135 us forward and 120 us transposed (library 126 us).  The matrix core
// is busy 60% (forward) and 67% (transposed) of 1.7 GHz cycles; LDS accesses,
// 1% of them bank conflicts, take 40%.  Wave priorities, 128 x 128 wave tiles and
// other placements of the vector work measured even or slower.
#include <atomic>
#include <type_traits>

#include "act.hpp"

namespace w4 {

constexpr int kXcd = 8;              // XCDs; workgroups go to them round-robin
constexpr int kBK = 64;              // contraction elements per stage
// Wave groups of a BM x BN workgroup, each with a share of the contraction.
constexpr int wide_groups(int bm, int bn) { return bm <= 128 && bn <= 128 ? 2 : 1; }

// LDS swizzles: 16-byte chunk c of row r sits at chunk c ^ key(r) of its row.
// Writes move 128 bytes a cycle (8 lanes), 16-byte reads 256 (16 lanes).
// Rows of 128 bytes (A, forward W; read and written down 16 and 8 rows at one
// c): 8 consecutive rows get different chunks, and rows 8 apart, which share a
// 128-byte half, too.
__device__ __forceinline__ int key_row(int r) { return (r & 7) ^ ((r >> 3) & 1); }
// Rows of 256 or 512 bytes (transposed W; written down 8 rows at one c, read as 4 rows
// x 4 chunks): bits 2, 3 tell 4 rows apart for the reads, bits 0..2 tell 8 rows
// apart for the writes.
__device__ __forceinline__ int key_t(int n) { return (n & 3) << 2 | (n & 2) | ((n >> 2) & 1); }

// Matrix-core step whose sources stay live past it (the destination must not
// share their registers), without ordering it against memory operations.
template <int DT>
__device__ __forceinline__ f32x16_t mfma_step(const u32x4_t &a, const u32x4_t &b, const f32x16_t &c) {
    f32x16_t r;
    if constexpr (DT == DT_BF16)
        r = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                    0, 0, 0);
    else
        r = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                   0, 0);
    asm("" : "+v"(r) : "v"(a), "v"(b));
    return r;
}

__global__ void __launch_bounds__(512) lin_colsum_kernel(const float *part, float *colsum, int64_t N, int blocks) {
    __shared__ float red[8 * 64];
    colsum_body(part, colsum, N, blocks, (int64_t)blockIdx.x * 64, red);
}

// Forward products: the sums of a column are held in units of its running scale.
// A new scale group multiplies them by unit / s first and its codes enter the
// matrix core as exact integers.
//
// bf16: of a scale m 2^e only m (1 <= |m| < 2) is the unit; 2^e goes into the codes, which
// stay exact.  So the sums have the size of the result: they pass fp32's range, and
// terms vanish, where those of x (u - z) s in fp32 would (with the whole scale as
// the unit, a group beside one 2^60 larger had to count as zero, and sums grew by the
// ratio of two scales).  Subnormal scales and those past 2^110 leave a part of 2^e in
// the unit.  fp16: scales lie within 2^40 of each other and sums of x (u - z) below 2^42,
// so the unit is the scale.  A scale of 0 leaves the unit alone and its codes
// enter as 0.
template <int DT>
struct ScaleUnit {
    float unit = 0.f, ratio = 1.f;
    float f = 512.f, zf, m;           // bf16: factor of the codes' conversion, zero point times 2^e; the group's own unit
    uint32_t z, sel;
    // A new group: what its codes need.
    __device__ __forceinline__ void next(float s, uint32_t zero) {
        z = zero;
        m = s;
        if constexpr (DT == DT_BF16) {
            uint32_t e = __float_as_uint(s) & 0x7F800000u;
            e = e < (1u << 23) ? 1u << 23 : e > (237u << 23) ? 237u << 23 : e;
            f = __uint_as_float(e + (9u << 23));
            zf = codes_f32<0>(zero, f)[0];
            m = s * __uint_as_float((254u << 23) - e);                            // NaN and infinity stay
        }
        // bf16: byte selector of the upper halves, or of zeros; fp16: mask
        sel = DT == DT_BF16 ? (s != 0.f ? 0x07060302u : 0x0C0C0C0Cu) : (s != 0.f ? ~0u : 0u);
    }
    // Its unit and the factor on the sums before it (lin_mid_kernel: later than the codes'
    // part, 333 rows gated 15.2 -> 15.0 us).
    __device__ __forceinline__ void change() {
        const bool live = m != 0.f;                                               // NaN among them
        const float q = unit * __builtin_amdgcn_rcpf(m);
        ratio = (live & (m != unit)) ? q : 1.f;
        unit = live ? m : unit;
    }
    // The 8 codes of a word as u - z (bf16: times 2^e), rows in order, in two halves: words HF
    // and HF + 2 of the operand (fp16: all of it with the second).
    template <int HF>
    __device__ __forceinline__ void dequant(uint32_t w, u32x4_t &o) const {
        if constexpr (DT == DT_BF16) {
            const uint32_t m = (HF ? w >> 4 : w) & 0x0F0F0F0Fu;            // bytes: rows 0, 4, 1, 5 or 2, 6, 3, 7
            const f32x2_t a = codes_f32<0>(m, f), b = codes_f32<1>(m, f);
            o[HF] = __builtin_amdgcn_perm(__float_as_uint(b[0] - zf), __float_as_uint(a[0] - zf), sel);
            o[HF + 2] = __builtin_amdgcn_perm(__float_as_uint(b[1] - zf), __float_as_uint(a[1] - zf), sel);
        } else if constexpr (HF == 1) {
            o = dequant_word<DT>(w, f16_negbias2(z));
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] &= sel;
        }
    }
};

struct TilePos { int slice; int64_t nt, mt; };
// XCD x takes a contiguous share of the list (slices, then groups of four row
// tiles by column tile by row tile): the workgroups of one L2 share operands.
__device__ __forceinline__ TilePos tile_pos(const LinArgs &p, uint32_t total) {
    constexpr uint32_t GM = 4;
    const uint32_t tiles = (uint32_t)p.mtiles * (uint32_t)p.ntiles;
    const uint32_t id = blockIdx.x, xcd = id % kXcd;
    const uint32_t r8 = total % kXcd, idx = xcd * (total / kXcd) + (xcd < r8 ? xcd : r8) + id / kXcd;
    const uint32_t slice = idx / tiles, tile = idx - slice * tiles;
    const uint32_t m_first = tile / (GM * p.ntiles) * GM;
    const uint32_t gmt = p.mtiles - m_first < GM ? p.mtiles - m_first : GM;
    const uint32_t rem = tile - m_first * p.ntiles;
    return {(int)slice, (int64_t)(rem / gmt), (int64_t)(m_first + rem % gmt)};
}

template <int DT, int MODE, int BM, int BN>
__global__ void __launch_bounds__(wide_groups(BM, BN) * 2 * BN, 2) lin_wide_kernel(const LinArgs p) {
    constexpr bool T = MODE == LIN_T;
    constexpr int NT = 2 * BN;                       // threads of a wave group: 2 x BN / 64 waves of (BM / 2) x 64
    constexpr int KS = wide_groups(BM, BN);
    constexpr int RT = BM / 64, CT = 2;              // 32 x 32 tiles per wave
    constexpr int AROWS = NT / 8;                    // rows of A per staging pass
    constexpr int XP = BM / AROWS;                   // 16-byte A chunks per thread and stage
    constexpr int ABYTES = BM * kBK * 2;
    constexpr int BBYTES = BN * kBK * 2;
    constexpr int kTRow = BN * 2;                    // LDS row (bytes) of the transposed W tile
    constexpr int OUTROW = 68;                       // floats per row of the output staging
    constexpr int LDSBYTES = 2 * (ABYTES + BBYTES);
    static_assert(LDSBYTES >= NT / 64 * 32 * OUTROW * 4, "output staging fits");
    __shared__ __attribute__((aligned(16))) uint8_t lds[KS * LDSBYTES];
    static_assert(T || KS == 1, "forward tiles of 128 columns: lin_mid_kernel");
    __shared__ float s_ratio[T ? 1 : BN];            // per column: factor on the sums at a new scale group

    const int tid = threadIdx.x % NT, lane = tid & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = wave_all / (NT / 64), wave = wave_all % (NT / 64);     // wave group, wave in it
    uint8_t *const lda_ = lds + grp * LDSBYTES, *const ldb_ = lda_ + 2 * ABYTES;
    const int wm = wave / (BN / 64), wn = wave % (BN / 64);
    const int l31 = lane & 31, kg = lane >> 5;

    // ---- tile of this workgroup ------------------------------------------------
    const uint32_t total = (uint32_t)p.mtiles * (uint32_t)p.ntiles * (uint32_t)p.slices;
    if constexpr (T) {
        // workgroups past the product's: the bias gradient, 64 columns each (one
        // launch less than a kernel of its own)
        if (blockIdx.x >= total) {
            colsum_body(p.cpart, p.colsum, p.N, p.cblocks, (int64_t)(blockIdx.x - total) * 64,
                        reinterpret_cast<float *>(lds));
            return;
        }
    }
    const TilePos tp = tile_pos(p, total);
    const int slice = tp.slice;
    const int64_t nt = tp.nt, row0 = tp.mt * BM;

    const int64_t G = p.K / kGroup;
    const int nst = (int)((T ? p.N : p.K) / kBK);
    // this slice's stages [b0, b1); wave group g takes `share` of them from b0 + g share
    // on (an even number: whole 128-row groups), fewer or none at the end
    const int b0 = slice * p.stages, b1 = b0 + p.stages < nst ? b0 + p.stages : nst;
    const int share = KS == 1 ? b1 - b0 : ((b1 - b0 + KS - 1) / KS + 1) & ~1;
    const int s0 = b0 + grp * share < b1 ? b0 + grp * share : b1, s1 = s0 + share < b1 ? s0 + share : b1;

    // ---- A operand: BM rows of 64 elements per stage ------------------------------
    // (the rows of a thread are AROWS apart: one LDS offset serves all)
    const uint8_t *const abase = reinterpret_cast<const uint8_t *>(p.a + row0 * p.lda);
    uint32_t aoff[XP];
    const int ar_ = tid >> 3, ac_ = tid & 7;
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        const int64_t r = row0 + i * AROWS + ar_ < p.M ? i * AROWS + ar_ : p.M - 1 - row0;
        aoff[i] = (uint32_t)(r * p.lda + ac_ * 8) * 2u;
    }
    uint8_t *const adst = lda_ + ar_ * (kBK * 2) + ((ac_ ^ key_row(ar_)) << 4);
    // Small tiles run a stage in less than a memory round trip: they hold two
    // stages of A on the way (DEEP), the 256-row tile has registers for one.
    constexpr bool DEEP = RT < 4;
    u32x4_t ar[DEEP ? 2 : 1][XP];
    auto load_a = [&](int d, int s, int i) {
        ar[DEEP ? d : 0][i] = ld128(abase + (int64_t)s * (kBK * 2) + aoff[i]);
    };
    auto store_a = [&](int d, int buf, int i) {
        *reinterpret_cast<u32x4_t *>(adst + buf * ABYTES + i * AROWS * (kBK * 2)) = ar[DEEP ? d : 0][i];
    };

    // ---- W operand: one 16-byte slot (32 rows of one column) per thread -----------
    const int j = lane & 15, c32 = T ? lane >> 4 : (lane >> 4) & 1;
    // without zero points the scales' own bytes are read and ignored: no branch
    // around a load
    const uint8_t *const zbase = p.zero ? p.zero : reinterpret_cast<const uint8_t *>(p.scale);
    uint32_t woff, soff;                              // bytes into W, columns into the scales
    int64_t wstep;                                    // bytes of W per stage
    uint32_t bdst;                                    // LDS byte of word 0; word t is at bdst ^ 16 t
    int wcol = 0;                                     // forward: column within the tile
    int64_t srow_t = 0;                               // transposed: scale row of this wave's 128 outputs
    if constexpr (!T) {
        const int cb = 2 * wave + (lane >> 5);
        int64_t nb;
        if constexpr (MODE == LIN_GLU) {
            // 4 blocks per consuming wave: two gate, then the two up blocks of the same columns
            const int64_t half = p.cols / 2;
            int64_t c0 = nt * (BN / 2) + (cb >> 2) * 32 + (cb & 1) * 16;
            if (c0 >= half) c0 = half - 16;
            nb = ((cb & 2) ? half + c0 : c0) / 16;
        } else {
            nb = nt * (BN / 16) + cb;
            if (nb >= p.cols / 16) nb = p.cols / 16 - 1;
        }
        wcol = cb * 16 + j;
        woff = (uint32_t)(nb * G * kTileBytes) + c32 * 256 + j * 16;
        wstep = 512;
        soff = (uint32_t)(nb * 16 + j);
        bdst = wcol * (kBK * 2) + (((4 * c32) ^ key_row(wcol)) << 4);
    } else {
        const int nbi = wave & 3, gi = wave >> 2;
        int64_t g = nt * (BN / 128) + gi;
        if (g >= G) g = G - 1;
        woff = (uint32_t)((nbi * G + g) * kTileBytes) + lane * 16;
        wstep = 4 * G * kTileBytes;
        srow_t = g / p.gm * p.N;
        const int n = nbi * 16 + j;
        soff = n;
        bdst = n * kTRow + (((gi * 16 + c32 * 4) ^ key_t(n)) << 4);
    }
    u32x4_t wr[2];                                    // raw codes of the next two stages
    auto load_w = [&](int d, int s) { wr[d] = ld128(p.wp + (int64_t)s * wstep + woff); };
    // Scales and zero points travel well ahead of the codes (a 2-byte load waits
    // as long as a 16-byte one).  Forward: those of the next 128-row group, two
    // stages ahead.  Transposed, where every stage has other columns: the four
    // lanes of a column fetch four stages at once, four stages ahead, and hand
    // them over with a lane permute.
    uint32_t scur = 0;                                // transposed: scale | zero << 16 of 4 stages
    uint16_t snext;
    uint8_t znext;
    auto load_s = [&](int s) {
        int64_t so;
        if constexpr (T) {
            const int sl = s + c32 < s1 ? s + c32 : s1 - 1;
            so = srow_t + (int64_t)sl * kBK + soff;
        } else {
            const int sl = s < s1 ? s : s1 - 1;
            so = (int64_t)(((uint64_t)(sl >> 1) * p.gm_inv) >> 32) * p.N + soff;
        }
        snext = p.scale[so];
        znext = zbase[so >> 1];
    };
    auto zero_of = [&](uint32_t zb) {
        return p.zero ? __builtin_amdgcn_ubfe(zb, (uint32_t)(j & 1) * 4u, 4) : 8u;
    };
    // Forward: the factors on the sums reach the waves that hold a column's sums
    // through LDS.  Transposed: W = u s - z s.
    ScaleUnit<DT> su;
    float ds, dzs;
    uint32_t dz;
    // stage st is about to be dequantized: its column's scale and zero point
    // (forward: once per 128-row group, from the loaded values)
    auto deq_begin = [&](int st) {
        if constexpr (T) {
            const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute((((st - s0) & 3) * 16 + j) << 2, (int)scur);
            ds = h2f<DT>((uint16_t)(v & 0xFFFFu));
            dz = v >> 16;
            dzs = -(float)dz * ds;
        } else {
            su.next(h2f<DT>(snext), zero_of(znext));
            su.change();
            s_ratio[wcol] = su.ratio;                 // both lanes of a column write the same value
        }
    };
    // Half-word i of the slot (word i / 2): codes of rows 0, 1, 4, 5 or 2, 3, 6, 7
    // of its 8; the second half writes the 16 bytes to LDS.
    u32x4_t dqo;
    auto deq_half = [&](int d, int buf, int i) {
        const int t = i >> 1, hf = i & 1;
        const uint32_t w = wr[d][t];
        if constexpr (!T) {
            if (hf) su.template dequant<1>(w, dqo);
            else su.template dequant<0>(w, dqo);
        } else if constexpr (DT == DT_BF16) {
            // bytes: rows 0, 4, 1, 5 (or 2, 6, 3, 7)
            const uint32_t m = (hf ? w >> 4 : w) & 0x0F0F0F0Fu;
            const f32x2_t c04 = codes_f32<0>(m), c15 = codes_f32<1>(m);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const bf16x2_t b = {(__bf16)__builtin_fmaf(c04[q], ds, dzs), (__bf16)__builtin_fmaf(c15[q], ds, dzs)};
                dqo[hf + 2 * q] = __builtin_bit_cast(uint32_t, b);
            }
        } else if (hf) {
            dqo = dequant_word<DT>(w, f16_negbias2(dz));
            const _Float16 m = (_Float16)ds;
            const f16x2_t m2 = {m, m};
#pragma unroll
            for (int q = 0; q < 4; ++q) dqo[q] = __builtin_bit_cast(uint32_t, as<f16x2_t>(dqo[q]) * m2);
        }
        if (hf) *reinterpret_cast<u32x4_t *>(ldb_ + buf * BBYTES + (bdst ^ (uint32_t)(t << 4))) = dqo;
    };

    // ---- main loop ---------------------------------------------------------------
    f32x16_t acc[RT][CT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[rt][ct][r] = 0.f;

    const int rkey = key_row(l31);                    // (every row base is a multiple of 16)
    const uint8_t *const afrag = lda_ + (wm * (BM / 2) + l31) * (kBK * 2);
    auto frag_a = [&](int buf, int rt, int t) {
        return *reinterpret_cast<const u32x4_t *>(afrag + buf * ABYTES + rt * 32 * (kBK * 2) +
                                                  (((2 * t + kg) ^ rkey) << 4));
    };
    const uint8_t *bfrag[T ? CT : 1][2];
    if constexpr (T) {
        const int qq = lane >> 4, tr = (lane & 15) >> 2, tc = lane & 3;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 8 * (qq >> 1) + 4 * h + tr, ch = wn * 8 + ct * 4 + 2 * (qq & 1) + (tc >> 1);
                bfrag[ct][h] = ldb_ + n * kTRow + ((ch ^ key_t(n)) << 4) + (tc & 1) * 8;
            }
    } else {
        bfrag[0][0] = ldb_ + (wn * 64 + l31) * (kBK * 2);
    }
    auto frag_b = [&](int buf, int ct, int t) -> u32x4_t {
        if constexpr (!T) {
            return *reinterpret_cast<const u32x4_t *>(bfrag[0][0] + buf * BBYTES + ct * 32 * (kBK * 2) +
                                                      (((2 * t + kg) ^ rkey) << 4));
        } else {
            const int o = buf * BBYTES + 16 * t * kTRow;
            const u32x2_t x0 = lds_tr16(bfrag[ct][0] + o), x1 = lds_tr16(bfrag[ct][1] + o);
            return u32x4_t{x0[0], x0[1], x1[0], x1[1]};
        }
    };

    // One stage: 4 steps of RT x CT products from buffer `buf`, while the next
    // stage's operands (in registers) go to the other buffer and the loads of
    // the one after are issued.  The one barrier stands before the last step's
    // products: by then every wave has read all of this buffer and written all
    // of the other, and the products still to be issued cover the barrier and
    // the first operand reads of the next stage.  A step is cut into slices of
    // one row tile (CT products), each with its share of the vector work, and
    // the scheduler may not move work between slices: left alone it gathers the
    // vector work in front of the products, where both waves of a SIMD then wait
    // for the vector unit and later for the matrix core.
    constexpr int FA = DEEP ? 2 : 1;                // operand sets of A: 128-row wave tiles re-read in place
    u32x4_t fa[FA][RT], fb[2][CT];
    float rr[CT];
    auto scale_tiles = [&](int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i / CT][i % CT][r] *= rr[i % CT];
    };
    auto stage = [&](auto bufc, int s) {
        constexpr int buf = decltype(bufc)::value;
        const int sl = s + (DEEP ? 3 : 2) < s1 ? s + (DEEP ? 3 : 2) : s1 - 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t == 3) {
                __syncthreads();
                if (DEEP) load_w(buf ^ 1, sl);
            }
            const int nbuf = t < 3 ? buf : buf ^ 1, tn = (t + 1) & 3;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) fb[(t + 1) & 1][ct] = frag_b(nbuf, ct, tn);
            if constexpr (FA == 2) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) fa[(t + 1) & 1][rt] = frag_a(nbuf, rt, tn);
            }
            if constexpr (!T && buf == 1) {
                if (t == 3) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) rr[ct] = s_ratio[wn * 64 + ct * 32 + l31];
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    acc[rt][ct] = mfma_step<DT>(fa[t % FA][rt], fb[t & 1][ct], acc[rt][ct]);
                // forward: the sums change their unit between a group's last step and
                // the next one's first, spread over the slices of both so that it
                // stays behind the one's products and ahead of the other's
                if constexpr (!T && RT == 4) {
                    if (buf == 1 && t == 3 && rt == 1) scale_tiles(0, 1);
                    if (buf == 1 && t == 3 && rt == 2) scale_tiles(1, 3);
                    if (buf == 1 && t == 3 && rt == 3) scale_tiles(3, 4);
                    if (buf == 0 && t == 0 && rt == 0) scale_tiles(4, 6);
                    if (buf == 0 && t == 0 && rt == 1) scale_tiles(6, 8);
                } else if constexpr (!T && RT == 2) {
                    if (buf == 1 && t == 3 && rt == 1) scale_tiles(0, 2);
                    if (buf == 0 && t == 0 && rt == 0) scale_tiles(2, 4);
                }
                if (FA == 1) fa[0][rt] = frag_a(nbuf, rt, tn);
                if (t == 0) {
                    if (rt == 0) {
                        if (!DEEP) load_w(buf, sl);
                        if constexpr (T) {
                            if (buf == 1 && ((s + 1 - s0) & 3) == 0) {
                                scur = snext | zero_of(znext) << 16;
                                load_s(s + 5);
                            }
                            deq_begin(s + 1);
                        } else if (buf == 1) {
                            deq_begin(s + 1);
                            load_s(s + 3);
                        }
                    }
#pragma unroll
                    for (int i = rt * XP / RT; i < (rt + 1) * XP / RT; ++i) {
                        store_a(buf ^ 1, buf ^ 1, i);
                        load_a(buf ^ 1, sl, i);
                    }
                }
                // the 8 half-words: over steps 1 and 2 (128-row wave tiles), or 0 to 2
                const int q = FA == 1 ? (t - 1) * RT + rt : t * RT + rt, nq = FA == 1 ? 2 * RT : 3 * RT;
                if (q >= 0 && t < 3) {
#pragma unroll
                    for (int i = 8 * q / nq; i < 8 * (q + 1) / nq; ++i) deq_half(buf ^ 1, buf ^ 1, i);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    if (s0 < s1) {
        // stage s reads buffer (s - s0) % 2, its codes come through register set
        // (s - s0) % 2
        const int sn = s0 + 1 < s1 ? s0 + 1 : s0, sn2 = s0 + 2 < s1 ? s0 + 2 : s1 - 1;
#pragma unroll
        for (int i = 0; i < XP; ++i) load_a(0, s0, i);
        load_s(s0);
        load_w(0, s0);
        load_w(1, sn);
        if (DEEP) {
#pragma unroll
            for (int i = 0; i < XP; ++i) load_a(1, sn, i);
        }
#pragma unroll
        for (int i = 0; i < XP; ++i) store_a(0, 0, i);
        if (T) {
            scur = snext | zero_of(znext) << 16;
            load_s(s0 + 4);
            deq_begin(s0);
        } else {
            deq_begin(s0);
            load_s(s0 + 2);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) deq_half(0, 0, i);
        if (DEEP) load_w(0, sn2);
#pragma unroll
        for (int i = 0; i < XP; ++i) load_a(0, DEEP ? sn2 : sn, i);
        __syncthreads();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) fa[0][rt] = frag_a(0, rt, 0);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) fb[0][ct] = frag_b(0, ct, 0);
        rr[0] = rr[1] = 1.f;                          // (the sums are 0)
        int s = s0;
        for (; s + 1 < s1; s += 2) {
            stage(std::integral_constant<int, 0>{}, s);
            stage(std::integral_constant<int, 1>{}, s + 1);
        }
        // (forward slices hold whole 128-row groups)
        if (T && s < s1) stage(std::integral_constant<int, 0>{}, s);
    }
    if constexpr (KS > 1) {
        // the first group met one barrier before its stages and one in each; the
        // others wait at the ones that they have not come to
        const int most = share < b1 - b0 ? share : b1 - b0;
        for (int i = s0 < s1 ? s1 - s0 + 1 : 0; i < most + 1; ++i) __syncthreads();
    }
    __syncthreads();

    // ---- epilogue: wave tiles through LDS, rows of 8 columns per lane -----------------
    float scl[CT] = {1.f, 1.f};
    if constexpr (!T) {
        // scale that the sums are held in, per column
        s_ratio[wcol] = su.unit;
        __syncthreads();
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) scl[ct] = s_ratio[wn * 64 + ct * 32 + l31];
    }
    float *const ot = reinterpret_cast<float *>(lds) + wave_all * 32 * OUTROW;
    // the same wave tile of all wave groups, added in their order
    const float *const os = reinterpret_cast<const float *>(lds) + wave * 32 * OUTROW;
    auto sum_of = [&](int i) {
        float v = os[i];
#pragma unroll
        for (int g = 1; g < KS; ++g) v += os[g * (NT / 64) * 32 * OUTROW + i];
        return v;
    };
    auto tile_sync = [&] {
        if constexpr (KS > 1) __syncthreads();
        else wave_lds_sync();
    };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                ot[(8 * (r >> 2) + 4 * kg + (r & 3)) * OUTROW + ct * 32 + l31] = acc[rt][ct][r] * scl[ct];
        tile_sync();
        const int64_t rbase = row0 + wm * (BM / 2) + rt * 32;
        if constexpr (MODE == LIN_GLU) {
            const int64_t c0 = nt * (BN / 2) + wn * 32;
            if (c0 < p.cols / 2) {
                for (int i = 0; i < 2; ++i) {
                    const int r = i * 16 + (lane >> 2), c = (lane & 3) * 8;
                    const int64_t row = rbase + r;
                    if (row < p.M) {
                        float g[8], u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = os[r * OUTROW + c + e], u[e] = os[r * OUTROW + 32 + c + e];
                        if (p.slices > 1) {
                            float *o = p.part + ((int64_t)slice * p.M + row) * p.cols + c0 + c;
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = g[e], o[p.cols / 2 + e] = u[e];
                        } else {
                            finish_glu<DT, 8>(p, g, u, row, c0 + c);
                        }
                    }
                }
            }
        } else {
            const int64_t c0 = nt * BN + wn * 64;
            if (c0 < p.cols) {
                for (int i = grp; i < 4; i += KS) {
                    const int r = i * 8 + (lane >> 3), c = (lane & 7) * 8;
                    const int64_t row = rbase + r;
                    if (row < p.M) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = sum_of(r * OUTROW + c + e);
                        if (p.slices > 1) {
                            float *o = p.part + ((int64_t)slice * p.M + row) * p.cols + c0 + c;
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = v[e];
                        } else {
                            finish_ep<DT, 8>(p, v, row, c0 + c);
                        }
                    }
                }
            }
        }
        tile_sync();
    }
}

// Forward products of few row tiles (BM = 64 or 128 rows, 128 columns).
//
// Two wave groups of four waves share the contraction (stages of 64 elements); a
// wave owns all BM rows of 32 columns.  No other wave of its group needs those
// columns, so W never enters LDS: a lane's 16-byte slot holds 32 rows of its
// column, word t of it (8 rows) is dequantized straight into the operand of
// step t (contraction elements 32 (lane / 32) + 8 t .. + 7), and the column's scale
// stays in the lane whose sums it divides.  Only x goes through LDS: 40 KB of
// accesses per stage and group at BM = 64, where a W tile in LDS would make it 72.
//
// Bound: vector and matrix instructions of two waves per SIMD (BM = 64: 0.55 us for
// a stage of both groups, 840 vector and 512 matrix cycles), and the join where the
// rows are so few that K is sliced.  More waves would not fit the registers (4 per
// SIMD, with spills: 22 -> 32 us).  Measured (bf16, graph replay), before with W in
// LDS and one wave group: M = 128, 4096 x 14336 gated 42.5 -> 24.5 us; M = 512, 4096^2
// 35.2 -> 25.6; M = 77, 14336 x 4096 in 8 slices 33.0 -> 27.1; M = 333, 2048 x 2816
// gated fp16 18.9 -> 14.4.
template <int DT, bool GLU, int BM>
__global__ void __launch_bounds__(512, 2) lin_mid_kernel(const LinArgs p) {
    constexpr int RT = BM / 32, XP = BM / 32, KS = 2;
    constexpr int ABYTES = BM * kBK * 2, OUTROW = 36;
    constexpr int OUTBYTES = 8 * 32 * OUTROW * 4;
    constexpr int LDSBYTES = KS * 2 * ABYTES > OUTBYTES ? KS * 2 * ABYTES : OUTBYTES;
    __shared__ __attribute__((aligned(16))) uint8_t lds[LDSBYTES];

    const int tid = threadIdx.x & 255, lane = tid & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = wave_all >> 2, wn = wave_all & 3;
    const int l31 = lane & 31, kg = lane >> 5, j = lane & 15;
    const TilePos tp = tile_pos(p, (uint32_t)p.mtiles * (uint32_t)p.ntiles * (uint32_t)p.slices);
    const int64_t nt = tp.nt, row0 = tp.mt * BM, half = p.cols / 2, G = p.K / kGroup;

    // this slice's stages [b0, b1), this wave group's [s0, s1): whole 128-row groups,
    // the second group's share is the smaller one (or none)
    const int nst = (int)(p.K / kBK);
    const int b0 = tp.slice * p.stages, b1 = b0 + p.stages < nst ? b0 + p.stages : nst;
    const int share = ((b1 - b0 + 1) / 2 + 1) & ~1;
    const int s0 = b0 + grp * share < b1 ? b0 + grp * share : b1, s1 = s0 + share < b1 ? s0 + share : b1;

    // ---- x: BM rows of 64 elements per stage, two stages on the way ------------------
    uint8_t *const la = lds + grp * 2 * ABYTES;
    const uint8_t *const abase = reinterpret_cast<const uint8_t *>(p.a + row0 * p.lda);
    const int ar_ = tid >> 3, ac_ = tid & 7;
    uint32_t aoff[XP];
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        const int64_t r = row0 + i * 32 + ar_ < p.M ? i * 32 + ar_ : p.M - 1 - row0;
        aoff[i] = (uint32_t)(r * p.lda + ac_ * 8) * 2u;
    }
    uint8_t *const adst = la + ar_ * (kBK * 2) + ((ac_ ^ key_row(ar_)) << 4);
    u32x4_t ar[2][XP];
    auto load_a = [&](int d, int s, int i) { ar[d][i] = ld128(abase + (int64_t)s * (kBK * 2) + aoff[i]); };
    auto store_a = [&](int d, int i) {
        *reinterpret_cast<u32x4_t *>(adst + d * ABYTES + i * 32 * (kBK * 2)) = ar[d][i];
    };
    const uint8_t *const afrag = la + l31 * (kBK * 2);
    const int rkey = key_row(l31);
    auto frag_a = [&](int buf, int rt, int t) {
        return *reinterpret_cast<const u32x4_t *>(afrag + buf * ABYTES + rt * 32 * (kBK * 2) +
                                                  (((4 * kg + t) ^ rkey) << 4));
    };

    // ---- W: this lane's column, four stages on the way -------------------------------
    int64_t nb;
    if constexpr (GLU) {
        nb = (nt * 64 + wn * 16 + (l31 >= 16 ? half : 0)) / 16;    // 16 gate and the same 16 up columns
    } else {
        nb = nt * 8 + wn * 2 + (l31 >> 4);
        if (nb >= p.cols / 16) nb = p.cols / 16 - 1;
    }
    const uint32_t woff = (uint32_t)(nb * G * kTileBytes) + kg * 256 + j * 16;
    const uint32_t soff = (uint32_t)(nb * 16 + j);
    const uint8_t *const zbase = p.zero ? p.zero : reinterpret_cast<const uint8_t *>(p.scale);
    u32x4_t wr[4], bq[4];
    auto load_w = [&](int d, int s) {
        const int sl = s < s1 ? s : s1 - 1;
        wr[d] = ld128(p.wp + (int64_t)sl * 512 + woff);
    };
    uint16_t snext;
    uint8_t znext;
    auto load_s = [&](int s) {
        const int sl = s < s1 ? s : s1 - 1;
        const int64_t so = (int64_t)(((uint64_t)(sl >> 1) * p.gm_inv) >> 32) * p.N + soff;
        snext = p.scale[so];
        znext = zbase[so >> 1];
    };
    ScaleUnit<DT> su;
    auto next_group = [&] {
        su.next(h2f<DT>(snext), p.zero ? __builtin_amdgcn_ubfe(znext, (uint32_t)(j & 1) * 4u, 4) : 8u);
    };

    f32x16_t acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[rt][r] = 0.f;
    auto scale_tile = [&](int rt) {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[rt][r] *= su.ratio;
    };

    // One stage, D = (s - s0) % 4.  Step t's products run beside the dequantization of
    // the operand that step t - 1 has just used up (for the next stage; step 3's in
    // the next stage's step 0).  The one barrier stands before the last step's
    // products, as in the kernel above.
    u32x4_t fa[2][RT];
    auto stage = [&](auto dc, int s) {
        constexpr int D = decltype(dc)::value, buf = D & 1;
        const int sa = s + 3 < s1 ? s + 3 : s1 - 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t == 3) __syncthreads();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) fa[(t + 1) & 1][rt] = frag_a(t < 3 ? buf : buf ^ 1, rt, (t + 1) & 3);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                // the sums take the new group's unit before its first products
                if (buf == 0 && t == 0) scale_tile(rt);
                acc[rt] = mfma_step<DT>(fa[t & 1][rt], bq[t], acc[rt]);
                if (t == 0) {
#pragma unroll
                    for (int i = rt * XP / RT; i < (rt + 1) * XP / RT; ++i) {
                        store_a(buf ^ 1, i);
                        load_a(buf ^ 1, sa, i);
                    }
                }
                const int q = (t + 3) & 3;
                const uint32_t w = wr[t == 0 ? D : (D + 1) & 3][q];
                if (rt == RT / 2 - 1) su.template dequant<0>(w, bq[q]);
                if (rt == RT - 1) su.template dequant<1>(w, bq[q]);
                if (t == 0 && rt == RT - 1) {
                    load_w(D, s + 4);
                    // the next stage's group, and the scales of the one after it
                    if (buf == 1) {
                        next_group();
                        load_s(s + 3);
                    }
                }
                if (t == 2 && rt == 0 && buf == 1) su.change();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    if (s0 < s1) {
        const int sn = s0 + 1 < s1 ? s0 + 1 : s1 - 1, sn2 = s0 + 2 < s1 ? s0 + 2 : s1 - 1;
#pragma unroll
        for (int i = 0; i < XP; ++i) load_a(0, s0, i);
        load_s(s0);
#pragma unroll
        for (int d = 0; d < 4; ++d) load_w(d, s0 + d);
#pragma unroll
        for (int i = 0; i < XP; ++i) load_a(1, sn, i);
#pragma unroll
        for (int i = 0; i < XP; ++i) store_a(0, i);
        next_group();
        su.change();
        load_s(s0 + 2);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            su.template dequant<0>(wr[0][t], bq[t]);
            su.template dequant<1>(wr[0][t], bq[t]);
        }
#pragma unroll
        for (int i = 0; i < XP; ++i) load_a(0, sn2, i);
        __syncthreads();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) fa[0][rt] = frag_a(0, rt, 0);
        int s = s0;
        for (; s + 2 < s1; s += 4) {
            stage(std::integral_constant<int, 0>{}, s);
            stage(std::integral_constant<int, 1>{}, s + 1);
            stage(std::integral_constant<int, 2>{}, s + 2);
            stage(std::integral_constant<int, 3>{}, s + 3);
        }
        if (s < s1) {
            stage(std::integral_constant<int, 0>{}, s);
            stage(std::integral_constant<int, 1>{}, s + 1);
        }
    }
    // The first group met one barrier before its stages and one in each; the second
    // waits at the ones that it has not come to.
    for (int i = s0 < s1 ? s1 - s0 + 1 : 0; i < (share < b1 - b0 ? share : b1 - b0) + 1; ++i) __syncthreads();

    // ---- epilogue: wave tiles through LDS, rows of 8 columns per lane; wave group g
    // finishes the row tiles rt = g (mod 2) -----------------------------------------------
    float *const ot = reinterpret_cast<float *>(lds) + wave_all * 32 * OUTROW;
    const float *const os = reinterpret_cast<const float *>(lds) + wn * 32 * OUTROW;
    auto sum_of = [&](int i) { return os[i] + os[4 * 32 * OUTROW + i]; };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; ++r) ot[(8 * (r >> 2) + 4 * kg + (r & 3)) * OUTROW + l31] = acc[rt][r] * su.unit;
        __syncthreads();
        if ((rt & 1) != grp) continue;
        const int64_t rbase = row0 + rt * 32;
        if constexpr (GLU) {
            const int r = lane >> 1, c = (lane & 1) * 8;
            const int64_t row = rbase + r, col = nt * 64 + wn * 16 + c;
            if (row < p.M) {
                float g[8], u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = sum_of(r * OUTROW + c + e), u[e] = sum_of(r * OUTROW + 16 + c + e);
                if (p.slices > 1) {
                    float *o = p.part + ((int64_t)tp.slice * p.M + row) * p.cols + col;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = g[e], o[half + e] = u[e];
                } else {
                    finish_glu<DT, 8>(p, g, u, row, col);
                }
            }
        } else {
            const int64_t col = nt * 128 + wn * 32 + (lane & 3) * 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = i * 16 + (lane >> 2), c = (lane & 3) * 8;
                const int64_t row = rbase + r;
                if (row >= p.M || col >= p.cols) continue;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = sum_of(r * OUTROW + c + e);
                if (p.slices > 1) {
                    float *o = p.part + ((int64_t)tp.slice * p.M + row) * p.cols + col;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = v[e];
                } else {
                    finish_ep<DT, 8>(p, v, row, col);
                }
            }
        }
    }
}

// Bound by memory: slices x M x cols x 4 bytes in; 4.3 us for three slices of
// 519 x 2048.
//
// Sum of the slices' partial results in ascending slice order, then the
// finishing step; 8 columns per thread.
template <int DT, bool GLU>
__global__ void __launch_bounds__(256) lin_join_kernel(const LinArgs p) {
    const int64_t width = GLU ? p.cols / 2 : p.cols, nv = width / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M * nv; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / nv, col = i % nv * 8;
        float v[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.f;
        for (int s = 0; s < p.slices; ++s) {
            const float *o = p.part + ((int64_t)s * p.M + row) * p.cols + col;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] += o[e];
                if constexpr (GLU) u[e] += o[width + e];
            }
        }
        if constexpr (GLU) finish_glu<DT, 8>(p, v, u, row, col);
        else finish_ep<DT, 8>(p, v, row, col);
    }
}

// Bound by memory: dy and h are read and d is written once (gated, 4096 x 28672:
// 587 MB in 98 us, 6.0 TB/s; the column sums come with it).
//
// d (and with it the column sums, of the unrounded values) from dy and the saved
// pre-activation.  The product reads d back as it is stored, in 16 bits: forming it again
// from dy and h per column tile cost 1.3 us a stage.  A
// workgroup takes 512 columns (glu: of each half) and every gridDim.y-th block
// of four rows; a thread owns 8 columns of one row in each block and sums its
// rows in ascending order.  The four rows' sums meet in LDS, the workgroups'
// sums in the product's extra workgroups: every sum has a fixed order.
template <int DT, bool GLU>
__global__ void __launch_bounds__(256)
lin_dact_kernel(const uint16_t *dy, int64_t lddy, const uint16_t *h, uint16_t *d, float *part, int64_t M, int64_t N,
                int act) {
    const int64_t W = GLU ? N / 2 : N;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t col = ((int64_t)blockIdx.x * 64 + tx) * 8;
    float s0[8], s1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s0[e] = s1[e] = 0.f;
    if (col < W) {
        for (int64_t row = (int64_t)blockIdx.y * 4 + ty; row < M; row += (int64_t)gridDim.y * 4) {
            float g[8], v[8];
            load_vec<DT, 8>(dy + row * lddy + col, v);
            if (GLU || act != ACT_NONE) load_vec<DT, 8>(h + row * N + col, g);
            if constexpr (GLU) {
                float u[8];
                load_vec<DT, 8>(h + row * N + W + col, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f, df;
                    act_both(g[e], act, f, df);
                    g[e] = v[e] * u[e] * df;
                    u[e] = v[e] * f;
                    s0[e] += g[e];
                    s1[e] += u[e];
                }
                store_vec<DT, 8>(d + row * N + col, g);
                store_vec<DT, 8>(d + row * N + W + col, u);
            } else {
                if (act != ACT_NONE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float f, df;
                        act_both(g[e], act, f, df);
                        v[e] *= df;
                    }
                    store_vec<DT, 8>(d + row * N + col, v);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s0[e] += v[e];
            }
        }
    }
    if (!part) return;
    __shared__ float red[4][GLU ? 2 : 1][8][64];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[ty][0][e][tx] = s0[e];
        if constexpr (GLU) red[ty][1][e][tx] = s1[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (GLU ? 2 : 1) * 512; i += 256) {
        const int half = i >> 9, c = i & 511;
        const int64_t cc = (int64_t)blockIdx.x * 512 + c;
        if (cc >= W) continue;
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) s += red[y][half][c & 7][c >> 3];
        part[(int64_t)blockIdx.y * N + half * W + cc] = s;
    }
}

// ---- plans and launches ---------------------------------------------------------

struct WidePlan { int bm, bn; int slices, stages, mtiles, ntiles; double us; };

// Tile shape and slice count by estimated time.  A workgroup's step (a stage, with
// two wave groups one of each) takes `alone` us while compute units are idle and
// `shared` us where all are busy (the clock drops and L2 is shared), plus `ends` us
// for its first loads and its epilogue; slices write and read their fp32 sums at
// about 5 TB/s and cost another launch.  The constants are fits to timings over
// 20 sizes (M = 64..4096, matrices from 1024 x 1024 to 4096 x 28672, both directions);
// on 40 random ones the choice was within 6% of the best of all shapes and slice
// counts on 38 and within 8% on another.  Few tiles want small ones and slices, many
// the large one, whose dequantization serves 256 rows: M = 128, 4096^2 16 us with
// 64 x 128 and four slices, 56 with 128 x 256 unsliced; M = 512, 4096 x 14336 70 us with
// 128 x 256, 95 with 64 x 128.
struct Shape { int bm, bn; double alone, shared, ends; };
static constexpr Shape kForward[] = {{64, 128, 0.55, 0.68, 2.0},
                                     {128, 128, 0.79, 1.09, 3.5},
                                     {128, 256, 0.88, 1.08, 4.0},
                                     {256, 256, 1.36, 1.62, 8.0}};
static constexpr Shape kTransposed[] = {{64, 128, 0.71, 0.85, 1.5},
                                        {128, 128, 0.89, 1.14, 3.0},
                                        {128, 256, 0.88, 1.08, 4.0},
                                        {256, 256, 1.38, 1.65, 8.0}};
constexpr int kShapeCount = (int)(sizeof(kForward) / sizeof(kForward[0]));
static std::atomic<int> g_lin_shape{-1}, g_lin_slices{0};     // test hook: -1 and 0 choose

int lin_shape_count() { return kShapeCount; }
void set_lin_plan(int shape, int slices) {
    g_lin_shape.store(shape, std::memory_order_relaxed);
    g_lin_slices.store(slices, std::memory_order_relaxed);
}

static WidePlan wide_plan(int mode, int64_t M, int64_t K, int64_t N) {
    static constexpr int kSlices[] = {1, 2, 3, 4, 6, 8, 12, 16};
    constexpr int64_t kCus = 256;
    const int shape = g_lin_shape.load(std::memory_order_relaxed);
    const int forced = g_lin_slices.load(std::memory_order_relaxed);
    const int64_t cols = mode == LIN_T ? K : N;
    const int nst = (int)((mode == LIN_T ? N : K) / kBK);
    WidePlan best{};
    const Shape *const shapes = mode == LIN_T ? kTransposed : kForward;
    for (int si = 0; si < kShapeCount; ++si)
        for (int want : kSlices) {
            const Shape &sh = shapes[si];
            if (shape >= 0 && shape < kShapeCount && si != shape) continue;
            if (forced > 0 && want != 1 && want != forced) continue;
            WidePlan w{};
            w.bm = sh.bm;
            w.bn = sh.bn;
            w.mtiles = (int)((M + w.bm - 1) / w.bm);
            w.ntiles = (int)((cols + w.bn - 1) / w.bn);
            w.stages = (nst + want - 1) / want;
            w.stages += w.stages & 1;                  // whole 128-row groups (forward)
            w.slices = (nst + w.stages - 1) / w.stages;
            if (want > 1 && (w.slices != want || (w.stages < 4 && want != forced))) continue;
            const int64_t wgs = (int64_t)w.mtiles * w.ntiles * w.slices;
            const double load = wgs <= kCus ? (double)wgs / kCus : (double)((wgs + kCus - 1) / kCus);
            const int groups = wide_groups(w.bm, w.bn);         // a wave group's share: as in the kernel
            const int steps = groups == 1 ? w.stages : ((w.stages + groups - 1) / groups + 1) & ~1;
            const double one = steps * sh.alone + sh.ends, all = load * (steps * sh.shared + sh.ends);
            double us = one > all ? one : all;
            if (w.slices > 1) us += 3.0 + 8e-6 / 5.0 * w.slices * (double)M * (double)cols;
            if (best.bm == 0 || us < best.us || want == forced) {
                best = w;
                best.us = us;
            }
        }
    return best;
}

LinPlan lin_plan(int mode, int64_t M, int64_t K, int64_t N) {
    LinPlan plan{};
    // a forced tile shape also takes the rows that the decode kernels would
    const bool free = g_lin_shape.load(std::memory_order_relaxed) < 0;
    plan.small = free && lin_small_ok(mode, M);
    if (!plan.small) {
        const WidePlan w = wide_plan(mode, M, K, N);
        // (a launch and its first loads take the tile kernels 2.8 us besides their stages;
        // 32 rows in more than eight slices 2 us more: each has few stages and more to join)
        const double tiles = w.us + 2.8 + (M <= 32 && w.slices > 8 ? 2.5 : 0.0);
        plan.small = free && lin_small_us(mode, M, K, N) < tiles;
        plan.bm = w.bm;
        plan.bn = w.bn;
        plan.slices = w.slices;
        plan.stages = w.stages;
        plan.mtiles = w.mtiles;
        plan.ntiles = w.ntiles;
        if (w.slices > 1)
            plan.workspace_bytes = (size_t)w.slices * (size_t)M * (size_t)(mode == LIN_T ? K : N) * sizeof(float);
    }
    if (plan.small) plan.workspace_bytes = lin_small_workspace_bytes(mode, M, K, N);
    return plan;
}

template <int DT, int MODE>
static hipError_t wide_launch(const LinArgs &p, int bm, int bn, hipStream_t stream) {
    const int64_t total = (int64_t)p.mtiles * p.ntiles * p.slices;
    const int64_t extra = MODE == LIN_T && p.colsum ? p.N / 64 : 0;
    if (total + extra > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(total + extra)), block((unsigned)(wide_groups(bm, bn) * 2 * bn));
    if constexpr (MODE != LIN_T) {
        if (bn == 128) {
            if (bm == 64) hipLaunchKernelGGL((lin_mid_kernel<DT, MODE == LIN_GLU, 64>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((lin_mid_kernel<DT, MODE == LIN_GLU, 128>), grid, block, 0, stream, p);
            return hipGetLastError();
        }
    } else if (bn == 128) {
        if (bm == 64) hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 64, 128>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 128, 128>), grid, block, 0, stream, p);
        return hipGetLastError();
    }
    if (bm == 128 && bn == 256) hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 128, 256>), grid, block, 0, stream, p);
    else if (bm == 256 && bn == 256) hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 256, 256>), grid, block, 0, stream, p);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

template <int DT, bool GLU>
static hipError_t join_go(const LinArgs &p, hipStream_t stream) {
    const int64_t work = p.M * ((GLU ? p.cols / 2 : p.cols) / 8), blocks = (work + 255) / 256;
    hipLaunchKernelGGL((lin_join_kernel<DT, GLU>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_lin_join(int mode, const LinArgs &p, int dt, hipStream_t stream) {
    if (dt == DT_BF16) return mode == LIN_GLU ? join_go<DT_BF16, true>(p, stream) : join_go<DT_BF16, false>(p, stream);
    return mode == LIN_GLU ? join_go<DT_F16, true>(p, stream) : join_go<DT_F16, false>(p, stream);
}

template <int DT>
static hipError_t wide_dt(int mode, const LinArgs &p, const LinPlan &plan, hipStream_t stream) {
    if (mode == LIN_EP) return wide_launch<DT, LIN_EP>(p, plan.bm, plan.bn, stream);
    if (mode == LIN_GLU) return wide_launch<DT, LIN_GLU>(p, plan.bm, plan.bn, stream);
    return wide_launch<DT, LIN_T>(p, plan.bm, plan.bn, stream);
}

hipError_t launch_lin(int mode, LinArgs p, const LinPlan &plan, int dt, void *workspace, hipStream_t stream) {
    if (plan.small) return launch_lin_small(mode, p, dt, workspace, stream);
    p.slices = plan.slices;
    p.stages = plan.stages;
    p.mtiles = plan.mtiles;
    p.ntiles = plan.ntiles;
    p.part = (float *)workspace;
    p.gm_inv = ((uint64_t(1) << 32) + p.gm - 1) / p.gm;
    hipError_t err = dt == DT_BF16 ? wide_dt<DT_BF16>(mode, p, plan, stream) : wide_dt<DT_F16>(mode, p, plan, stream);
    return err == hipSuccess && p.slices > 1 ? launch_lin_join(mode, p, dt, stream) : err;
}

// Row blocks of the activation gradient, one partial row of column sums each:
// one row per thread (four per block) up to 64 blocks.
int lin_dact_blocks(int64_t M) {
    const int64_t b = (M + 3) / 4;
    return (int)(b < 1 ? 1 : b > 64 ? 64 : b);
}

size_t lin_dact_workspace_bytes(int64_t M, int64_t N) { return (size_t)lin_dact_blocks(M) * (size_t)N * sizeof(float); }

hipError_t launch_lin_dact(bool glu, const uint16_t *dy, int64_t lddy, const uint16_t *h, uint16_t *d, int64_t M,
                           int64_t N, int act, int dt, float *part, hipStream_t stream) {
    const int64_t W = glu ? N / 2 : N;
    const dim3 grid((unsigned)((W + 511) / 512), (unsigned)lin_dact_blocks(M));
#define W4_DACT(DTV, GLUV)                                                                                       \
    hipLaunchKernelGGL((lin_dact_kernel<DTV, GLUV>), grid, dim3(256), 0, stream, dy, lddy, h, d, part, M, N, act)
    if (dt == DT_BF16) {
        if (glu) W4_DACT(DT_BF16, true);
        else W4_DACT(DT_BF16, false);
    } else {
        if (glu) W4_DACT(DT_F16, true);
        else W4_DACT(DT_F16, false);
    }
#undef W4_DACT
    return hipGetLastError();
}

hipError_t launch_lin_zero_colsum(float *colsum, int64_t N, hipStream_t stream) {
    hipLaunchKernelGGL(lin_colsum_kernel, dim3((unsigned)(N / 64)), dim3(512), 0, stream, nullptr, colsum, N, 0);
    return hipGetLastError();
}

}  // namespace w4
