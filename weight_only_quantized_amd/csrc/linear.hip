// linear.hip — products of the fused linear operators on tiles of 256 columns:
// forward (x . W with its epilogue, plain or gated) and transposed (d . W^T).
#include "act.hpp"

namespace w4 {

constexpr int kXcd = 8;              // XCDs; workgroups go to them round-robin
constexpr int kBK = 64;              // contraction elements per stage
constexpr int kWideN = 256;          // columns per workgroup
constexpr int kTRow = 576;           // LDS row stride (bytes) of the transposed W tile

typedef short v4s_t __attribute__((__vector_size__(8)));
typedef v4s_t __attribute__((address_space(3))) *lds_v4s_ptr;

// Four 16-bit elements of one column from four LDS rows: the 16 lanes of a
// group read 4 rows x 16 columns (lane 4 r + c addresses row r, columns 4 c ..)
// and lane i gets column i.
__device__ __forceinline__ u32x2_t lds_tr16(const uint8_t *p) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_ptr)(v4s_t *)(uint8_t *)p));
}

template <int DT, int MODE, int BM>
__global__ void __launch_bounds__(512, 2) lin_wide_kernel(const LinArgs p) {
    constexpr bool T = MODE == LIN_T;
    constexpr int RT = BM / 64, CT = 2;              // 32 x 32 tiles per wave (2 x 4 waves)
    constexpr int XP = BM / 64;                      // 16-byte A chunks per thread and stage
    constexpr int ABYTES = BM * kBK * 2;
    constexpr int BBYTES = T ? kBK * kTRow : kWideN * kBK * 2;
    constexpr int OUTROW = 68;                       // floats per row of the output staging
    constexpr int LDSBYTES = 2 * (ABYTES + BBYTES);
    static_assert(LDSBYTES >= 8 * 32 * OUTROW * 4, "output staging fits");
    __shared__ __attribute__((aligned(16))) uint8_t lds[LDSBYTES];
    __shared__ float s_ratio[2][kWideN];             // per column: factor on the sums at a new scale group
    uint8_t *const lda_ = lds, *const ldb_ = lds + 2 * ABYTES;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int l31 = lane & 31, kg = lane >> 5;

    // ---- tile of this workgroup ------------------------------------------------
    const int64_t total = (int64_t)p.mtiles * p.ntiles * p.slices;
    const int64_t id = blockIdx.x, xcd = id % kXcd;
    const int64_t q8 = total / kXcd, r8 = total % kXcd;
    const int64_t idx = xcd * q8 + (xcd < r8 ? xcd : r8) + id / kXcd;
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
    const int slice = (int)(idx / tiles);
    const int64_t tile = idx % tiles;
    constexpr int GM = 4;
    const int64_t grp = tile / (GM * p.ntiles), m_first = grp * GM;
    const int64_t gmt = p.mtiles - m_first < GM ? p.mtiles - m_first : GM;
    const int64_t rem = tile - m_first * p.ntiles;
    const int64_t row0 = (m_first + rem % gmt) * BM;
    const int64_t nt = rem / gmt;

    const int64_t G = p.K / kGroup;
    const int nst = (int)((T ? p.N : p.K) / kBK);
    const int s0 = slice * p.stages, s1 = s0 + p.stages < nst ? s0 + p.stages : nst;

    // ---- A operand: BM rows of 64 elements per stage ------------------------------
    const uint16_t *arow[XP];
    int aoff[XP];
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        const int id16 = i * 512 + tid, r = id16 >> 3, c = id16 & 7;
        const int64_t gr = row0 + r < p.M ? row0 + r : p.M - 1;
        arow[i] = p.a + gr * p.lda + c * 8;
        aoff[i] = r * (kBK * 2) + ((c ^ (r & 7)) << 4);
    }
    u32x4_t ar[XP];
    auto load_a = [&](int s) {
#pragma unroll
        for (int i = 0; i < XP; ++i) ar[i] = ld128(arow[i] + (int64_t)s * kBK);
    };
    auto store_a = [&](int buf) {
#pragma unroll
        for (int i = 0; i < XP; ++i) *reinterpret_cast<u32x4_t *>(lda_ + buf * ABYTES + aoff[i]) = ar[i];
    };

    // ---- W operand: one 16-byte slot (32 rows of one column) per thread -----------
    const int j = lane & 15;
    const uint8_t *wptr;
    const uint16_t *sptr;
    // without zero points the scales' own bytes are read and ignored: no branch
    // around a load
    const uint8_t *zptr = p.zero ? p.zero : reinterpret_cast<const uint8_t *>(p.scale);
    int64_t wstep;
    int boff[4];
    int wcol = 0;                                     // forward: column within the tile
    int64_t ncol = 0;                                 // forward: column of W
    if constexpr (!T) {
        const int cb = 2 * wave + (lane >> 5), c32 = (lane >> 4) & 1;
        int64_t nb;
        if constexpr (MODE == LIN_GLU) {
            // 4 blocks per consuming wave: two gate, then the two up blocks of the same columns
            const int64_t half = p.cols / 2;
            int64_t c0 = nt * (kWideN / 2) + (cb >> 2) * 32 + (cb & 1) * 16;
            if (c0 >= half) c0 = half - 16;
            nb = ((cb & 2) ? half + c0 : c0) / 16;
        } else {
            nb = nt * (kWideN / 16) + cb;
            if (nb >= p.cols / 16) nb = p.cols / 16 - 1;
        }
        wcol = cb * 16 + j;
        ncol = nb * 16 + j;
        wptr = p.wp + nb * G * kTileBytes + c32 * 256 + j * 16;
        wstep = 512;
        sptr = p.scale + ncol;
        zptr += ncol >> 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) boff[t] = wcol * (kBK * 2) + (((4 * c32 + t) ^ (wcol & 7)) << 4);
    } else {
        const int nbi = wave & 3, gi = wave >> 2, c32 = lane >> 4;
        int64_t g = nt * 2 + gi;
        if (g >= G) g = G - 1;
        wptr = p.wp + (nbi * G + g) * kTileBytes + lane * 16;
        wstep = 4 * G * kTileBytes;
        sptr = p.scale + g / p.gm * p.N + nbi * 16 + j;
        zptr += (g / p.gm * p.N + nbi * 16 + j) >> 1;
        const int n = nbi * 16 + j;
#pragma unroll
        for (int t = 0; t < 4; ++t) boff[t] = n * kTRow + (((gi * 16 + c32 * 4 + t) ^ ((n >> 2) & 1)) << 4);
    }
    u32x4_t wr;
    uint16_t sr;
    uint8_t zr;
    auto load_w = [&](int s) {
        wr = ld128(wptr + (int64_t)s * wstep);
        const int64_t so = T ? (int64_t)s * kBK : (int64_t)(s >> 1) / p.gm * p.N;
        sr = sptr[so];
        zr = zptr[so >> 1];
    };
    float se = 0.f;                                   // forward: scale the sums are held in
    auto store_w = [&](int buf) {
        const float s = h2f<DT>(sr);
        const uint32_t z = p.zero ? __builtin_amdgcn_ubfe((uint32_t)zr, (uint32_t)(j & 1) * 4u, 4) : 8u;
        uint8_t *base = ldb_ + buf * BBYTES;
        float f = 1.f;
        if constexpr (!T) {
            float ratio;
            const float as_ = __builtin_fabsf(s);
            if (as_ >= 0x1p-60f * __builtin_fabsf(se) && as_ >= 0x1p-100f) {
                ratio = se * __builtin_amdgcn_rcpf(s);
                se = s;
            } else {
                if (se == 0.f) se = 1.f;
                ratio = 1.f;
                f = s * __builtin_amdgcn_rcpf(se);
            }
            if (((lane >> 4) & 1) == 0) s_ratio[buf][wcol] = ratio;
        }
        const bool rare = !T && __any(f != 1.f);
        if constexpr (DT == DT_BF16) {
            const float zf = (float)z, zs = -zf * s;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t w = wr[t];
                const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
                // bytes of lo: rows 0, 4, 1, 5; of hi: rows 2, 6, 3, 7
                float v[8];
                v[0] = (float)(lo & 0xFFu), v[4] = (float)((lo >> 8) & 0xFFu);
                v[1] = (float)((lo >> 16) & 0xFFu), v[5] = (float)(lo >> 24);
                v[2] = (float)(hi & 0xFFu), v[6] = (float)((hi >> 8) & 0xFFu);
                v[3] = (float)((hi >> 16) & 0xFFu), v[7] = (float)(hi >> 24);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = T ? __builtin_fmaf(v[i], s, zs) : v[i] - zf;
                if (rare) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= f;
                }
                u32x4_t o;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bf16x2_t b = {(__bf16)v[2 * q], (__bf16)v[2 * q + 1]};
                    o[q] = __builtin_bit_cast(uint32_t, b);
                }
                *reinterpret_cast<u32x4_t *>(base + boff[t]) = o;
            }
        } else {
            const _Float16 m = (_Float16)(T ? s : f);
            const f16x2_t m2 = {m, m};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u32x4_t o = dequant_word<DT>(wr[t], f16_negbias2(z));
                if (T || rare) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[q] = __builtin_bit_cast(uint32_t, as<f16x2_t>(o[q]) * m2);
                }
                *reinterpret_cast<u32x4_t *>(base + boff[t]) = o;
            }
        }
    };

    // ---- main loop ---------------------------------------------------------------
    f32x16_t acc[RT][CT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[rt][ct][r] = 0.f;

    const int abase = (wm * (BM / 2) + l31) * (kBK * 2);
    auto frag_a = [&](int buf, int rt, int t) {
        return *reinterpret_cast<const u32x4_t *>(lda_ + buf * ABYTES + abase + rt * 32 * (kBK * 2) +
                                                  (((2 * t + kg) ^ (lane & 7)) << 4));
    };
    const int qq = lane >> 4, tr = (lane & 15) >> 2, tc = lane & 3;
    auto frag_b = [&](int buf, int ct, int t) -> u32x4_t {
        if constexpr (!T) {
            const int col = wn * 64 + ct * 32 + l31;
            return *reinterpret_cast<const u32x4_t *>(ldb_ + buf * BBYTES + col * (kBK * 2) +
                                                      (((2 * t + kg) ^ (lane & 7)) << 4));
        } else {
            const int n = 16 * t + 8 * (qq >> 1) + tr;
            const int ch = wn * 8 + ct * 4 + 2 * (qq & 1) + (tc >> 1);
            const uint8_t *b = ldb_ + buf * BBYTES + n * kTRow + (tc & 1) * 8;
            const u32x2_t x0 = lds_tr16(b + (ch << 4)), x1 = lds_tr16(b + 4 * kTRow + ((ch ^ 1) << 4));
            return u32x4_t{x0[0], x0[1], x1[0], x1[1]};
        }
    };

    if (s0 < s1) {
        load_a(s0);
        load_w(s0);
        store_a(0);
        store_w(0);
        const int sn = s0 + 1 < s1 ? s0 + 1 : s0;
        load_a(sn);
        load_w(sn);
        __syncthreads();
        for (int s = s0; s < s1; ++s) {
            const int buf = (s - s0) & 1;
            if constexpr (!T) {
                if (s == s0 || s % (2 * p.gm) == 0) {
                    float rr[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) rr[ct] = s_ratio[buf][wn * 64 + ct * 32 + l31];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[rt][ct][r] *= rr[ct];
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u32x4_t a[RT], b[CT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) a[rt] = frag_a(buf, rt, t);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) b[ct] = frag_b(buf, ct, t);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = mfma32x32x16<DT>(a[rt], b[ct], acc[rt][ct]);
                if (t == 1) {
                    // the next stage's operands: their buffer was last read before
                    // the previous barrier
                    store_a(buf ^ 1);
                    store_w(buf ^ 1);
                    const int sl = s + 2 < s1 ? s + 2 : s1 - 1;
                    load_a(sl);
                    load_w(sl);
                }
            }
            __syncthreads();
        }
    }

    // ---- epilogue: wave tiles through LDS, rows of 8 columns per lane -----------------
    float scl[CT] = {1.f, 1.f};
    if constexpr (!T) {
        // scale that the sums are held in, per column
        if (((lane >> 4) & 1) == 0) s_ratio[0][wcol] = se;
        __syncthreads();
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) scl[ct] = s_ratio[0][wn * 64 + ct * 32 + l31];
    }
    float *const ot = reinterpret_cast<float *>(lds) + wave * 32 * OUTROW;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                ot[(8 * (r >> 2) + 4 * kg + (r & 3)) * OUTROW + ct * 32 + l31] = acc[rt][ct][r] * scl[ct];
        __syncthreads();
        const int64_t rbase = row0 + wm * (BM / 2) + rt * 32;
        if constexpr (MODE == LIN_GLU) {
            const int64_t c0 = nt * (kWideN / 2) + wn * 32;
            if (c0 < p.cols / 2) {
                for (int i = 0; i < 2; ++i) {
                    const int r = i * 16 + (lane >> 2), c = (lane & 3) * 8;
                    const int64_t row = rbase + r;
                    if (row < p.M) {
                        float g[8], u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = ot[r * OUTROW + c + e], u[e] = ot[r * OUTROW + 32 + c + e];
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
            const int64_t c0 = nt * kWideN + wn * 64;
            if (c0 < p.cols) {
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 3), c = (lane & 7) * 8;
                    const int64_t row = rbase + r;
                    if (row < p.M) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = ot[r * OUTROW + c + e];
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
        __syncthreads();
    }
}

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

// d (and with it the column sums) from dy and the saved pre-activation.  A
// workgroup takes 512 columns (glu: of each half) and every gridDim.y-th block
// of four rows; a thread owns 8 columns of one row in each block and sums its
// rows in ascending order.  The four rows' sums meet in LDS, the workgroups'
// sums in lin_colsum_kernel: every sum has a fixed order.
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

__global__ void __launch_bounds__(256) lin_colsum_kernel(const float *part, float *colsum, int64_t N, int blocks) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= N) return;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += part[(int64_t)b * N + c];
    colsum[c] = s;
}

// ---- plans and launches ---------------------------------------------------------

struct WidePlan { int bm; int slices, stages, mtiles, ntiles; };

static WidePlan wide_plan(int mode, int64_t M, int64_t K, int64_t N) {
    WidePlan w{};
    const int64_t cols = mode == LIN_T ? K : N;
    const int nst = (int)((mode == LIN_T ? N : K) / kBK);
    w.ntiles = (int)((cols + kWideN - 1) / kWideN);
    w.bm = M <= 64 ? 64 : M <= 128 ? 128 : 256;
    w.mtiles = (int)((M + w.bm - 1) / w.bm);
    int slices = 1;
    while ((int64_t)w.mtiles * w.ntiles * slices < 192 && nst / (2 * slices) >= 8) slices *= 2;
    w.stages = (nst + slices - 1) / slices;
    w.slices = (nst + w.stages - 1) / w.stages;
    return w;
}

size_t lin_workspace_bytes(int mode, int64_t M, int64_t K, int64_t N) {
    if (M <= 0 || (mode != LIN_T && lin_small_ok(mode, M, K, N))) return 0;
    const WidePlan w = wide_plan(mode, M, K, N);
    return w.slices > 1 ? (size_t)w.slices * (size_t)M * (size_t)(mode == LIN_T ? K : N) * sizeof(float) : 0;
}

template <int DT, int MODE>
static hipError_t wide_launch(const LinArgs &p, int bm, hipStream_t stream) {
    const int64_t total = (int64_t)p.mtiles * p.ntiles * p.slices;
    if (total > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)total), block(512);
    if (bm == 64) hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 64>), grid, block, 0, stream, p);
    else if (bm == 128) hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 128>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((lin_wide_kernel<DT, MODE, 256>), grid, block, 0, stream, p);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.slices == 1) return err;
    const int64_t work = p.M * ((MODE == LIN_GLU ? p.cols / 2 : p.cols) / 8);
    const int64_t blocks = (work + 255) / 256;
    hipLaunchKernelGGL((lin_join_kernel<DT, MODE == LIN_GLU>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0,
                       stream, p);
    return hipGetLastError();
}

hipError_t launch_lin(int mode, LinArgs p, int dt, void *workspace, hipStream_t stream) {
    if (mode != LIN_T && lin_small_ok(mode, p.M, p.K, p.N)) return launch_lin_small(mode, p, dt, stream);
    const WidePlan w = wide_plan(mode, p.M, p.K, p.N);
    p.slices = w.slices;
    p.stages = w.stages;
    p.mtiles = w.mtiles;
    p.ntiles = w.ntiles;
    p.part = (float *)workspace;
    if (dt == DT_BF16) {
        if (mode == LIN_EP) return wide_launch<DT_BF16, LIN_EP>(p, w.bm, stream);
        if (mode == LIN_GLU) return wide_launch<DT_BF16, LIN_GLU>(p, w.bm, stream);
        return wide_launch<DT_BF16, LIN_T>(p, w.bm, stream);
    }
    if (mode == LIN_EP) return wide_launch<DT_F16, LIN_EP>(p, w.bm, stream);
    if (mode == LIN_GLU) return wide_launch<DT_F16, LIN_GLU>(p, w.bm, stream);
    return wide_launch<DT_F16, LIN_T>(p, w.bm, stream);
}

// Row blocks of the column sums: enough workgroups to fill the machine, at
// least four rows per thread, at most 64 partial rows.
static int dact_blocks(int64_t M) {
    const int64_t b = (M + 15) / 16;
    return (int)(b < 1 ? 1 : b > 64 ? 64 : b);
}

size_t lin_dact_workspace_bytes(int64_t M, int64_t N) { return (size_t)dact_blocks(M) * (size_t)N * sizeof(float); }

hipError_t launch_lin_dact(bool glu, const uint16_t *dy, int64_t lddy, const uint16_t *h, uint16_t *d, float *colsum,
                           int64_t M, int64_t N, int act, int dt, void *part, hipStream_t stream) {
    const int64_t W = glu ? N / 2 : N;
    int blocks = 0;
    if (M > 0) {
        blocks = dact_blocks(M);
        const dim3 grid((unsigned)((W + 511) / 512), (unsigned)blocks);
        float *ps = colsum ? (float *)part : nullptr;
#define W4_DACT(DTV, GLUV)                                                                                       \
    hipLaunchKernelGGL((lin_dact_kernel<DTV, GLUV>), grid, dim3(256), 0, stream, dy, lddy, h, d, ps, M, N, act)
        if (dt == DT_BF16) {
            if (glu) W4_DACT(DT_BF16, true);
            else W4_DACT(DT_BF16, false);
        } else {
            if (glu) W4_DACT(DT_F16, true);
            else W4_DACT(DT_F16, false);
        }
#undef W4_DACT
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (!colsum) return hipSuccess;
    hipLaunchKernelGGL(lin_colsum_kernel, dim3((unsigned)((N + 255) / 256)), dim3(256), 0, stream, (const float *)part,
                       colsum, N, blocks);
    return hipGetLastError();
}

}  // namespace w4
