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
// A group of LPT lanes owns a token, EPL experts each, all of a token's work in
// registers; 64 / LPT tokens share a wave.  Choosing takes topk rounds of "largest that is left",
// each a maximum over EPL registers and log2 LPT lane exchanges (16-bit types: over the lanes' first keys,
// which each lane has sorted).  Bounds: up to a few hundred tokens the launch (16 x 64 with counts and loss
// 5.3 us); then the forward pass's instructions, about 6 us for 16384 x 256 and as much again for the
// counts, whose join over workgroups is a launch of its own (13.1 us; the workspace comes with any contents, so no
// workgroup can know that it is the last before a launch has cleared the ticket); the backward pass, whose
// workgroups have few passes each: a load, the softmax, five steps through LDS and a store in turn (16384
// x 256 in bf16: 7.0 us, 2.6 TB/s of the 4.9 of a large copy; 100 experts 5.7, 318 13.0; fp32: 9.4).
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace w4 {

enum { DT_F32 = 2 };

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
    return lane_reduce<LPT>(v, [](float a, float b) { return a + b; });
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
    return lane_reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}

// ---- logits -----------------------------------------------------------------

template <int DT>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float v) {
    if constexpr (DT == DT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<uint16_t *>(p)[i] = f2h<DT>(v);
}

// Experts of a lane.  VEC (E a multiple of the chunk, rows on 16 bytes): chunks of 16 bytes, a token's
// lanes side by side, so that every wide load of a token is contiguous (fp32, 16384 x 256 backward: 12.8 us with
// a lane's experts all in a row, 7.9 us so);
// else every LPT-th expert.
template <int DT, int EPL>
constexpr int kChunk = (DT == DT_F32 ? 4 : 8) < EPL ? (DT == DT_F32 ? 4 : 8) : EPL;
template <int DT, int LPT, int EPL, bool VEC>
__device__ __forceinline__ int expert_of(int i, int sub) {
    constexpr int C = kChunk<DT, EPL>;
    return VEC ? (i / C * LPT + sub) * C + i % C : i * LPT + sub;
}

// A lane's logits as they are stored (16 or 32 bits); -inf behind the last expert.
template <int DT, int LPT, int EPL, bool VEC>
__device__ __forceinline__ void load_row(const void *logits, int64_t at, int E, int sub, uint32_t (&raw)[EPL]) {
    constexpr uint32_t none = DT == DT_F32 ? 0xFF800000u : DT == DT_BF16 ? 0xFF80u : 0xFC00u;
    if constexpr (VEC) {
        constexpr int C = kChunk<DT, EPL>, size = DT == DT_F32 ? 4 : 2, W = C * size / 4;
        typedef uint32_t words __attribute__((__vector_size__(W * sizeof(uint32_t))));
#pragma unroll
        for (int v = 0; v < EPL / C; ++v) {
            const int e = expert_of<DT, LPT, EPL, VEC>(v * C, sub);
            words w;
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = DT == DT_F32 ? none : none | none << 16;
            if (e < E) w = *reinterpret_cast<const words *>(static_cast<const uint8_t *>(logits) + (at + e) * size);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if constexpr (DT == DT_F32) raw[v * C + i] = w[i];
                else raw[v * C + i] = (w[i / 2] >> (16 * (i % 2))) & 0xFFFFu;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * LPT + sub;
            if constexpr (DT == DT_F32) raw[i] = e < E ? static_cast<const uint32_t *>(logits)[at + e] : none;
            else raw[i] = e < E ? static_cast<const uint16_t *>(logits)[at + e] : none;
        }
    }
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t raw) {
    if constexpr (DT == DT_F32) return __uint_as_float(raw);
    else return h2f<DT>((uint16_t)raw);
}

// Logits in an order that unsigned integers compare by; -0 counts as +0, and keys up to kNoKey
// (-inf's, and 0 for an expert already chosen) are no choice.  16-bit types carry the expert
// along (a lower one is larger), so one maximum decides ties too.
template <int DT>
constexpr uint32_t kNoKey = DT == DT_F32 ? 0x007FFFFFu : DT == DT_BF16 ? 0x007FFFFFu : 0x03FFFFFFu;

template <int DT, int LPT, int EPL, bool VEC>
__device__ __forceinline__ void make_keys(uint32_t (&key)[EPL], int sub) {
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint32_t u = key[i] == 0x80000000u ? 0u : key[i];
            key[i] = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
        }
    } else {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        typedef short i16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < EPL; i += 2) {
            const uint32_t w = key[i] | key[i + 1] << 16;
            const uint32_t neg = __builtin_bit_cast(uint32_t, as<i16x2>(w) >> 15);          // all ones in negative halves
            const uint32_t o = w ^ (neg | 0x80008000u);
            // -0 came to 0x7FFF, +0 to 0x8000
            const u16x2 up = u16x2{1, 1} - __builtin_elementwise_min(as<u16x2>(o ^ 0x7FFF7FFFu), u16x2{1, 1});
            const uint32_t k = __builtin_bit_cast(uint32_t, as<u16x2>(o) + up);
            key[i] = k << 16 | (0xFFFFu - (uint32_t)expert_of<DT, LPT, EPL, VEC>(i, sub));
            key[i + 1] = (k & 0xFFFF0000u) | (0xFFFFu - (uint32_t)expert_of<DT, LPT, EPL, VEC>(i + 1, sub));
        }
    }
}
// Falling order of N keys in registers (odd-even merge sort, 63 exchanges of 16 keys).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + k];
                        key[i + j] = a > b ? a : b;
                        key[i + j + k] = a > b ? b : a;
                    }
                }
}

template <int DT>
__device__ __forceinline__ float key_value(uint32_t key) {
    if constexpr (DT == DT_F32) {
        return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    } else {
        const uint32_t o = key >> 16;
        return h2f<DT>((uint16_t)(o & 0x8000u ? o ^ 0x8000u : o ^ 0xFFFFu));
    }
}

// What a token's logits are good for: a distribution, nothing (every logit
// -inf), or NaN (a NaN or +inf among them).
enum { ROW_OK = 0, ROW_EMPTY = 1, ROW_NAN = 2 };

// exp(z - max) as exp2 of the difference times log2(e): the difference and the product round
// once each and log2(e) is off by a quarter of a half step, so the result is off by
// 2.25 |z - max| half steps and exp2's one step.  -inf gives 0, a NaN or +inf in the row NaN.  Results below 2^-126
// may be 0.
constexpr float kLog2e = 0x1.715476p+0f;
__device__ __forceinline__ float exp_from(float z, float top) { return __builtin_amdgcn_exp2f((z - top) * kLog2e); }

// The same for a chosen expert, whose weight is an output: what the difference, the product and log2(e) lost is
// added to the result, which is then off by exp2's one step and a rounding at any distance (uncorrected, by up to
// 120 half steps at fp32 logits up to 80 below the largest, 60 at 16-bit ones; the call takes 0.1 us more).
__device__ __forceinline__ float exp_chosen(float z, float top) {
    constexpr float kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float d = z - top, b = d - z, lost = (z - (d - b)) - (top + b);       // d + lost = z - top
    const float t = d * kLog2e;
    const float rest = __builtin_fmaf(d, kLog2e, -t) + __builtin_fmaf(d, kLog2eLow, lost * kLog2e);
    const float e = __builtin_amdgcn_exp2f(t);
    return e > 0.0f ? __builtin_fmaf(e * kLn2, rest, e) : 0.0f;                 // (d may be past fp32's range)
}

// A row's exponentials, one over their sum, and its kind.  The reciprocal of a row
// without a distribution is 0 or NaN (the exponentials of a row of nothing but -inf are set to 0).
template <int DT, int LPT, int EPL>
__device__ __forceinline__ int row_softmax(const uint32_t (&raw)[EPL], float (&p)[EPL], float &top, float &inv) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = value_of<DT>(raw[i]);
        m = fmaxf(m, p[i]);                       // a NaN does not count here
    }
    top = group_max<LPT>(m);
    if (top == -INFINITY) {                       // nothing but -inf, or NaN among it
        uint32_t nan = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            nan |= p[i] != p[i] ? 1u : 0u;
            p[i] = 0.0f;
        }
        const bool any = lane_umax<LPT>(nan) != 0;
        inv = any ? __builtin_nanf("") : 0.0f;
        return any ? ROW_NAN : ROW_EMPTY;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = exp_from(p[i], top);
        s += p[i];
    }
    s = group_sum<LPT>(s);
    inv = 1.0f / s;
    return s == s ? ROW_OK : ROW_NAN;
}

// ---- forward ------------------------------------------------------------------

constexpr int kRouteThreads = 256;         // without counts, and backward
constexpr int kCountThreads = 1024;        // with counts: few blocks, whose sums are read back

// loss = E x / (n tokens) from x = sum_e c_e P_e, n = sum_e c_e (0 without tokens)
__device__ __forceinline__ float balance_loss(int E, double x, int n, int tokens) {
    const double tv = tokens > 0 ? tokens : 1, cc = n > 0 ? n : 1;
    return (float)(E * x / (cc * tv));
}

// Workspace: the blocks' sums of probabilities [blocks][E] and counts [blocks][E + 1], and
// the joining blocks' sums and ticket.
struct RouteSpace {
    float *p;
    int32_t *c;
    double *x;
    int32_t *n;
    int32_t *tokens;
    uint32_t *ticket;
};
constexpr int kMaxBlocks = 256;            // of a counting call
constexpr int kJoinRows = 16, kMaxJoins = kMoeMaxExperts / 64 + 1;
static_assert(kMaxJoins <= 64, "one wave adds up the joining workgroups");

// Sums of v over the 64 / LPT token groups of a wave.  Within a row of 16 lanes by rotation; across
// rows by exchanging halves of two registers, which adds up both in one register: a lane is left with the
// first EPL / 4 (LPT 32: EPL / 2) sums from the index that is returned on.
template <int LPT, int EPL>
__device__ __forceinline__ int join_groups(float (&v)[EPL]) {
    if constexpr (LPT == 64) return 0;
    if constexpr (LPT <= 8) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            auto turn = [&](auto ctrl) {
                const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v[i]), decltype(ctrl)::value, 0xF, 0xF, true);
                v[i] += __int_as_float(o);
            };
            if constexpr (LPT == 4) turn(std::integral_constant<int, 0x124>{});       // row_ror:4
            turn(std::integral_constant<int, 0x128>{});                               // row_ror:8
        }
    }
    const int row = lane_id() >> 4;
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + EPL / 2]), false, false);
        v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    if constexpr (LPT == 32) return (row >> 1) * (EPL / 2);
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + EPL / 4]), false, false);
        v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    }
    return (row >> 1) * (EPL / 2) + (row & 1) * (EPL / 4);
}

// Counts are kept where COUNT; a single block finishes by itself.
template <int DT, int LPT, int EPL, bool VEC, bool COUNT>
__global__ void __launch_bounds__(COUNT ? kCountThreads : kRouteThreads) route_kernel(RouteArgs p, RouteSpace ws) {
    constexpr int NT = COUNT ? kCountThreads : kRouteThreads, NW = NT / 64, TPB = NT / LPT;
    __shared__ int cnt[COUNT ? LPT * EPL + 1 : 1];
    __shared__ float psum[COUNT ? NW : 1][COUNT ? LPT * EPL : 1];
    __shared__ float xs[NW];
    __shared__ int ns[NW];
    const int E = p.E, tid = threadIdx.x, sub = tid % LPT;
    float pacc[COUNT ? EPL : 1];
    if constexpr (COUNT) {
        for (int e = tid; e <= E; e += NT) cnt[e] = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) pacc[i] = 0.0f;
        if (blockIdx.x == 0 && tid == 0 && gridDim.x > 1) *ws.ticket = 0;
        __syncthreads();
    }
    for (int64_t t = (int64_t)blockIdx.x * TPB + tid / LPT; t < p.T; t += (int64_t)gridDim.x * TPB) {
        int32_t *ids = p.ids + t * p.topk;
        float *w = p.w + t * p.topk;
        const bool live = !p.mask || p.mask[t] != 0;
        uint32_t key[EPL];
        float pe[EPL], top = 0.0f, inv = 0.0f;
        int kind = ROW_EMPTY;
        if (live) {
            load_row<DT, LPT, EPL, VEC>(p.logits, t * p.ld, E, sub, key);
            kind = row_softmax<DT, LPT, EPL>(key, pe, top, inv);
            if constexpr (COUNT) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) pacc[i] = __builtin_fmaf(pe[i], inv, pacc[i]);
                if (sub == 0 && kind != ROW_EMPTY) atomicAdd(&cnt[E], 1);
            }
        }
        if (kind != ROW_OK) {
            const float fill = kind == ROW_NAN ? __builtin_nanf("") : 0.0f;
            for (int k = sub; k < p.topk; k += LPT) {
                ids[k] = -1;
                w[k] = fill;
            }
            continue;
        }
        make_keys<DT, LPT, EPL, VEC>(key, sub);
        // the largest that is left, topk times; lane k % LPT keeps choice k until LPT of them
        // are written together
        float chosen = 0.0f;
        uint32_t mine = 0;
        int my_id = -1;
        auto flush = [&](int k0, int n) {
            const float ex = my_id >= 0 ? exp_chosen(key_value<DT>(mine), top) : 0.0f;
            if (sub < n) {
                ids[k0 + sub] = my_id;
                w[k0 + sub] = ex;
                if constexpr (COUNT) {
                    if (my_id >= 0) atomicAdd(&cnt[my_id], 1);
                }
            }
            chosen += sub < n ? ex : 0.0f;
            return ex;
        };
        auto keep = [&](int k, uint32_t best, int be) {
            const bool here = sub == k % LPT;
            mine = here ? best : mine;
            my_id = here ? (best <= kNoKey<DT> ? -1 : be) : my_id;
            if (k % LPT == LPT - 1 && k + 1 < p.topk) flush(k - (LPT - 1), LPT);
        };
        if constexpr (DT == DT_F32) {
            for (int k = 0; k < p.topk; ++k) {
                uint32_t m = key[0];
#pragma unroll
                for (int i = 1; i < EPL; ++i) m = key[i] > m ? key[i] : m;
                const uint32_t best = lane_umax<LPT>(m);
                uint32_t at = 0;                                 // the lowest expert at the best value, as 0xFFFF - e
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const uint32_t v = 0xFFFFu - (uint32_t)expert_of<DT, LPT, EPL, VEC>(i, sub);
                    const uint32_t c = key[i] == best ? v : 0u;
                    at = c > at ? c : at;
                }
                const int be = 0xFFFF - (int)lane_umax<LPT>(at);
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = expert_of<DT, LPT, EPL, VEC>(i, sub) == be ? 0u : key[i];
                keep(k, best, be);
            }
        } else {
            // Unequal keys: each lane sorts its own once, a round compares the lanes' first ones and
            // its winner moves up.  Per wave 126 instructions and 25 a round, against 80 a round with a
            // maximum over all keys and a pass that takes the winner out (16384 tokens, 256 experts, 8 of
            // them: 15.4 -> 14.5 us with the counts).
            sort_keys(key);
            auto rounds = [&](auto depth) {
                constexpr int DEPTH = decltype(depth)::value;    // at most so many of a lane's keys are chosen
                for (int k = 0; k < p.topk; ++k) {
                    const uint32_t best = lane_umax<LPT>(key[0]);
                    const bool won = key[0] == best;
#pragma unroll
                    for (int i = 0; i + 1 < DEPTH; ++i) key[i] = won ? key[i + 1] : key[i];
                    key[DEPTH - 1] = won ? 0u : key[DEPTH - 1];
                    keep(k, best, 0xFFFF - (int)(best & 0xFFFFu));
                }
            };
            if (EPL > 8 && p.topk <= 8) rounds(std::integral_constant<int, 8 < EPL ? 8 : EPL>{});
            else rounds(std::integral_constant<int, EPL>{});
        }
        const int k0 = (p.topk - 1) / LPT * LPT;
        const float ex = flush(k0, p.topk - k0);
        const float scale = p.renorm ? 1.0f / group_sum<LPT>(chosen) : inv;
        if (k0 + sub < p.topk) w[k0 + sub] = ex * scale;
        for (int k = sub; k < k0; k += LPT) w[k] *= scale;               // each lane its own values
    }
    if constexpr (COUNT) {
        // sums over the token groups of a wave, then over the waves
        const int left = join_groups<LPT, EPL>(pacc);
        constexpr int KEPT = LPT <= 16 ? EPL / 4 : LPT == 32 ? EPL / 2 : EPL;
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            const int e = expert_of<DT, LPT, EPL, VEC>(i + left, sub);
            if ((tid & 15) < LPT && e < E) psum[tid >> 6][e] = pacc[i];
        }
        __syncthreads();
        float x = 0.0f;
        int n = 0;
        for (int e = tid; e <= E; e += NT) {
            const int c = cnt[e];
            float v = 0.0f;
            if (e < E) {
#pragma unroll
                for (int w = 0; w < NW; ++w) v += psum[w][e];
                x += (float)c * v;
                n += c;
            }
            if (gridDim.x == 1) {
                p.counts[e] = c;
            } else {
                ws.c[(int64_t)blockIdx.x * (E + 1) + e] = c;
                if (e < E) ws.p[(int64_t)blockIdx.x * E + e] = v;
            }
        }
        if (gridDim.x == 1 && p.loss) {
            x = group_sum<64>(x);
            n = lane_reduce<64>(n, [](int u, int v) { return u + v; });
            if (lane_id() == 0) {
                xs[tid >> 6] = x;
                ns[tid >> 6] = n;
            }
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < NW; ++w) {
                    x += xs[w];
                    n += ns[w];
                }
                *p.loss = balance_loss(E, x, n, cnt[E]);
            }
        }
    }
}

// Counts and loss from the blocks' sums, in a fixed order: a workgroup sums 64 experts
// (index E: the tokens), kJoinRows waves taking every kJoinRows-th block; the last one to finish adds up the
// workgroups' shares of the loss.
__global__ void __launch_bounds__(kJoinRows * 64)
route_join_kernel(RouteSpace ws, int blocks, int E, int32_t *__restrict__ counts, float *__restrict__ loss) {
    constexpr int BATCH = kMaxBlocks / kJoinRows;
    __shared__ float ps[kJoinRows][64];
    __shared__ int cs[kJoinRows][64];
    const int lane = lane_id(), row = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane, ec = e < E ? e : E;
    float pv[BATCH];
    int cv[BATCH];
    // all loads are on their way before the first is used
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
        const int64_t b = row + u * kJoinRows < blocks ? row + u * kJoinRows : blocks - 1;
        cv[u] = ws.c[b * (E + 1) + ec];
        pv[u] = ws.p[b * E + (e < E ? e : E - 1)];
    }
    float s = 0.0f;
    int c = 0;
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
        if (row + u * kJoinRows < blocks) {
            s += pv[u];
            c += cv[u];
        }
    ps[row][lane] = s;
    cs[row][lane] = c;
    __syncthreads();
    if (row != 0) return;
#pragma unroll
    for (int r = 1; r < kJoinRows; ++r) {
        s += ps[r][lane];
        c += cs[r][lane];
    }
    if (e <= E) counts[e] = c;
    if (!loss) return;
    double x = e < E ? (double)c * s : 0.0;
    const int n = lane_reduce<64>(e < E ? c : 0, [](int a, int b) { return a + b; });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    // expert index E, the tokens, is in the last workgroup
    int tokens = __builtin_amdgcn_readlane(c, E & 63);
    if (gridDim.x == 1) {
        if (lane == 0) *loss = balance_loss(E, x, n, tokens);
        return;
    }
    // One lane writes the workgroup's shares and takes a ticket, which releases them; whoever draws the last
    // one has acquired all (the caches' write-back included, the whole call takes 13.1 us for 16384 x 256, against 13.0
    // with stores past the caches and no order but the hardware's).
    unsigned order = 0;
    if (lane == 0) {
        ws.x[blockIdx.x] = x;
        ws.n[blockIdx.x] = n;
        if (blockIdx.x == gridDim.x - 1) *ws.tokens = tokens;
        order = __hip_atomic_fetch_add(ws.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(order) != gridDim.x - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");           // for the other lanes
    const bool in = lane < (int)gridDim.x;
    x = in ? ws.x[lane] : 0.0;
    const int part = in ? ws.n[lane] : 0;
    tokens = *ws.tokens;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    const int all = lane_reduce<64>(part, [](int a, int b) { return a + b; });
    if (lane == 0) *loss = balance_loss(E, x, all, tokens);
}

// ---- backward -----------------------------------------------------------------

// (Four waves per SIMD hold the 1024 workgroups of 16384 tokens of 256 experts at once.  All forms fit its 128 registers
// without spilling; left alone, one would take more: 142 for wide fp32 rows of 513 to 1024 experts.)
template <int DT, int LPT, int EPL, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, 4) route_backward_kernel(RouteArgs p) {
    constexpr int TPB = kRouteThreads / LPT;
    // a token's gradients through its chosen weights, one place per expert
    __shared__ __attribute__((aligned(16))) float spread[TPB][LPT * EPL];
    const int E = p.E, tid = threadIdx.x, sub = tid % LPT;
    __shared__ __attribute__((aligned(16))) float hs[LPT * EPL];
    float *const mine = spread[tid / LPT];
    // What the lanes of a wave wrote to LDS in front of it is there for all of them behind it.
    auto meet = []() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    // the first row is on its way while the loss's part of h is formed
    int64_t t = (int64_t)blockIdx.x * TPB + tid / LPT;
    uint32_t raw[EPL];
    if (t < p.T) load_row<DT, LPT, EPL, VEC>(p.logits, t * p.ld, E, sub, raw);
    // lane k of a token keeps entry k (of LPT at a time)
    int32_t id = -1;
    float w = 0.0f, dw = 0.0f;
    auto entries = [&](int64_t tok, int k0) {
        const int k = k0 + sub;
        const bool held = p.dw && tok < p.T && k < p.topk;
        id = held ? p.ids[tok * p.topk + k] : -1;
        w = held ? p.w[tok * p.topk + k] : 0.0f;
        dw = held ? p.dw[tok * p.topk + k] : 0.0f;
    };
    entries(t, 0);
    float h0[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) h0[i] = 0.0f;
    if (p.dloss) {
        int C = 0;                                           // sum of the counts: below 2^31
        constexpr int CL = (LPT * EPL + 63) / 64;
        int cv[CL];
#pragma unroll
        for (int i = 0; i < CL; ++i) {
            const int e = (tid & 63) + 64 * i;
            cv[i] = p.counts[e < E ? e : E];
        }
#pragma unroll
        for (int i = 0; i < CL; ++i) C += (tid & 63) + 64 * i < E ? cv[i] : 0;
        C = lane_reduce<64>(C, [](int u, int v) { return u + v; });
        const int tv = p.counts[E];
        const float f = C > 0 && tv > 0 ? *p.dloss / ((float)C * (float)tv) : 0.0f;
        for (int e = tid; e < LPT * EPL; e += kRouteThreads)
            hs[e] = e < E ? f * (float)__builtin_fma((double)E, (double)p.counts[e], -(double)C) : 0.0f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EPL; ++i) h0[i] = hs[expert_of<DT, LPT, EPL, VEC>(i, sub)];
    }
    for (; t < p.T; t += (int64_t)gridDim.x * TPB) {
        const bool live = !p.mask || p.mask[t] != 0;
        float pe[EPL], out[EPL], top = 0.0f, inv = 0.0f;
        int kind = ROW_EMPTY;
        if (live) kind = row_softmax<DT, LPT, EPL>(raw, pe, top, inv);
        if (t + (int64_t)gridDim.x * TPB < p.T)
            load_row<DT, LPT, EPL, VEC>(p.logits, (t + (int64_t)gridDim.x * TPB) * p.ld, E, sub, raw);
        if (kind != ROW_OK) {
            const float fill = kind == ROW_NAN ? __builtin_nanf("") : 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) out[i] = fill;
        } else {
            float sel[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) sel[i] = 0.0f;
            if (p.dw) {
                float mean = 0.0f;
                if (p.renorm) {
                    mean = id >= 0 ? w * dw : 0.0f;
                    for (int k = sub + LPT; k < p.topk; k += LPT)
                        mean += p.ids[t * p.topk + k] >= 0 ? p.w[t * p.topk + k] * p.dw[t * p.topk + k] : 0.0f;
                    mean = group_sum<LPT>(mean);
                }
                // Through LDS: entry k's value to its expert's place (the lanes of a token are in one wave,
                // whose steps meet() orders), unless an expert comes twice (the entry that it finds in its
                // place is another) or topk is past the lanes.
                const float v = p.renorm ? w * (dw - mean) : dw;
                const bool held = id >= 0 && id < E;
                bool twice = p.topk > LPT;
                if (!twice) {
#pragma unroll
                    for (int i = 0; i < EPL; i += 4) *reinterpret_cast<f32x4_t *>(mine + sub * EPL + i) = f32x4_t{};
                    meet();
                    float *const place = mine + (held ? id : 0);
                    if (held) *place = (float)sub;
                    meet();
                    const bool other_entry = held && *place != (float)sub;
                    twice = lane_umax<LPT>(other_entry ? 1u : 0u) != 0;
                    meet();
                    if (held) *place = v;
                    meet();
                    if constexpr (VEC) {
#pragma unroll
                        for (int i = 0; i < EPL; i += 4) {
                            const f32x4_t q = *reinterpret_cast<const f32x4_t *>(mine + expert_of<DT, LPT, EPL, VEC>(i, sub));
#pragma unroll
                            for (int u = 0; u < 4; ++u) sel[i + u] = q[u];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < EPL; ++i) sel[i] = mine[i * LPT + sub];
                    }
                    meet();
                }
                if (twice) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) sel[i] = 0.0f;
                    for (int k0 = 0; k0 < p.topk; k0 += LPT) {
                        if (k0 > 0) entries(t, k0);
                        const float kept = p.renorm ? w * (dw - mean) : dw;
                        const int most = p.topk - k0 < LPT ? p.topk - k0 : LPT;
                        for (int k = 0; k < most; ++k) {
                            const int kid = __shfl(id, k, LPT);
                            const float kv = __shfl(kept, k, LPT);
#pragma unroll
                            for (int i = 0; i < EPL; ++i)
                                sel[i] += kid == expert_of<DT, LPT, EPL, VEC>(i, sub) ? kv : 0.0f;
                        }
                    }
                }
            }
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                pe[i] *= inv;
                out[i] = h0[i] + (p.renorm ? 0.0f : sel[i]);
                dot += pe[i] * out[i];
            }
            dot = group_sum<LPT>(dot);
#pragma unroll
            for (int i = 0; i < EPL; ++i) out[i] = pe[i] * (out[i] - dot) + (p.renorm ? sel[i] : 0.0f);
        }
        entries(t + (int64_t)gridDim.x * TPB, 0);
        if constexpr (VEC) {
            constexpr int C = kChunk<DT, EPL>, size = DT == DT_F32 ? 4 : 2, W = C * size / 4;
            typedef uint32_t words __attribute__((__vector_size__(W * sizeof(uint32_t))));
#pragma unroll
            for (int v = 0; v < EPL / C; ++v) {
                const int e = expert_of<DT, LPT, EPL, VEC>(v * C, sub);
                words q;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if constexpr (DT == DT_F32) q[i] = __float_as_uint(out[v * C + i]);
                    else q[i] = f2h<DT>(out[v * C + 2 * i]) | (uint32_t)f2h<DT>(out[v * C + 2 * i + 1]) << 16;
                }
                if (e < E)
                    *reinterpret_cast<words *>(static_cast<uint8_t *>(p.dlogits) + (t * p.ldd + e) * size) = q;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * LPT + sub;
                if (e < E) store_logit<DT>(p.dlogits, t * p.ldd + e, out[i]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

// Lanes and experts per lane of a token.
struct RouteShape { int lpt, epl; };
static RouteShape route_shape(int64_t E) {
    if (E <= 16) return {4, 4};
    if (E <= 32) return {4, 8};
    if (E <= 64) return {8, 8};
    if (E <= 128) return {8, 16};
    if (E <= 256) return {16, 16};
    return E <= 512 ? RouteShape{32, 16} : RouteShape{64, 16};
}

// Blocks of a counting call: one while it has at most two rounds of tokens (a second
// launch costs as much as a round).
static int64_t route_blocks(int64_t T, int64_t E) {
    const int64_t tpb = kCountThreads / route_shape(E).lpt;
    if (T <= 2 * tpb) return 1;
    const int64_t b = (T + tpb - 1) / tpb;
    return b < kMaxBlocks ? b : kMaxBlocks;
}

static size_t route_space(int64_t blocks, int64_t E, void *workspace, RouteSpace *out) {
    if (blocks == 1) return 0;
    uint8_t *at = (uint8_t *)workspace;
    RouteSpace r;
    r.x = (double *)at;
    r.n = (int32_t *)(r.x + kMaxJoins);
    r.tokens = r.n + kMaxJoins;
    r.ticket = (uint32_t *)(r.tokens + 1);
    r.p = (float *)(r.ticket + 4);
    r.c = (int32_t *)(r.p + blocks * E);
    if (out) *out = r;
    return (size_t)((uint8_t *)(r.c + blocks * (E + 1)) - at);
}

size_t route_workspace_bytes(int64_t T, int64_t E) { return route_space(route_blocks(T, E), E, nullptr, nullptr); }

// Wide loads: rows of whole chunks on 16 bytes.
static bool route_vec(const void *p, int64_t ld, int E, int size) {
    const int chunk = 16 / size < route_shape(E).epl ? 16 / size : route_shape(E).epl;
    return E % chunk == 0 && ld * size % 16 == 0 && (uintptr_t)p % 16 == 0;
}

template <int DT, int LPT, int EPL>
static hipError_t route_launch(const RouteArgs &p, void *workspace, hipStream_t stream) {
    const bool vec = route_vec(p.logits, p.ld, p.E, DT == DT_F32 ? 4 : 2);
    if (!p.counts) {
        constexpr int TPB = kRouteThreads / LPT;
        const int64_t b = (p.T + TPB - 1) / TPB;
        auto kern = vec ? route_kernel<DT, LPT, EPL, true, false> : route_kernel<DT, LPT, EPL, false, false>;
        hipLaunchKernelGGL(kern, dim3((unsigned)(b < 4096 ? b : 4096)), dim3(kRouteThreads), 0, stream, p, RouteSpace{});
        return hipGetLastError();
    }
    const int64_t nb = route_blocks(p.T, p.E);
    RouteSpace ws{};
    route_space(nb, p.E, workspace, &ws);
    auto kern = vec ? route_kernel<DT, LPT, EPL, true, true> : route_kernel<DT, LPT, EPL, false, true>;
    hipLaunchKernelGGL(kern, dim3((unsigned)nb), dim3(kCountThreads), 0, stream, p, ws);
    if (nb > 1)
        hipLaunchKernelGGL(route_join_kernel, dim3((unsigned)(p.E / 64 + 1)), dim3(kJoinRows * 64), 0, stream,
                           ws, (int)nb, p.E, p.counts, p.loss);
    return hipGetLastError();
}

template <int DT, int LPT, int EPL>
static hipError_t route_backward_launch(const RouteArgs &p, hipStream_t stream) {
    constexpr int TPB = kRouteThreads / LPT, size = DT == DT_F32 ? 4 : 2;
    const bool vec = route_vec(p.logits, p.ld, p.E, size) && route_vec(p.dlogits, p.ldd, p.E, size);
    const int64_t b = (p.T + TPB - 1) / TPB;
    auto kern = vec ? route_backward_kernel<DT, LPT, EPL, true> : route_backward_kernel<DT, LPT, EPL, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(b < 2048 ? b : 2048)), dim3(kRouteThreads), 0, stream, p);
    return hipGetLastError();
}

template <int DT, bool BACKWARD>
static hipError_t route_dispatch(const RouteArgs &p, void *workspace, hipStream_t stream) {
    const RouteShape s = route_shape(p.E);
#define W4_ROUTE(L, P)                                                                                 \
    if (s.lpt == L && s.epl == P)                                                                      \
        return BACKWARD ? route_backward_launch<DT, L, P>(p, stream) : route_launch<DT, L, P>(p, workspace, stream);
    W4_ROUTE(4, 4) W4_ROUTE(4, 8) W4_ROUTE(8, 8) W4_ROUTE(8, 16) W4_ROUTE(16, 16) W4_ROUTE(32, 16) W4_ROUTE(64, 16)
#undef W4_ROUTE
    return hipErrorInvalidValue;
}

hipError_t launch_route(const RouteArgs &p, int dt, void *workspace, hipStream_t stream) {
    if (dt == DT_F32) return route_dispatch<DT_F32, false>(p, workspace, stream);
    return dt == DT_BF16 ? route_dispatch<DT_BF16, false>(p, workspace, stream)
                         : route_dispatch<DT_F16, false>(p, workspace, stream);
}

hipError_t launch_route_backward(const RouteArgs &p, int dt, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    if (dt == DT_F32) return route_dispatch<DT_F32, true>(p, nullptr, stream);
    return dt == DT_BF16 ? route_dispatch<DT_BF16, true>(p, nullptr, stream)
                         : route_dispatch<DT_F16, true>(p, nullptr, stream);
}

}  // namespace w4
