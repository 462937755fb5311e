// prefix_attn.hip -- attention of one new token a row where rows share a long prefix
// (ssm_prefix_attn_decode_fwd in include/ssm_longctx.h).
//
// Three steps: attention over each row's own tokens (paged_attn.hip, its output in fp32), attention of
// all rows over the prefixes (prefix_attn_kernel), and the join of both by their maxima and sums.
//
// The prefix kernel has up to 64 (row, query head) pairs of a kv head in a block, as 16 NQ columns of the matrix
// products, so a prefix's K and V are read from HBM once and by a block once for 64 columns; its 4 waves
// walk tiles of tokens of their own and join at the end.  Operands go from global memory straight
// into the matrix instructions' registers as in paged_attn_kernel.hpp (scores S^T = K Q^T, output O^T = V^T P^T,
// V transposed by byte permutations, here once for all columns); q waits in shared memory.
// A block's share is (16 NQ columns, kv head, one of `splits` parts of the prefix).  Blocks of the same part and
// other columns run on one XCD at one time, so that all but the first of them find K and V in its L2.
// Bound: for few columns HBM; from about 100 columns a kv head on the matrix cores and the exponentials beside them.
//
// The running maximum is raised only where a score exceeds it by more than 2^8 in its weight: weights up
// to 2^8 lose nothing in fp32, and the outputs are not rescaled for every new maximum.  Weights enter their
// product with v as two bf16 values (an error below 2^-17 of each; one alone would be 2^-9, and a third
// would cost half as much again on the matrix cores for what the output's rounding to bf16 hides).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_device.hpp"
#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

constexpr int kW = 4, kNT = kW * 64;
constexpr int kCUs = 256;
constexpr float kSlack = 8.0f;      // log2 of what a weight may exceed 1 by

struct Pp {
    const char *q; const char *k; const char *v; const int32_t *prefix; const int32_t *table; const int32_t *lens;
    float *part;                    // unnormalised outputs (split, row, head, d)
    float *ml;                      // and their maxima and sums (split, row, head, 2)
    const float *o_own; const float *lse_own; char *o; float *lse;
    int64_t table_stride, q_sr, q_sh, c_sh, c_sp, c_st;       // q and cache strides in bytes
    int batch, n_heads, n_kv, group, gm, passes, rows, tiles; // gm query heads and `rows` rows make a block's columns
    int d, n_prefixes, n_pages, page_size, max_len, splits, combos;
    float scale2, v_scale;
};

template <int CT, int DP> struct PTile {
    static constexpr int E = CT == KF32 ? 4 : CT == KBF16 ? 2 : 1;
    static constexpr int NT = CT == KF32 ? 16 : 32;            // tokens
    static constexpr int SUB = NT / 16;
    static constexpr int KD = 16 / E, KC = DP / (4 * KD);      // dims of a load of K, loads of a row (four lanes each)
    static constexpr int VD = CT == KF32 || DP % 128 ? 4 : 8;  // dims of a lane's load of V
    static constexpr int VB = DP / (16 * VD);                  // loads of a V row (16 lanes each)
    static constexpr int VW = VD * E / 4;                      // dwords of one
    static constexpr int VR = NT / 4;                          // V rows of a lane
    static constexpr int QW = CT == KF8 ? 2 : 1;               // operands of q to a load of K
    static constexpr int UNIT = kW * NT;
};
// columns of 16 that a block can take by the registers of their outputs
constexpr int most_nq(int dp) { return dp <= 128 ? 4 : 2; }

template <int CT, int DP, bool EXACT, int NQ>
__global__ void __launch_bounds__(kNT, 1) prefix_attn_kernel(Pp a) {
    using T = PTile<CT, DP>;
    constexpr int VD = T::VD, VB = T::VB, PITCH = DP + 4;
    extern __shared__ float lds[];          // q, and at the end the waves' outputs, 16 columns at a time
    u32x4 *q_lds = (u32x4 *)lds;
    __shared__ float wave_m[kW][16 * NQ], wave_l[kW][16 * NQ];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    const int j = blockIdx.x >> 3, combo = j / a.tiles * 8 + (blockIdx.x & 7), tile = j % a.tiles;
    if (combo >= a.combos) return;
    const int split = combo % a.splits, kp = combo / a.splits, pass = kp % a.passes, kv = kp / a.passes;
    const int row0 = tile * a.rows, nrows = min(a.rows, a.batch - row0);
    const int nh = min(a.gm, a.group - pass * a.gm), h0 = kv * a.group + pass * a.gm;
    const PageSize ps(a.page_size);

    // this lane's columns: their row in the block (-1: none) and head
    int crow[NQ], chead[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int c = n * 16 + col, r = c / a.gm;
        chead[n] = c - r * a.gm;
        crow[n] = r < nrows && chead[n] < nh ? r : -1;
    }
    // q (with the sign of the scale), as the scores' second operand
    const uint32_t flip = a.scale2 < 0.0f ? (CT == KF32 ? 0x80000000u : 0x80008000u) : 0u;
    const float scale2 = fabsf(a.scale2);
#pragma unroll
    for (int i = 0; i < T::KC * T::QW; ++i) {
        if (i % kW != wave) continue;
        const int dim = i / T::QW * 4 * T::KD + grp * T::KD + i % T::QW * 8;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            u32x4 x = {0, 0, 0, 0};
            if (crow[n] >= 0 && (EXACT || dim < a.d))
                x = *(const u32x4 *)(a.q + (row0 + crow[n]) * a.q_sr + (h0 + chead[n]) * a.q_sh + dim * (CT == KF32 ? 4 : 2));
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] ^= flip;
            q_lds[(i * NQ + n) * 64 + lane] = x;
        }
    }
    const int id = lane < nrows ? a.prefix[row0 + lane] : -1;
    uint64_t left = __ballot((uint32_t)id < (uint32_t)a.n_prefixes);
    __syncthreads();

    float m[NQ], l[NQ];                      // of the columns; l over this lane's tokens only
    f32x4 acc[NQ][VB][VD];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.0f;
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < VD; ++i) acc[n][b][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    const char *kb = a.k + kv * a.c_sh + grp * 16, *vb = a.v + kv * a.c_sh;

    // one prefix after the other, with the columns of its rows
    while (left) {
        const int p = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(id == p);
        left &= ~mine;
        const int len = min(max(a.lens[p], 0), a.max_len), units = (len + T::UNIT - 1) / T::UNIT;
        const int u0 = (int)((int64_t)split * units / a.splits), u1 = (int)((int64_t)(split + 1) * units / a.splits);
        const int t_end = min(len, u1 * T::UNIT);
        const int32_t *table = a.table + (int64_t)p * a.table_stride;
        bool in[NQ], all_in = true;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            in[n] = crow[n] >= 0 && (mine >> crow[n] & 1);
            all_in = all_in && (in[n] || crow[n] < 0);
        }
        all_in = __all(all_in);

        // a lane's token of a tile: its page (-1: none); tokens that are none read the cache's first row
        auto page_of = [&](int t0) {
            const int t = t0 + (lane & (T::NT - 1));
            return t < t_end ? table[ps.of(t)] : -1;
        };
        auto off_of = [&](int t0, int page) -> uint64_t {
            const int t = t0 + (lane & (T::NT - 1));
            return (uint32_t)page < (uint32_t)a.n_pages ? (uint64_t)page * (uint64_t)a.c_sp + (uint64_t)ps.place(t, ps.of(t)) * (uint64_t)a.c_st : 0;
        };
        auto row_of = [&](uint64_t off, int tok) {
            const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, tok), hi = (uint32_t)__shfl((int)(off >> 32), tok);
            return (uint64_t)hi << 32 | lo;
        };
        constexpr uint64_t ALL = (uint64_t(1) << T::NT) - 1;
        u32x4 kf[T::SUB][T::KC];
        auto load_k = [&](uint64_t off) {
#pragma unroll
            for (int s = 0; s < T::SUB; ++s) {
                const char *r = kb + row_of(off, 16 * s + col);
#pragma unroll
                for (int c = 0; c < T::KC; ++c) {
                    const bool is = EXACT || (c * 4 + grp) * T::KD < a.d;
                    const u32x4 x = *(const u32x4 *)(r + (is ? c * 64 : -grp * 16));
                    kf[s][c] = is ? x : (u32x4){0, 0, 0, 0};
                }
            }
        };
        int t0 = u0 * T::UNIT + wave * T::NT;
        if (t0 >= t_end) continue;
        int page = page_of(t0);
        uint64_t ok = __ballot((uint32_t)page < (uint32_t)a.n_pages) & ALL;
        uint64_t off = off_of(t0, page);
        load_k(off);
        page = page_of(t0 + T::UNIT);

        for (; t0 < t_end; t0 += T::UNIT) {
            const bool full = ok == ALL;
            Words<T::VW> vf[T::VR][VB];
#pragma unroll
            for (int x = 0; x < T::VR; ++x) {
                const char *r = vb + row_of(off, (x >> 2) * 16 + grp * 4 + (x & 3));
#pragma unroll
                for (int b = 0; b < VB; ++b) {       // past headdim: the row's first dims, in rows of the result that are not kept
                    const int dim = (b * 16 + col) * VD;
                    vf[x][b] = ld_words<T::VW>(r + (EXACT || dim < a.d ? dim * T::E : 0));
                }
            }
            f32x4 s[NQ][T::SUB];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < T::SUB; ++i) s[n][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < T::KC; ++c) {
                u32x4 q[T::QW][NQ];
#pragma unroll
                for (int w = 0; w < T::QW; ++w)
#pragma unroll
                    for (int n = 0; n < NQ; ++n) q[w][n] = q_lds[((c * T::QW + w) * NQ + n) * 64 + lane];
#pragma unroll
                for (int i = 0; i < T::SUB; ++i) {
                    const u32x4 k = kf[i][c];
                    if constexpr (CT == KBF16) {
#pragma unroll
                        for (int n = 0; n < NQ; ++n) s[n][i] = mfma_bf16(k, q[0][n], s[n][i]);
                    } else if constexpr (CT == KF8) {
                        const u32x4 k0 = {widen<false>(k[0]), widen<true>(k[0]), widen<false>(k[1]), widen<true>(k[1])};
                        const u32x4 k1 = {widen<false>(k[2]), widen<true>(k[2]), widen<false>(k[3]), widen<true>(k[3])};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            s[n][i] = mfma_bf16(k0, q[0][n], s[n][i]);
                            s[n][i] = mfma_bf16(k1, q[T::QW - 1][n], s[n][i]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                s[n][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(q[0][n][e]), s[n][i], 0, 0, 0);
                    }
                }
            }
            // the next tile's K
            const uint64_t ok_now = ok;
            ok = __ballot((uint32_t)page < (uint32_t)a.n_pages) & ALL;
            off = off_of(t0 + T::UNIT, page);
            if (t0 + T::UNIT < t_end) load_k(off);
            page = page_of(t0 + 2 * T::UNIT);

            float x[NQ][T::VR];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < T::VR; ++i) x[n][i] = s[n][i >> 2][i & 3] * scale2;
            if (!full) {                     // no weight, and not 0 * what stands in a row that is not the prefix's
                const uint32_t bits = (uint32_t)(ok_now >> (grp * 4));
#pragma unroll
                for (int i = 0; i < T::VR; ++i) {
                    const bool is = bits >> ((i >> 2) * 16 + (i & 3)) & 1;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) x[n][i] = is ? x[n][i] : -INFINITY;
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int w = 0; w < T::VW; ++w) vf[i][b].w[w] = is ? vf[i][b].w[w] : 0u;
                }
            }
            if (!all_in) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < T::VR; ++i) x[n][i] = in[n] ? x[n][i] : -INFINITY;
            }
            bool higher = false;
            float top[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                top[n] = x[n][0];
#pragma unroll
                for (int i = 1; i < T::VR; ++i) top[n] = fmaxf(top[n], x[n][i]);
                higher = higher || top[n] > m[n] + kSlack;
            }
            if (__any(higher)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float m_new = fmaxf(m[n], head_max(top[n]));
                    const float f = m_new == -INFINITY ? 1.0f : exp2_fast(m[n] - m_new);
                    m[n] = m_new;
                    l[n] *= f;
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int i = 0; i < VD; ++i) acc[n][b][i] *= f;
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const float m_use = m[n] == -INFINITY ? 0.0f : m[n];         // no token yet: all p are 0
#pragma unroll
                for (int i = 0; i < T::VR; ++i) {
                    x[n][i] = exp2_fast(x[n][i] - m_use);
                    l[n] += x[n][i];
                }
            }
            if constexpr (CT == KF32) {
#pragma unroll
                for (int i = 0; i < T::VR; ++i)
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                acc[n][b][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[i][b].w[e]), x[n][i], acc[n][b][e], 0, 0, 0);
            } else {
                u32x4 ph[NQ], pl[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ph[n][i] = pack_bf16(x[n][2 * i], x[n][2 * i + 1]);
                        pl[n][i] = pack_bf16(x[n][2 * i] - lo_f(ph[n][i]), x[n][2 * i + 1] - hi_f(ph[n][i]));
                    }
#pragma unroll
                for (int b = 0; b < VB; ++b) {
                    if constexpr (CT == KBF16) {
#pragma unroll
                        for (int i = 0; i < VD; ++i) {
                            u32x4 vt;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                vt[e] = perm(vf[2 * e + 1][b].w[i / 2], vf[2 * e][b].w[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(vt, ph[n], acc[n][b][i]);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(vt, pl[n], acc[n][b][i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VD; i += 2) {
                            u32x4 v0, v1;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t w = perm(vf[2 * e + 1][b].w[i / 4], vf[2 * e][b].w[i / 4], i & 2 ? 0x07030602u : 0x05010400u);
                                v0[e] = widen<false>(w);
                                v1[e] = widen<true>(w);
                            }
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                acc[n][b][i] = mfma_bf16(v0, ph[n], acc[n][b][i]);
                                acc[n][b][i + 1] = mfma_bf16(v1, ph[n], acc[n][b][i + 1]);
                            }
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                acc[n][b][i] = mfma_bf16(v0, pl[n], acc[n][b][i]);
                                acc[n][b][i + 1] = mfma_bf16(v1, pl[n], acc[n][b][i + 1]);
                            }
                        }
                    }
                }
            }
        }
    }

    // ---- join the block's waves, 16 columns at a time
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        l[n] = head_sum(l[n]);
        if (grp == 0) { wave_m[wave][n * 16 + col] = m[n]; wave_l[wave][n * 16 + col] = l[n]; }
    }
    const int d4 = a.d / 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        __syncthreads();                     // readers of q, or of the 16 columns before
        float top = wave_m[0][n * 16 + col];
#pragma unroll
        for (int w = 1; w < kW; ++w) top = fmaxf(top, wave_m[w][n * 16 + col]);
        const float f = top == -INFINITY ? 0.0f : exp2_fast(m[n] - top);
        float *to = lds + (wave * 16 + col) * PITCH;
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < VD; i += 4)
                    *(float4 *)(to + (b * 16 + grp * 4 + r) * VD + i) =
                        make_float4(acc[n][b][i][r] * f, acc[n][b][i + 1][r] * f, acc[n][b][i + 2][r] * f, acc[n][b][i + 3][r] * f);
        __syncthreads();
        for (int i = tid; i < 16 * d4; i += kNT) {
            const int cc = i / d4, e = (i - cc * d4) * 4, c = n * 16 + cc, r = c / a.gm, h = c - r * a.gm;
            if (r >= nrows || h >= nh) continue;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            float ls = 0.0f, mt = -INFINITY;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                v += *(const f32x4 *)(lds + (w * 16 + cc) * PITCH + e);
                mt = fmaxf(mt, wave_m[w][c]);
            }
#pragma unroll
            for (int w = 0; w < kW; ++w) ls += wave_l[w][c] * (mt == -INFINITY ? 1.0f : exp2_fast(wave_m[w][c] - mt));
            const int64_t at = ((int64_t)split * a.batch + row0 + r) * a.n_heads + h0 + h;
            *(f32x4 *)(a.part + at * a.d + e) = v;
            if (e == 0) *(float2 *)(a.ml + at * 2) = make_float2(mt, ls);
        }
    }
}

// Joins the parts of a (row, query head), a wave each, lanes of 4 dims; the row's own tokens are one
// more part, already normalised.
template <bool BF16>
__global__ void __launch_bounds__(kNT) prefix_join_kernel(Pp a) {
    const int lane = threadIdx.x & 63;
    const int64_t rh = (int64_t)blockIdx.x * kW + (threadIdx.x >> 6), all = (int64_t)a.batch * a.n_heads;
    if (rh >= all) return;
    const int e = lane * 4;
    const bool has = e < a.d;
    const float own = a.lse_own[rh] * kLog2e;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (has) o = *(const f32x4 *)(a.o_own + rh * a.d + e);
    float m = own;
    for (int s = lane; s < a.splits; s += 64) m = fmaxf(m, a.ml[(s * all + rh) * 2]);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float m_use = m == -INFINITY ? 0.0f : m;
    float sum = exp2_fast(own - m_use);
    o *= sum;
    for (int s = 0; s < a.splits; ++s) {
        const float2 w = *(const float2 *)(a.ml + (s * all + rh) * 2);
        const float f = exp2_fast(w.x - m_use);
        sum += w.y == 0.0f ? 0.0f : w.y * f;
        if (has && f > 0.0f && w.y != 0.0f) o += *(const f32x4 *)(a.part + (s * all + rh) * a.d + e) * (f * a.v_scale);
    }
    const float n = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    if (has) {
        if constexpr (BF16) *(uint2 *)(a.o + (rh * a.d + e) * 2) = make_uint2(pack_bf16(o[0] * n, o[1] * n), pack_bf16(o[2] * n, o[3] * n));
        else *(f32x4 *)(a.o + (rh * a.d + e) * 4) = o * n;
    }
    if (lane == 0 && a.lse) a.lse[rh] = m_use * kLn2 + logf(sum);
}

// ------------------------------------------------------------------ host ----
int64_t align16(int64_t n) { return (n + 15) & ~int64_t(15); }

// How the columns of all rows are cut into blocks
struct Cut { int nq, gm, passes, rows, tiles, splits; };
Cut cut_of(int64_t batch, int64_t n_heads, int64_t n_kv, int64_t d, int64_t max_len) {
    Cut c;
    const int64_t group = n_heads / n_kv, cols = batch * group;
    c.nq = (int)std::min<int64_t>(d <= 128 ? 4 : 2, cols > 32 ? 4 : cols > 16 ? 2 : 1);
    c.gm = (int)std::min<int64_t>(group, 16 * c.nq);
    c.passes = (int)((group + c.gm - 1) / c.gm);
    c.rows = (int)std::min<int64_t>(batch, 16 * c.nq / c.gm);
    c.tiles = (int)((batch + c.rows - 1) / c.rows);
    // one block a compute unit, of at least a unit of 64 tokens
    const int64_t heads = c.tiles * n_kv * c.passes, units = std::max<int64_t>(1, max_len / 128);
    c.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(kCUs / heads, units), 64));
    return c;
}

template <int CT, int DP, bool EXACT, int NQ>
hipError_t go_q(const Pp &k, hipStream_t stream) {
    using T = PTile<CT, DP>;
    const size_t lds = std::max((size_t)kW * 16 * (DP + 4) * sizeof(float), (size_t)T::KC * T::QW * NQ * 1024);
    if (lds > 32 * 1024) {               // more than a block has unasked, from 64 KiB on
        const hipError_t e = hipFuncSetAttribute((const void *)prefix_attn_kernel<CT, DP, EXACT, NQ>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const unsigned grid = (unsigned)((k.combos + 7) / 8 * 8 * k.tiles);
    hipLaunchKernelGGL((prefix_attn_kernel<CT, DP, EXACT, NQ>), dim3(grid), dim3(kNT), lds, stream, k);
    return hipGetLastError();
}
template <int CT, int DP, bool EXACT>
hipError_t go(const Pp &k, int nq, hipStream_t stream) {
    if constexpr (DP <= 128) {
        if (nq == 4) return go_q<CT, DP, EXACT, 4>(k, stream);
    }
    return nq == 2 ? go_q<CT, DP, EXACT, 2>(k, stream) : go_q<CT, DP, EXACT, 1>(k, stream);
}
template <int CT, int DP>
hipError_t go_d(const Pp &k, int nq, hipStream_t stream) {
    return k.d == DP ? go<CT, DP, true>(k, nq, stream) : go<CT, DP, false>(k, nq, stream);
}
template <int CT>
hipError_t go_type(const Pp &k, int nq, hipStream_t stream) {
    if (k.d <= 64) return go_d<CT, 64>(k, nq, stream);
    if (k.d <= 128) return go_d<CT, 128>(k, nq, stream);
    if (k.d <= 192) return go_d<CT, 192>(k, nq, stream);
    return go_d<CT, 256>(k, nq, stream);
}

}  // namespace

size_t prefix_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                   int64_t max_prefix_pages, int64_t max_pages, int64_t page_size) {
    const Cut c = cut_of(batch, n_heads, n_kv_heads, headdim, max_prefix_pages * page_size);
    const int64_t rh = batch * n_heads;
    return align16(paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, max_pages, page_size)) +
           align16(rh * headdim * 4) + align16(rh * 4) + align16(c.splits * rh * 8) + c.splits * rh * headdim * 4;
}

hipError_t launch_prefix_attn(const PrefixAttnArgs &p, hipStream_t stream, const char **kernel_name) {
    PagedAttnArgs a = p.own;
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    const int64_t rh = a.batch * a.n_heads;
    const Cut c = cut_of(a.batch, a.n_heads, a.n_kv_heads, a.headdim, p.max_prefix_pages * a.page_size);
    char *ws = (char *)a.workspace + align16(paged_attn_workspace_bytes(a.batch, a.n_heads, a.n_kv_heads, a.headdim, a.max_pages, a.page_size));
    Pp k = {};
    k.o_own = (const float *)ws; ws += align16(rh * a.headdim * 4);
    k.lse_own = (const float *)ws; ws += align16(rh * 4);
    k.ml = (float *)ws; ws += align16(c.splits * rh * 8);
    k.part = (float *)ws;
    k.q = (const char *)a.q; k.k = (const char *)a.k_cache; k.v = (const char *)a.v_cache;
    k.prefix = p.prefix; k.table = p.prefix_table; k.lens = p.prefix_lens; k.o = (char *)a.o; k.lse = a.lse;
    k.table_stride = p.prefix_stride; k.q_sr = a.q_sr * qe; k.q_sh = a.q_sh * qe;
    k.c_sp = a.c_sp * e; k.c_st = a.c_st * e; k.c_sh = a.c_sh * e;
    k.batch = (int)a.batch; k.n_heads = (int)a.n_heads; k.n_kv = (int)a.n_kv_heads; k.group = (int)(a.n_heads / a.n_kv_heads);
    k.gm = c.gm; k.passes = c.passes; k.rows = c.rows; k.tiles = c.tiles; k.splits = c.splits;
    k.combos = (int)(a.n_kv_heads * c.passes * c.splits);
    k.d = a.headdim; k.n_prefixes = (int)p.n_prefixes; k.n_pages = (int)a.n_pages; k.page_size = (int)a.page_size;
    k.max_len = (int)(p.max_prefix_pages * a.page_size);
    k.scale2 = a.scale * (a.kv_dtype == SSM_KV_F8E4M3 ? a.k_scale : 1.0f) * kLog2e;
    k.v_scale = a.kv_dtype == SSM_KV_F8E4M3 ? a.v_scale : 1.0f;

    a.o = (void *)k.o_own; a.lse = (float *)k.lse_own; a.o_f32 = true;
    hipError_t rc = launch_paged_attn(a, stream, kernel_name);
    if (rc != hipSuccess) return rc;
    *kernel_name = "prefix_attn_kernel";
    rc = a.kv_dtype == SSM_KV_F32 ? go_type<KF32>(k, c.nq, stream)
       : a.kv_dtype == SSM_KV_BF16 ? go_type<KBF16>(k, c.nq, stream) : go_type<KF8>(k, c.nq, stream);
    if (rc != hipSuccess) return rc;
    *kernel_name = "prefix_join_kernel";
    const dim3 grid((unsigned)((rh + kW - 1) / kW));
    if (a.kv_dtype != SSM_KV_F32) hipLaunchKernelGGL((prefix_join_kernel<true>), grid, dim3(kNT), 0, stream, k);
    else hipLaunchKernelGGL((prefix_join_kernel<false>), grid, dim3(kNT), 0, stream, k);
    return hipGetLastError();
}

}  // namespace ssm
