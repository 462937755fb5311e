// prefix_attn.hip -- attention of one new token a row where rows share a long prefix
// (ssm_prefix_attn_decode_fwd in include/ssm_longctx.h).
//
// One launch has the blocks of the prefixes and, behind them, those of the rows' own tokens (paged_attn_kernel.hpp's
// work, its output in fp32 and unnormalised); another joins both by their maxima and sums, o = sum_i o_i 2^(m_i - m) / l.
// Own tokens of a length that is cut into pieces are joined by a launch of their own before it.
//
// The (row, query head) pairs of a kv head are columns of the matrix products: scores S^T = K Q^T, output O^T = V^T P^T.
// A block has the columns of some rows and one of `splits` parts of their prefixes, end to end, so a prefix is read from
// HBM once and by a block once for all its columns.  Blocks of the same part and other columns run on one XCD at one
// time, so that all but the first of them find K and V in its L2.  Two forms:
//   few: up to 32 columns; the 4 waves walk tiles of tokens of their own, K and V straight from global memory into the
//     matrix instructions' registers (V transposed by byte permutations), and join at the end.
//   many: 4 waves of 16 or 32 columns each; K and V come through shared memory once for all, the next tile's while
//     one is worked on.
//
// A row's columns are done where its prefix ends: their part is written there and all columns start anew, so that a V
// that is not finite reaches the rows behind its own prefix alone (weights of 0 for the others would not do: 0 times it is
// NaN).  In the form for few, q then comes to shared memory again, where the outputs were.
//
// Figures (us): 64 rows of 32 + 8 heads of 128, bf16, behind 16384 tokens, 512 own, 74 a call; in a trace of the kernels, 70
// for both kinds of blocks and 9 for the join.  Its 134 MB would take 26; the prefix' part is bound by matrix and vector
// instructions (21 and 25 us of issue at the 1.7 GHz that both together leave) that two waves on a SIMD overlap in
// part.  13 rows of 20 + 4 heads, 8 bits, behind three prompts of 4001 17.4, and 2 rows behind 8192 tokens 15.3: the way
// through a block (its prefixes, pages, first loads; then the parts) and the second launch.
//
// The running maximum is raised only where a score exceeds it by more than 2^8 in its weight: weights up
// to 2^8 lose nothing in fp32, and the outputs are not rescaled for every new maximum.  Weights enter their
// product with a bf16 or 8-bit v as the sum of three bf16 values, all of their 24 bits.  (Two keep 17, and outputs in which
// the tokens' shares cancel show it: us with two and with three, 64 rows behind 16384 tokens, bf16 72.1, 79.2, 8 bits
// 57.4, 62.5; 128 rows behind five prompts 49.4, 57.0; 13 rows of three prompts in 8 bits 17.2, 17.7.  The figures beside
// the choices below were taken with two.)
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "paged_attn_kernel.hpp"

namespace ssm {
namespace {

constexpr int kW = 4;               // waves of a block (of kNT threads)
constexpr float kSlack = 8.0f;      // log2 of what a weight may exceed 1 by

struct Pp {
    const char *q; const char *k; const char *v; const int32_t *prefix; const int32_t *table; const int32_t *lens;
    float *part;                    // unnormalised outputs (split, row, head, d)
    float *ml;                      // and their maxima and sums (split, row, head, 2)
    const float *o_own;             // and those of the rows' own tokens (row, head, d), (row, head, 2)
    const float *ml_own;
    char *o; float *lse;
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

// A block's place in the work: 16-column groups are (row, head) pairs of one kv head
struct Place { int split, tile, kv, row0, nrows, nh, h0; };
__device__ __forceinline__ bool place_of(const Pp &a, int block, Place &p) {
    const int j = block >> 3, combo = j / a.tiles * 8 + (block & 7);
    if (combo >= a.combos) return false;
    p.tile = j % a.tiles;
    p.split = combo % a.splits;
    const int kp = combo / a.splits, pass = kp % a.passes;
    p.kv = kp / a.passes;
    p.row0 = p.tile * a.rows;
    p.nrows = min(a.rows, a.batch - p.row0);
    p.nh = min(a.gm, a.group - pass * a.gm);
    p.h0 = p.kv * a.group + pass * a.gm;
    return true;
}

// The prefixes of a block's rows, each at its first row's lane, in one line of units of `unit` tokens; the block's
// part of it.
struct Line { int id, len, units, upto, first, last; uint64_t leaders; };
__device__ __forceinline__ Line line_of(const Pp &a, const Place &p, int lane, int unit) {
    Line n;
    n.id = lane < p.nrows ? a.prefix[p.row0 + lane] : -1;
    if ((uint32_t)n.id >= (uint32_t)a.n_prefixes) n.id = -1;
    n.len = n.id >= 0 ? min(max(a.lens[n.id], 0), a.max_len) : 0;
    n.leaders = 0;
    for (uint64_t left = __ballot(n.id >= 0); left;) {
        const int l = __builtin_ctzll(left);
        n.leaders |= uint64_t(1) << l;
        left &= ~__ballot(n.id == __builtin_amdgcn_readlane(n.id, l));
    }
    n.units = n.leaders >> lane & 1 ? (n.len + unit - 1) / unit : 0;
    n.upto = wave_scan(n.units);
    const int all = __builtin_amdgcn_readlane(n.upto, 63);
    n.first = (int)((int64_t)p.split * all / a.splits);
    n.last = (int)((int64_t)(p.split + 1) * all / a.splits);
    return n;
}

// A lane's number out of the compiler's sight: what is formed from it behind the loop over tokens is formed there, and takes
// no registers of the loop.
__device__ __forceinline__ int formed_here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

template <int CT, int DP, bool EXACT, int NQ>
__device__ __forceinline__ void prefix_few_block(const Pp &a, int block, float *lds) {
    using T = PTile<CT, DP>;
    constexpr int VD = T::VD, VB = T::VB, PITCH = DP + 4;
    u32x4 *q_lds = (u32x4 *)lds;            // q, and at the end the waves' outputs, 16 columns at a time
    __shared__ float wave_m[kW][16 * NQ], wave_l[kW][16 * NQ];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    Place at;
    if (!place_of(a, block, at)) return;
    const int split = at.split, kv = at.kv, row0 = at.row0, nrows = at.nrows, nh = at.nh, h0 = at.h0;
    const PageSize ps(a.page_size);

    // this lane's columns: their row in the block (-1: none)
    int crow[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int c = n * 16 + col, r = c / a.gm;
        crow[n] = r < nrows && c - r * a.gm < nh ? r : -1;
    }
    // q (with the sign of the scale), as the scores' second operand
    const uint32_t flip = a.scale2 < 0.0f ? (CT == KF32 ? 0x80000000u : 0x80008000u) : 0u;
    const float scale2 = fabsf(a.scale2);
    auto load_q = [&](int lane) {
        const int col = lane & 15, grp = lane >> 4;
#pragma unroll
        for (int i = 0; i < T::KC * T::QW; ++i) {
            if (i % kW != wave) continue;
            const int dim = i / T::QW * 4 * T::KD + grp * T::KD + i % T::QW * 8;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                u32x4 x = {0, 0, 0, 0};
                const int c = n * 16 + col, r = c / a.gm, h = c - r * a.gm;
                if (r < nrows && h < nh && (EXACT || dim < a.d))
                    x = *(const u32x4 *)(a.q + (row0 + r) * a.q_sr + (h0 + h) * a.q_sh + dim * (CT == KF32 ? 4 : 2));
#pragma unroll
                for (int w = 0; w < 4; ++w) x[w] ^= flip;
                q_lds[(i * NQ + n) * 64 + lane] = x;
            }
        }
    };
    load_q(lane);
    Line line = line_of(a, at, lane, T::UNIT);
    const int first = line.first, last = line.last;
    __syncthreads();

    float m[NQ], l[NQ];                      // of the columns; l over this lane's tokens only
    f32x4 acc[NQ][VB][VD];
    auto restart = [&]() {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int i = 0; i < VD; ++i) acc[n][b][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    restart();
    const int64_t to0 = ((int64_t)split * a.batch + row0) * a.n_heads + h0;
    bool left = false;                       // the part of column `tid` has been written
    const char *kb = a.k + kv * a.c_sh + grp * 16, *vb = a.v + kv * a.c_sh;

    // one prefix after the other, with the columns of its rows
    for (; line.leaders; line.leaders &= line.leaders - 1) {
        const int lead = __builtin_ctzll(line.leaders), end = __builtin_amdgcn_readlane(line.upto, lead);
        const int begin = end - __builtin_amdgcn_readlane(line.units, lead);
        const int u0 = max(first, begin) - begin, u1 = min(last, end) - begin;
        if (u0 >= u1) continue;
        const int p = __builtin_amdgcn_readlane(line.id, lead), len = __builtin_amdgcn_readlane(line.len, lead);
        const uint64_t mine = __ballot(line.id == p);
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
        int t0 = u0 * T::UNIT + wave * T::NT;    // (a wave without a tile reads the cache's first row)
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
                u32x4 ph[NQ], pm[NQ], pl[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ph[n][i] = pack_bf16(x[n][2 * i], x[n][2 * i + 1]);
                        const float r0 = x[n][2 * i] - lo_f(ph[n][i]), r1 = x[n][2 * i + 1] - hi_f(ph[n][i]);
                        pm[n][i] = pack_bf16(r0, r1);
                        pl[n][i] = pack_bf16(r0 - lo_f(pm[n][i]), r1 - hi_f(pm[n][i]));
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
                            for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(vt, pm[n], acc[n][b][i]);
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
                                acc[n][b][i] = mfma_bf16(v0, pm[n], acc[n][b][i]);
                                acc[n][b][i + 1] = mfma_bf16(v1, pm[n], acc[n][b][i + 1]);
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

        // ---- join the block's waves, for the columns of this prefix; the others start anew: their weights were 0, but 0
        // times a V that is not finite is NaN
        const int t = formed_here(tid), t_col = t & 15, t_grp = (t & 63) >> 4, t_wave = t >> 6;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            l[n] = head_sum(l[n]);
            if (t_grp == 0) { wave_m[t_wave][n * 16 + t_col] = m[n]; wave_l[t_wave][n * 16 + t_col] = l[n]; }
        }
        __syncthreads();                     // (readers of q, too)
        auto has = [&](int r, int h) { return r < nrows && h < nh && (mine >> r & 1); };
        // a column's maximum and sum, by one thread
        if (t < 16 * NQ) {
            const int r = t / a.gm, h = t - r * a.gm;
            float mt = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int w = 0; w < kW; ++w) mt = fmaxf(mt, wave_m[w][t]);
#pragma unroll
            for (int w = 0; w < kW; ++w) ls += wave_l[w][t] * (mt == -INFINITY ? 1.0f : exp2_fast(wave_m[w][t] - mt));
            if (has(r, h)) {
                *(float2 *)(a.ml + (to0 + r * a.n_heads + h) * 2) = make_float2(mt, ls);
                left = true;
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float top = wave_m[0][n * 16 + t_col];
#pragma unroll
            for (int w = 1; w < kW; ++w) top = fmaxf(top, wave_m[w][n * 16 + t_col]);
            const float f = top == -INFINITY ? 0.0f : exp2_fast(m[n] - top);
            float *to = lds + (t_wave * 16 * NQ + n * 16 + t_col) * PITCH;
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < VD; i += 4)
                        *(float4 *)(to + (b * 16 + t_grp * 4 + r) * VD + i) =
                            make_float4(acc[n][b][i][r] * f, acc[n][b][i + 1][r] * f, acc[n][b][i + 2][r] * f, acc[n][b][i + 3][r] * f);
        }
        __syncthreads();
        constexpr int D4 = DP / 4, SIDE = kNT / D4;          // columns side by side, 4 dims a thread
        const int cc = t / D4, e = (t - cc * D4) * 4;
        if (cc < SIDE && (EXACT || e < a.d)) {
#pragma unroll 4
            for (int c = cc; c < 16 * NQ; c += SIDE) {
                const int r = c / a.gm, h = c - r * a.gm;
                if (!has(r, h)) continue;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kW; ++w) v += *(const f32x4 *)(lds + (w * 16 * NQ + c) * PITCH + e);
                *(f32x4 *)(a.part + (to0 + r * a.n_heads + h) * a.d + e) = v;
            }
        }
        if (end >= last) break;
        __syncthreads();                     // the next prefix: q again, where the outputs were
        load_q(formed_here(lane));
        restart();
        __syncthreads();
    }
    // columns without a token in this part weigh nothing
    if (tid < 16 * NQ && !left) {
        const int r = tid / a.gm, h = tid - r * a.gm;
        if (r < nrows && h < nh) *(float2 *)(a.ml + (to0 + r * a.n_heads + h) * 2) = make_float2(-INFINITY, 0.0f);
    }
}

// ---- many columns: a block's waves have columns of their own and share the tokens
template <int CT, int DP> struct FTile {
    using P = PTile<CT, DP>;
    static constexpr bool F32 = CT == KF32;
    static constexpr int E = P::E, KD = P::KD, KC = P::KC, QW = P::QW, VD = P::VD, VB = P::VB, VW = P::VW;
    // tokens of a tile: 32 KiB of K and V in shared memory, as operands (8-bit ones widened)
    static constexpr int NT = F32 ? (DP <= 64 ? 64 : DP <= 128 ? 32 : 16) : DP <= 128 ? 64 : 32;
    static constexpr int PT = F32 ? 16 : 32;                   // tokens that are weighed at a time
    static constexpr int SUB = NT / 16, KOPS = SUB * KC * QW;
    static constexpr int VOPS = F32 ? NT / 4 * VB : NT / 32 * VB * VD;
    static constexpr int BUF = (KOPS + VOPS) * 64;             // 16-byte operands of a lane, of one buffer
    // V is brought by the first waves, K by the others
    static constexpr int VWAVES = F32 ? 2 : NT / 32 * VB, KWAVES = kW - VWAVES;
    static constexpr int KL = SUB * KC / KWAVES;               // loads of K of a wave
    static constexpr int VL = F32 ? NT / 4 * VB / 2 : 8;       // and of V
    static constexpr int REGS = KL * 4 > VL * VW ? KL * 4 : VL * VW;
    static constexpr uint64_t ALL = NT == 64 ? ~uint64_t(0) : (uint64_t(1) << NT) - 1;
    static_assert(SUB * KC % KWAVES == 0 && VWAVES < kW, "");
};

// For the compiler's order of a run of READS operands from shared memory with PER matrix instructions each: AHEAD
// operands are on their way before the first is used, and one more is asked for with each.
template <int READS, int PER, int AHEAD = 3>
__device__ __forceinline__ void ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD < READS ? AHEAD : READS, 0);
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
        if (i + AHEAD < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
}

// x minus the bf16 value of ph that `which`, a pair of bf16 values, has a -1 for (exact: x is rounded in ph)
__device__ __forceinline__ float minus(uint32_t ph, uint32_t which, float x) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, ph), __builtin_bit_cast(bf16x2, which), x, false);
}

template <int CT, int DP, bool EXACT, int NQ>
__device__ __forceinline__ void prefix_many_block(const Pp &a, int block, u32x4 *bufs) {
    using T = FTile<CT, DP>;                 // bufs: two of: K's operands, V's operands
    constexpr int VD = T::VD, VB = T::VB;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    Place at;
    if (!place_of(a, block, at)) return;
    const PageSize ps(a.page_size);
    Line line = line_of(a, at, lane, T::NT);

    // this lane's columns: their row in the block (-1: none); q with the sign of the scale
    const uint32_t flip = a.scale2 < 0.0f ? (T::F32 ? 0x80000000u : 0x80008000u) : 0u;
    const float scale2 = fabsf(a.scale2);
    int crow[NQ];
    u32x4 q[NQ][T::KC * T::QW];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int c = (wave * NQ + n) * 16 + col, r = c / a.gm;
        const int h = c - r * a.gm;
        crow[n] = r < at.nrows && h < at.nh ? r : -1;
#pragma unroll
        for (int i = 0; i < T::KC * T::QW; ++i) {
            const int dim = i / T::QW * 4 * T::KD + grp * T::KD + i % T::QW * 8;
            u32x4 x = {0, 0, 0, 0};
            if (crow[n] >= 0 && (EXACT || dim < a.d))
                x = *(const u32x4 *)(a.q + (at.row0 + crow[n]) * a.q_sr + (at.h0 + h) * a.q_sh + dim * (T::F32 ? 4 : 2));
#pragma unroll
            for (int w = 0; w < 4; ++w) x[w] ^= flip;
            q[n][i] = x;
        }
    }
    bool any = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) any = any || crow[n] >= 0;
    const bool works = __any(any);           // (a wave without columns only brings K and V)

    float m[NQ], l[NQ];                      // of the columns; l over this lane's tokens only
    f32x4 acc[NQ][VB][VD];
    auto restart = [&]() {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int i = 0; i < VD; ++i) acc[n][b][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    restart();
    bool left[NQ] = {};                      // the column's part has been written
    auto place = [&](int n) {
        const int c = formed_here((wave * NQ + n) * 16 + col), r = c / a.gm;
        return ((int64_t)at.split * a.batch + at.row0 + r) * a.n_heads + at.h0 + c - r * a.gm;
    };
    // -1 in the low or the high half of a pair.  (Out of the compiler's sight: as a constant, 0x0000bf80 becomes the
    // instruction's own -1.0, which stands in the high half.)
    uint32_t low = 0xbf80u, high = 0xbf800000u;
    asm("" : "+s"(low), "+s"(high));
    const char *kb = a.k + at.kv * a.c_sh, *vb = a.v + at.kv * a.c_sh;
    const uint32_t sp16 = (uint32_t)(a.c_sp / 16), st16 = (uint32_t)(a.c_st / 16);

    // one prefix after the other, with the columns of its rows
    for (; line.leaders; line.leaders &= line.leaders - 1) {
        const int lead = __builtin_ctzll(line.leaders), end = __builtin_amdgcn_readlane(line.upto, lead);
        const int begin = end - __builtin_amdgcn_readlane(line.units, lead);
        const int u0 = max(line.first, begin) - begin, u1 = min(line.last, end) - begin;
        if (u0 >= u1) continue;
        const int p = __builtin_amdgcn_readlane(line.id, lead), t_end = min(__builtin_amdgcn_readlane(line.len, lead), u1 * T::NT);
        const uint64_t mine = __ballot(line.id == p);
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
        // (places in 16 bytes: a cache is smaller than 2^36)
        auto off_of = [&](int t0, int page) -> uint32_t {
            const int t = t0 + (lane & (T::NT - 1));
            return (uint32_t)page < (uint32_t)a.n_pages ? (uint32_t)page * sp16 + (uint32_t)ps.place(t, ps.of(t)) * st16 : 0u;
        };
        auto row_of = [&](uint32_t off, int tok) { return (uint64_t)(uint32_t)__shfl((int)off, tok) * 16; };
        uint32_t reg[T::REGS];
        // the wave's part of a tile, from memory
        auto bring = [&](uint32_t off) {
            if (wave < T::VWAVES) {
#pragma unroll
                for (int x = 0; x < T::VL; ++x) {
                    const int i = T::F32 ? wave * T::VL + x : x, g = T::F32 ? i / VB : wave / VB * 8 + x, b = T::F32 ? i % VB : wave % VB;
                    const int dim = (b * 16 + col) * VD;      // past headdim: the row's first dims, in rows of the result that are not kept
                    const Words<T::VW> v = ld_words<T::VW>(vb + row_of(off, (g >> 2) * 16 + grp * 4 + (g & 3)) + (EXACT || dim < a.d ? dim * T::E : 0));
#pragma unroll
                    for (int w = 0; w < T::VW; ++w) reg[x * T::VW + w] = v.w[w];
                }
            } else {
#pragma unroll
                for (int x = 0; x < T::KL; ++x) {
                    const int i = (wave - T::VWAVES) * T::KL + x, s = i / T::KC, c = i - s * T::KC;
                    const bool is = EXACT || (c * 4 + grp) * T::KD < a.d;        // past headdim: the row's own first dims, and zero instead
                    const u32x4 k = *(const u32x4 *)(kb + row_of(off, 16 * s + col) + (is ? c * 64 + grp * 16 : 0));
#pragma unroll
                    for (int w = 0; w < 4; ++w) reg[x * 4 + w] = is ? k[w] : 0u;
                }
            }
        };
        // and as operands into a buffer; tokens that are none get V = 0
        auto put = [&](u32x4 *buf, uint64_t ok) {
            if (wave < T::VWAVES) {
                u32x4 *to = buf + T::KOPS * 64 + lane;
                if (ok != T::ALL) {
#pragma unroll
                    for (int x = 0; x < T::VL; ++x) {
                        const int g = T::F32 ? (wave * T::VL + x) / VB : wave / VB * 8 + x;
                        const bool is = ok >> ((g >> 2) * 16 + grp * 4 + (g & 3)) & 1;
#pragma unroll
                        for (int w = 0; w < T::VW; ++w) reg[x * T::VW + w] = is ? reg[x * T::VW + w] : 0u;
                    }
                }
                if constexpr (T::F32) {
#pragma unroll
                    for (int x = 0; x < T::VL; ++x)
                        to[(wave * T::VL + x) * 64] = (u32x4){reg[x * 4], reg[x * 4 + 1], reg[x * 4 + 2], reg[x * 4 + 3]};
                } else if constexpr (CT == KBF16) {
#pragma unroll
                    for (int i = 0; i < VD; ++i) {
                        u32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = perm(reg[(2 * e + 1) * T::VW + i / 2], reg[2 * e * T::VW + i / 2], i & 1 ? 0x07060302u : 0x05040100u);
                        to[(wave * VD + i) * 64] = v;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VD; i += 2) {
                        u32x4 v0, v1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = perm(reg[(2 * e + 1) * T::VW + i / 4], reg[2 * e * T::VW + i / 4], i & 2 ? 0x07030602u : 0x05010400u);
                            v0[e] = widen<false>(w);
                            v1[e] = widen<true>(w);
                        }
                        to[(wave * VD + i) * 64] = v0;
                        to[(wave * VD + i + 1) * 64] = v1;
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < T::KL; ++x) {
                    u32x4 *to = buf + ((wave - T::VWAVES) * T::KL + x) * T::QW * 64 + lane;
                    const uint32_t *k = reg + x * 4;
                    if constexpr (CT == KF8) {
                        to[0] = (u32x4){widen<false>(k[0]), widen<true>(k[0]), widen<false>(k[1]), widen<true>(k[1])};
                        to[64] = (u32x4){widen<false>(k[2]), widen<true>(k[2]), widen<false>(k[3]), widen<true>(k[3])};
                    } else {
                        to[0] = (u32x4){k[0], k[1], k[2], k[3]};
                    }
                }
            }
        };

        // The pipeline: a tile is weighed from one buffer while the next is on its way to registers, and goes to the
        // other buffer behind it; pages are asked for two tiles ahead.
        int t0 = u0 * T::NT, side = 0;
        int page = page_of(t0);
        uint64_t ok = __ballot((uint32_t)page < (uint32_t)a.n_pages) & T::ALL, ok_next = 0;
        bring(off_of(t0, page));
        page = page_of(t0 + T::NT);
        __syncthreads();                     // readers of the prefix before
        put(bufs, ok);
        ok_next = __ballot((uint32_t)page < (uint32_t)a.n_pages) & T::ALL;
        if (t0 + T::NT < t_end) bring(off_of(t0 + T::NT, page));
        page = page_of(t0 + 2 * T::NT);
        __syncthreads();
        for (; t0 < t_end; t0 += T::NT, side ^= 1) {
            const u32x4 *kop = bufs + side * T::BUF + lane, *vop = kop + T::KOPS * 64;
            if (works) {
                const bool masked = ok != T::ALL || !all_in;
                const uint64_t bits = ok >> (grp * 4);
#pragma unroll
                for (int part = 0; part < T::NT / T::PT; ++part) {
                    constexpr int SUB = T::PT / 16, NX = T::PT / 4, KN = T::KC * T::QW;
                    f32x4 s[NQ][SUB];
                    const u32x4 *kp = kop + part * SUB * KN * 64;
#pragma unroll
                    for (int i = 0; i < SUB; ++i) {
#pragma unroll
                        for (int n = 0; n < NQ; ++n) s[n][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < KN; ++c) {
                            const u32x4 k = kp[(i * KN + c) * 64];
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                if constexpr (T::F32) {
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        s[n][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(q[n][c][e]), s[n][i], 0, 0, 0);
                                } else {
                                    s[n][i] = mfma_bf16(k, q[n][c], s[n][i]);
                                }
                            }
                        }
                    }
                    ahead<SUB * KN, NQ * (T::F32 ? 4 : 1)>();
                    // Scores that do not count are -inf for the maximum, and their weights 0.
                    auto counts = [&](int n, int i) { return (bits >> ((part * SUB + (i >> 2)) * 16 + (i & 3)) & 1) && in[n]; };
                    if (masked) {
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int i = 0; i < NX; ++i) s[n][i >> 2][i & 3] = counts(n, i) ? s[n][i >> 2][i & 3] : -INFINITY;
                    }
                    float top[NQ];
                    bool higher = false;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        top[n] = s[n][0][0];
#pragma unroll
                        for (int i = 1; i < NX; ++i) top[n] = fmaxf(top[n], s[n][i >> 2][i & 3]);
                        top[n] = top[n] == -INFINITY ? -INFINITY : top[n] * scale2;
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
                        const float m_use = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
                        for (int i = 0; i < NX; ++i) s[n][i >> 2][i & 3] = exp2_fast(fmaf(s[n][i >> 2][i & 3], scale2, -m_use));
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < NX; ++i) s[n][i >> 2][i & 3] = counts(n, i) ? s[n][i >> 2][i & 3] : 0.0f;
                        }
#pragma unroll
                        for (int i = 0; i < NX; ++i) l[n] += s[n][i >> 2][i & 3];
                    }
                    if constexpr (T::F32) {
                        const u32x4 *vp = vop + part * NX * VB * 64;
#pragma unroll
                        for (int i = 0; i < NX; ++i)
#pragma unroll
                            for (int b = 0; b < VB; ++b) {
                                const u32x4 v = vp[(i * VB + b) * 64];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
#pragma unroll
                                    for (int n = 0; n < NQ; ++n)
                                        acc[n][b][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[e]), s[n][i >> 2][i & 3], acc[n][b][e], 0, 0, 0);
                            }
                        ahead<NX * VB, NQ * 4>();
                    } else {
                        const u32x4 *vp = vop + part * VB * VD * 64;
                        u32x4 ph[NQ], pm[NQ], pl[NQ];
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float x0 = s[n][i >> 1][2 * i & 3], x1 = s[n][i >> 1][(2 * i & 3) + 1];
                                ph[n][i] = pack_bf16(x0, x1);
                                const float r0 = minus(ph[n][i], low, x0), r1 = minus(ph[n][i], high, x1);
                                pm[n][i] = pack_bf16(r0, r1);
                                pl[n][i] = pack_bf16(minus(pm[n][i], low, r0), minus(pm[n][i], high, r1));
                            }
#pragma unroll
                        for (int b = 0; b < VB; ++b)
#pragma unroll
                            for (int i = 0; i < VD; ++i) {
                                const u32x4 v = vp[(b * VD + i) * 64];
#pragma unroll
                                for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(v, ph[n], acc[n][b][i]);
#pragma unroll
                                for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(v, pm[n], acc[n][b][i]);
#pragma unroll
                                for (int n = 0; n < NQ; ++n) acc[n][b][i] = mfma_bf16(v, pl[n], acc[n][b][i]);
                            }
                        ahead<VB * VD, NQ * 3>();
                    }
                }
            }
            ok = ok_next;
            if (t0 + T::NT < t_end) {
                put(bufs + (side ^ 1) * T::BUF, ok);
                ok_next = __ballot((uint32_t)page < (uint32_t)a.n_pages) & T::ALL;
                if (t0 + 2 * T::NT < t_end) bring(off_of(t0 + 2 * T::NT, page));
                page = page_of(t0 + 3 * T::NT);
            }
            __syncthreads();
        }

        // The columns of this prefix are done, since a row has one.  All start anew, the others too: their weights were 0,
        // but 0 times a V that is not finite is NaN.
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const float sum = head_sum(l[n]);
            if (!in[n]) continue;
            const int64_t to = place(n);
            const int g = formed_here(grp);
            if (g == 0) *(float2 *)(a.ml + to * 2) = make_float2(m[n], sum);
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int dim = (b * 16 + g * 4 + r) * VD;
                    if (!EXACT && dim >= a.d) continue;
#pragma unroll
                    for (int i = 0; i < VD; i += 4)
                        *(f32x4 *)(a.part + to * a.d + dim + i) =
                            (f32x4){acc[n][b][i][r], acc[n][b][i + 1][r], acc[n][b][i + 2][r], acc[n][b][i + 3][r]};
                }
            left[n] = true;
        }
        restart();
    }

    if (grp != 0) return;
#pragma unroll
    for (int n = 0; n < NQ; ++n)             // no token in this part: weighs nothing
        if (crow[n] >= 0 && !left[n]) *(float2 *)(a.ml + place(n) * 2) = make_float2(-INFINITY, 0.0f);
}

// Waves on a SIMD.  Heads of 256 of few columns are left to one where own tokens' share would spill (4 rows of 4 fp32
// kv heads behind 3000 tokens 30.3 us with two, 20.9; in bf16 behind 4000 19.9, 16.1); of many columns two hide more (in bf16
// 512 columns behind 16384 99 with two, 138 with one).
template <int CT, int DP, int NQ, bool MANY>
constexpr int waves_of_prefix() { return MANY || (DP * NQ <= 256 && (DP < 256 || CT == KF8)) ? 2 : 1; }

// The prefixes' blocks, and behind them those of the rows' own tokens (o: paged_attn_kernel.hpp's work).  Behind, since a prefix'
// block takes longer and own ones fill what is left: 64 rows behind 16384 tokens 69 us, 74 in launches of their own, 90 with
// 8 blocks of one kind and 8 of the other in turn; 13 rows of three prompts 24.8, 30.7 in launches of their own.
template <int CT, int DP, bool EXACT, int NQ, bool MANY>
__global__ void __launch_bounds__(kNT, (waves_of_prefix<CT, DP, NQ, MANY>())) prefix_attn_kernel(Pp a, Kp o, int prefix_blocks, int own_blocks) {
    extern __shared__ u32x4 lds[];
    if ((int)blockIdx.x < prefix_blocks) {
        if constexpr (MANY) prefix_many_block<CT, DP, EXACT, NQ>(a, blockIdx.x, lds);
        else prefix_few_block<CT, DP, EXACT, NQ>(a, blockIdx.x, (float *)lds);
    } else {
        paged_attn_block<CT, DP, EXACT, kW, false>(o, blockIdx.x - prefix_blocks, own_blocks, (float *)lds);
    }
}

// Joins the parts of a (row, query head), a wave each; the row's own tokens are one more part.  Lane i forms the weight of part i; then 64 / (d / 4) parts at a time are added up, 4 dims a lane.
template <bool BF16>
__global__ void __launch_bounds__(kNT) prefix_join_kernel(Pp a) {
    const int lane = threadIdx.x & 63;
    const int64_t rh = (int64_t)blockIdx.x * kW + (threadIdx.x >> 6), all = (int64_t)a.batch * a.n_heads;
    if (rh >= all) return;
    const int d4 = a.d / 4, side = 64 / d4, sub = lane / d4, e = (lane - sub * d4) * 4;
    const bool has = sub < side;
    const float2 own = *(const float2 *)(a.ml_own + rh * 2);
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (lane < d4) o = *(const f32x4 *)(a.o_own + rh * a.d + e);
    float2 w = make_float2(-INFINITY, 0.0f);                  // (at most 64 parts)
    if (lane < a.splits) w = *(const float2 *)(a.ml + (lane * all + rh) * 2);
    float m = fmaxf(own.x, w.x);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float m_use = m == -INFINITY ? 0.0f : m, f = exp2_fast(w.x - m_use), own_f = exp2_fast(own.x - m_use);
    float sum = w.y == 0.0f ? 0.0f : w.y * f;
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
    sum += own.y == 0.0f ? 0.0f : own.y * own_f;
    // what weighs nothing is not added, and of a part may never have been written
    o = own_f > 0.0f && own.y != 0.0f ? o * (own_f * a.v_scale) : (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    const float part_f = f > 0.0f && w.y != 0.0f ? f * a.v_scale : 0.0f;
    // (read all the same, eight on their way together, and not used)
    const float *part = a.part + rh * a.d + (has ? e : 0);
    for (int s0 = 0; s0 < a.splits; s0 += 8 * side) {
        f32x4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *(const f32x4 *)(part + min(s0 + i * side + sub, a.splits - 1) * all * a.d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = s0 + i * side + sub;
            const float x = __shfl(part_f, s & 63);
            o += has && s < a.splits && x != 0.0f ? v[i] * x : (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    for (int s = 1; s < side; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = __shfl(o[i], lane + s * d4);
            o[i] += sub == 0 ? x : 0.0f;
        }
    const float n = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    if (lane < d4) {
        if constexpr (BF16) *(uint2 *)(a.o + (rh * a.d + e) * 2) = make_uint2(pack_bf16(o[0] * n, o[1] * n), pack_bf16(o[2] * n, o[3] * n));
        else *(f32x4 *)(a.o + (rh * a.d + e) * 4) = o * n;
    }
    if (lane == 0 && a.lse) a.lse[rh] = m_use * kLn2 + logf(sum);
}

// ------------------------------------------------------------------ host ----
// How the columns of all rows are cut into blocks.  us, all rows behind one prefix, 100 tokens of their own
// (few of 16 columns, few of 32, many of 64, many of 128; for d = 256 the last is not built):
//   heads of 128, bf16, 8 kv heads, 16384 tokens:  16 columns 25.4, 26.1, 26.0, 30.2;  40: 29.8, 27.6, 29.1, 34.1;
//     128: 53, 38, 38, 46;  256: 89, 57, 55, 57;  384: 153, 78, 70, 71;  1024: 311, 178, 157, 145
//   of 128, 8 bits, 4 kv heads, 16384 tokens:  256: 38, 33, 42, 42;  512: 64, 50, 60, 53;  1024: 111, 82, 97, 80
//   of 64, bf16, 4 kv heads, 16384 tokens:  256: 35, 27, 30, 33;  512: 58, 40, 42, 41;  1024: 106, 66, 67, 61
//   of 128, fp32, 4 kv heads, 4000 tokens:  16: 13.8, 16.3, 20.3, 30.2;  128: 30.5, 33.2, 29.4, 38.8;  1024: 118, 109, 109, 113
//   of 256, bf16, 4 kv heads, 4000 tokens:  16: 18.0, 17.5, 19.1;  32: 22.6, 19.3, 21.4;  64: 32, 27.5, 25.5;  1024: 115, 89, 81
// So 32 columns to a block, 16 if there are no more; up to 128 dims many of 128 from 2^25 scores on, where K and V out of
// the L2s cost more than the way through shared memory; above 128 dims, where a wave of 32 columns keeps one block a
// compute unit, many of 64 from 33 columns on.
//
// Form and parts go by the room of prefix_table, since the host does not know the lengths: the 13 rows of three prompts of up to 4001
// tokens take 17.3 us with room for up to 32768, and 23.3 with room for 131072, where they are of the form for many.
//
// Two blocks a compute unit from 2^24 scores on, one below, where the own tokens' blocks then run beside them and there are
// fewer parts to join (two, one): 48 columns of the 8-bit heads above 24.2, 18.3;  160 of them 35.5, 29.1;
// 256 33.3, 36.7;  512 50.4, 61;  256 of 4 kv heads of 128, 8 bits, 4000 tokens 23.1, 17.7;  1024 of these 40.7, 37.1.
struct Cut { int nq, gm, passes, rows, tiles, splits; bool many; };
Cut cut_of(int64_t batch, int64_t n_heads, int64_t n_kv, int64_t d, int64_t max_len, int64_t n_prefixes) {
    Cut c;
    const int64_t group = n_heads / n_kv, all = batch * group;
    const double scores = (double)n_kv * all * max_len;       // of all rows with one prefix
    c.many = d > 128 ? all > 32 : all > 64 && scores >= 1 << 25;
    c.nq = d > 128 && c.many ? 1 : all > 16 ? 2 : 1;
    const int64_t cols = 16 * c.nq * (c.many ? kW : 1);
    c.gm = (int)std::min<int64_t>(group, cols);
    c.passes = (int)((group + c.gm - 1) / c.gm);
    c.rows = (int)std::min<int64_t>(std::min<int64_t>(batch, cols / c.gm), 64);
    c.tiles = (int)((batch + c.rows - 1) / c.rows);
    // the same number of blocks on each XCD, of at least some 128 tokens (2 rows of 4 kv heads of 128, 8 bits, behind 4000:
    // of 64 14.6 us, 128 11.8, 256 11.1, 512 13.0; bf16 of 64 11.9, 10.0, 10.7, 12.7)
    const int64_t units = std::max<int64_t>(1, (max_len + 127) / 128 * std::min<int64_t>(n_prefixes, c.rows));
    const int64_t each = kCUs / 8 * (scores >= 1 << 24 ? 2 : 1) / c.tiles;
    c.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(8 * each / (n_kv * c.passes), units), 64));
    return c;
}

int blocks_of(const Pp &k) { return (k.combos + 7) / 8 * 8 * k.tiles; }

template <typename F, typename... A>
hipError_t launch_with(F kernel, size_t lds, int grid, hipStream_t stream, A... args) {
    if (lds > 32 * 1024) {               // more than a block has unasked, from 64 KiB on
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kNT), lds, stream, args...);
    return hipGetLastError();
}

// A call: `own` the rows' own tokens, whose output goes to the workspace.
struct Call { const PagedAttnArgs &own; const Cut &cut; hipStream_t stream; const char **kernel_name; };

template <int CT, int DP, bool EXACT, int NQ, bool MANY>
hipError_t go_m(const Pp &k, const Call &c) {
    using T = PTile<CT, DP>;
    const size_t lds = MANY ? 2 * FTile<CT, DP>::BUF * 16
                            : std::max((size_t)kW * 16 * NQ * (DP + 4) * sizeof(float), (size_t)T::KC * T::QW * NQ * 1024);
    Kp o = kernel_args(c.own);
    o.whole = form_of<CT, DP>(o).whole;
    int own_blocks = 0;
    const int blocks = blocks_of(k);
    const size_t own_lds = plan_w<CT, DP, kW>(o, own_blocks);
    *c.kernel_name = "prefix_attn_kernel";
    const hipError_t e = launch_with(prefix_attn_kernel<CT, DP, EXACT, NQ, MANY>, std::max(lds, own_lds), blocks + own_blocks, c.stream,
                                     k, o, blocks, own_blocks);
    return e != hipSuccess || o.whole ? e : launch_join(c.own, o, own_blocks, c.stream, c.kernel_name);
}
template <int CT, int DP, bool EXACT, int NQ>
hipError_t go_q(const Pp &k, const Call &c) {
    if constexpr (NQ == (DP <= 128 ? 2 : 1)) {
        if (c.cut.many) return go_m<CT, DP, EXACT, NQ, true>(k, c);
    }
    return go_m<CT, DP, EXACT, NQ, false>(k, c);
}
template <int CT, int DP>
hipError_t go_d(const Pp &k, const Call &c) {
    if (k.d == DP) return c.cut.nq == 2 ? go_q<CT, DP, true, 2>(k, c) : go_q<CT, DP, true, 1>(k, c);
    return c.cut.nq == 2 ? go_q<CT, DP, false, 2>(k, c) : go_q<CT, DP, false, 1>(k, c);
}
template <int CT>
hipError_t go_type(const Pp &k, const Call &c) {
    if (k.d <= 64) return go_d<CT, 64>(k, c);
    if (k.d <= 128) return go_d<CT, 128>(k, c);
    if (k.d <= 192) return go_d<CT, 192>(k, c);
    return go_d<CT, 256>(k, c);
}

}  // namespace

size_t prefix_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                   int64_t max_prefix_pages, int64_t max_pages, int64_t page_size) {
    const Cut c = cut_of(batch, n_heads, n_kv_heads, headdim, max_prefix_pages * page_size, batch);   // (the most splits that any number has)
    const int64_t rh = batch * n_heads;
    return align16(paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, headdim, max_pages, page_size)) +
           align16(rh * headdim * 4) + align16(rh * 8) + align16(c.splits * rh * 8) + c.splits * rh * headdim * 4;
}

hipError_t launch_prefix_attn(const PrefixAttnArgs &p, hipStream_t stream, const char **kernel_name) {
    PagedAttnArgs a = p.own;
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    const int64_t rh = a.batch * a.n_heads;
    const Cut c = cut_of(a.batch, a.n_heads, a.n_kv_heads, a.headdim, p.max_prefix_pages * a.page_size, p.n_prefixes);
    char *ws = (char *)a.workspace + align16(paged_attn_workspace_bytes(a.batch, a.n_heads, a.n_kv_heads, a.headdim, a.max_pages, a.page_size));
    Pp k = {};
    k.o_own = (const float *)ws; ws += align16(rh * a.headdim * 4);
    k.ml_own = (const float *)ws; ws += align16(rh * 8);
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

    a.o = (void *)k.o_own; a.lse = (float *)k.ml_own; a.raw = true;
    const Call call{a, c, stream, kernel_name};
    const hipError_t rc = a.kv_dtype == SSM_KV_F32 ? go_type<KF32>(k, call)
                        : a.kv_dtype == SSM_KV_BF16 ? go_type<KBF16>(k, call) : go_type<KF8>(k, call);
    if (rc != hipSuccess) return rc;
    *kernel_name = "prefix_join_kernel";
    const dim3 grid((unsigned)((rh + kW - 1) / kW));
    if (a.kv_dtype != SSM_KV_F32) hipLaunchKernelGGL((prefix_join_kernel<true>), grid, dim3(kNT), 0, stream, k);
    else hipLaunchKernelGGL((prefix_join_kernel<false>), grid, dim3(kNT), 0, stream, k);
    return hipGetLastError();
}

}  // namespace ssm
