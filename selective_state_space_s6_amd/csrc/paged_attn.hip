// paged_attn.hip -- attention of one new token over a paged key-value cache
// (ssm_paged_attn_decode_fwd in include/ssm_attn.h).
//
// Every cached byte is read once, for the query heads that share it, so the bound
// is HBM (one request alone: latency).  The work is cut by length: a unit is 128
// tokens of one (row, kv head), the units of all rows stand in one line, and each
// block takes an equal piece of it, whatever the rows' lengths are.  A piece that
// does not hold a whole (row, kv head) leaves its unnormalised output, maximum and
// sum in the workspace, and a second kernel joins those.
//
// Inside a block every wave walks tiles of 32 (fp32: 16) tokens of its own with a
// running maximum and sum, and takes its operands from global memory straight into
// the matrix instructions' registers:
//  - scores S^T = K Q^T: a lane's 16 bytes of a K row are its operand as they
//    are.  Up to 16 query heads are the columns; unused ones are zero.
//  - output O^T = V^T P^T: a lane of the scores' result holds head lane % 16 and
//    tokens 4 (lane / 16) + {0..3} (+ 16), and that is the lane's share of P^T as an
//    operand if the contraction takes the tokens in that order.  So each lane loads
//    those V rows (its own 8 or 4 dims of them), and transposes them in registers
//    with byte permutations.  Nothing passes through LDS before a piece's end.
//  - the result's columns are heads too, so the running maximum and sum that scale
//    it are the lane's own.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kNT = 256;
constexpr int kWaves = kNT / 64;
constexpr int kHeads = 16;          // query heads of a pass
constexpr int kUnit = 128;          // tokens of a unit of work
constexpr int kBlocks = 768;        // pieces of work: 3 blocks on each of 256 compute units

enum { KBF16, KF8, KF32 };

struct Kp {
    const char *q; const char *k; const char *v; const int32_t *table; const int32_t *lens; char *o; float *lse;
    int32_t *start;                 // units before each row (batch + 1)
    float *part;                    // unjoined outputs: (2 blocks, heads of a pass, d)
    float *ml;                      // and their maxima and sums: (2 blocks, heads of a pass, 2)
    int64_t table_stride, q_sr, q_sh, c_sh;    // q and cache strides in bytes
    uint32_t c_sp16, c_st16;        // cache strides of page and token in 16 bytes
    int batch, n_heads, n_kv, group, passes, gmax;   // group: query heads a kv head; passes of gmax <= 16 of them
    int d, n_pages, page_size, max_len, window;
    float scale2, v_scale;          // scale2: score -> log2 units
};

// The tokens of a row: [lo, hi), from `base` (a multiple of a tile) in `units` units
struct Span { int lo, hi, base, units; };
__device__ __forceinline__ Span span_of(const Kp &a, int r) {
    Span s;
    s.hi = min(max(a.lens[r], 0), a.max_len);
    s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
    s.base = s.lo & ~31;
    s.units = (s.hi - s.base + kUnit - 1) / kUnit;
    return s;
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);   // to nearest even
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// two 8-bit values -> two bf16, exact
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
    return __builtin_bit_cast(uint32_t, r);
}
// bytes of lo (0-3) and hi (4-7) picked by sel
__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
    return __builtin_amdgcn_perm(hi, lo, sel);
}
// over the four lanes that hold a head
__device__ __forceinline__ float head_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float head_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// One (cache type, padded head size): register shapes of a tile
template <int CT, int DP> struct Tile {
    static constexpr int NT = CT == KF32 ? 16 : 32;            // tokens
    static constexpr int SUB = NT / 16;                        // 16-token blocks of scores
    static constexpr int E = CT == KF32 ? 4 : CT == KBF16 ? 2 : 1;
    static constexpr int KD = 16 / E;                          // dims of a 16-byte load of K
    static constexpr int KC = DP / (4 * KD);                   // loads of a K row (four lanes each)
    static constexpr int VD = CT == KF32 || DP % 128 ? 4 : 8;  // dims of a lane's load of V
    static constexpr int VB = DP / (16 * VD);                  // loads of a V row (16 lanes each)
    static constexpr int VW = VD * E / 4;                      // dwords of one
    static constexpr int VR = NT / 4;                          // V rows of a lane
    static constexpr int QW = CT == KF8 ? 2 : 1;               // operands of q to a K load
};

template <int N> struct Words { uint32_t w[N]; };
template <int N>
__device__ __forceinline__ Words<N> ld_words(const char *p) {
    Words<N> r;
    if constexpr (N == 4) {
        const uint4 u = *(const uint4 *)p;
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *(const uint2 *)p;
        r.w[0] = u.x; r.w[1] = u.y;
    } else {
        r.w[0] = *(const uint32_t *)p;
    }
    return r;
}

template <int CT, int DP, bool EXACT>      // EXACT: headdim == DP
__global__ void __launch_bounds__(kNT, 2) paged_attn_kernel(Kp a) {
    using T = Tile<CT, DP>;
    constexpr int VD = T::VD, VB = T::VB;
    extern __shared__ float lds[];          // the waves' outputs, at a piece's end
    __shared__ int scan[kWaves], found[3];
    __shared__ float wave_m[kWaves][kHeads], wave_l[kWaves][kHeads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 15, grp = lane >> 4;

    // ---- this block's piece [u, u_end) of the line of units, and the row that u is in
    const int per = a.n_kv * a.passes;      // (kv head, pass) of a row
    int units = 0;
    for (int r0 = 0; r0 < a.batch; r0 += kNT) {
        const int r = r0 + tid;
        units += r < a.batch ? span_of(a, r).units : 0;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) units += __shfl_xor(units, o);
    if (lane == 0) scan[wave] = units;
    __syncthreads();
    units = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) units += scan[w];
    units *= per;
    const int blocks = min((int)gridDim.x, units), blk = blockIdx.x;
    if (blk > 0 && blk >= blocks) return;
    int u = blocks ? (int)((int64_t)blk * units / blocks) : 0;
    const int u_end = blocks ? (int)((int64_t)(blk + 1) * units / blocks) : 0;
    for (int r0 = 0, base = 0; r0 < a.batch; r0 += kNT) {
        const int r = r0 + tid;
        const int n = r < a.batch ? span_of(a, r).units * per : 0;
        int v = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int b = __shfl_up(v, o);
            if (lane >= o) v += b;
        }
        __syncthreads();
        if (lane == 63) scan[wave] = v;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            v += w < wave ? scan[w] : 0;
            total += scan[w];
        }
        v += base - n;                       // units before row r
        if (n > 0 && u >= v && u < v + n) { found[0] = r; found[1] = v; }
        if (blk == 0 && r < a.batch) a.start[r] = v;
        base += total;
    }
    if (blk == 0 && tid == 0) a.start[a.batch] = units;
    __syncthreads();
    if (u >= u_end) return;
    int row = found[0], row_u = found[1];

    while (u < u_end) {
        Span sp = span_of(a, row);
        while (u >= row_u + sp.units * per) {
            row_u += sp.units * per;
            sp = span_of(a, ++row);
        }
        const int at = u - row_u, hp = at / sp.units, first = at - hp * sp.units;
        const int last = min(sp.units, first + (u_end - u));          // units [first, last) of this head
        const int kv = hp / a.passes, pass = hp - kv * a.passes;
        const int nh = min(a.gmax, a.group - pass * a.gmax);          // query heads of this pass
        const int h0 = kv * a.group + pass * a.gmax;
        u += last - first;

        // q, as the scores' second operand
        u32x4 qf[T::KC * T::QW];
#pragma unroll
        for (int c = 0; c < T::KC; ++c)
#pragma unroll
            for (int w = 0; w < T::QW; ++w) {
                const int dim = c * 4 * T::KD + grp * T::KD + w * 8;
                u32x4 x = {0, 0, 0, 0};
                if (col < nh && (EXACT || dim < a.d))
                    x = *(const u32x4 *)(a.q + row * a.q_sr + (h0 + col) * a.q_sh + dim * (CT == KF32 ? 4 : 2));
                qf[c * T::QW + w] = x;
            }

        float m = -INFINITY, l = 0.0f;       // of head col; l over this lane's tokens only
        f32x4 acc[VB][VD];
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < VD; ++i) acc[b][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

        const char *kb = a.k + kv * a.c_sh + grp * 16, *vb = a.v + kv * a.c_sh + col * VD * T::E;
        const int32_t *table = a.table + row * a.table_stride;
        const int t_end = min(sp.hi, sp.base + last * kUnit);
        for (int t0 = sp.base + first * kUnit + wave * T::NT; t0 < t_end; t0 += kWaves * T::NT) {
            // this lane's token of the tile: its place in the cache, in 16 bytes; rows that
            // are not the request's are read at the cache's first row and masked
            const int t = t0 + (lane & (T::NT - 1));
            bool valid = t >= sp.lo && t < sp.hi;
            uint32_t off = 0;
            if (valid) {
                const uint32_t p = (uint32_t)t / (uint32_t)a.page_size;
                const int page = table[p];
                valid = page >= 0 && page < a.n_pages;
                if (valid) off = (uint32_t)page * a.c_sp16 + ((uint32_t)t - p * (uint32_t)a.page_size) * a.c_st16;
            }
            const uint32_t ok = (uint32_t)__ballot(valid);
            const bool full = T::NT == 32 ? ok == 0xffffffffu : (ok & 0xffffu) == 0xffffu;

            u32x4 kf[T::SUB][T::KC];
#pragma unroll
            for (int s = 0; s < T::SUB; ++s) {
                const char *p = kb + (uint64_t)__shfl(off, 16 * s + col) * 16;
#pragma unroll
                for (int c = 0; c < T::KC; ++c) {
                    kf[s][c] = (u32x4){0, 0, 0, 0};
                    if (EXACT || (c * 4 + grp) * T::KD < a.d) kf[s][c] = *(const u32x4 *)(p + c * 64);
                }
            }
            Words<T::VW> vf[T::VR][VB];
#pragma unroll
            for (int j = 0; j < T::VR; ++j) {
                const int tok = (j >> 2) * 16 + grp * 4 + (j & 3);
                const char *p = vb + (uint64_t)__shfl(off, tok) * 16;
                const bool have = full || (ok >> tok & 1);
#pragma unroll
                for (int b = 0; b < VB; ++b) {
#pragma unroll
                    for (int w = 0; w < T::VW; ++w) vf[j][b].w[w] = 0;
                    if (have && (EXACT || (b * 16 + col) * VD < a.d)) vf[j][b] = ld_words<T::VW>(p + b * 16 * VD * T::E);
                }
            }

            f32x4 s[T::SUB];
#pragma unroll
            for (int i = 0; i < T::SUB; ++i) {
                s[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < T::KC; ++c) {
                    const u32x4 k = kf[i][c];
                    if constexpr (CT == KBF16) {
                        s[i] = mfma_bf16(k, qf[c], s[i]);
                    } else if constexpr (CT == KF8) {
                        const u32x4 k0 = {widen<false>(k[0]), widen<true>(k[0]), widen<false>(k[1]), widen<true>(k[1])};
                        const u32x4 k1 = {widen<false>(k[2]), widen<true>(k[2]), widen<false>(k[3]), widen<true>(k[3])};
                        s[i] = mfma_bf16(k0, qf[2 * c], s[i]);
                        s[i] = mfma_bf16(k1, qf[2 * c + 1], s[i]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(qf[c][e]), s[i], 0, 0, 0);
                    }
                }
            }
            float x[T::VR], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < T::VR; ++j) {
                const int tok = (j >> 2) * 16 + grp * 4 + (j & 3);
                const float v = s[j >> 2][j & 3] * a.scale2;
                x[j] = full || (ok >> tok & 1) ? v : -INFINITY;
                top = fmaxf(top, x[j]);
            }
            const float m_new = fmaxf(m, head_max(top));
            const float m_use = m_new == -INFINITY ? 0.0f : m_new;     // no token yet: all p are 0
            if (__any(m_new > m)) {
                const float f = exp2_fast(m - m_use);
                l *= f;
#pragma unroll
                for (int b = 0; b < VB; ++b)
#pragma unroll
                    for (int i = 0; i < VD; ++i) acc[b][i] *= f;
                m = m_new;
            }
#pragma unroll
            for (int j = 0; j < T::VR; ++j) {
                x[j] = exp2_fast(x[j] - m_use);
                l += x[j];
            }
            if constexpr (CT == KF32) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[j][b].w[i]), x[j], acc[b][i], 0, 0, 0);
            } else {
                // p as the sum of two bf16 values: one alone would double the output's error
                u32x4 ph, pl;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ph[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                    pl[j] = pack_bf16(x[2 * j] - lo_f(ph[j]), x[2 * j + 1] - hi_f(ph[j]));
                }
#pragma unroll
                for (int b = 0; b < VB; ++b) {
                    if constexpr (CT == KBF16) {
#pragma unroll
                        for (int i = 0; i < VD; ++i) {
                            u32x4 vt;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                vt[j] = perm(vf[2 * j + 1][b].w[i / 2], vf[2 * j][b].w[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
                            acc[b][i] = mfma_bf16(vt, ph, acc[b][i]);
                            acc[b][i] = mfma_bf16(vt, pl, acc[b][i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VD; i += 2) {
                            u32x4 v0, v1;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t w = perm(vf[2 * j + 1][b].w[i / 4], vf[2 * j][b].w[i / 4], i & 2 ? 0x07030602u : 0x05010400u);
                                v0[j] = widen<false>(w);
                                v1[j] = widen<true>(w);
                            }
                            acc[b][i] = mfma_bf16(v0, ph, acc[b][i]);
                            acc[b][i] = mfma_bf16(v0, pl, acc[b][i]);
                            acc[b][i + 1] = mfma_bf16(v1, ph, acc[b][i + 1]);
                            acc[b][i + 1] = mfma_bf16(v1, pl, acc[b][i + 1]);
                        }
                    }
                }
            }
        }

        // ---- join the four waves
        l = head_sum(l);
        __syncthreads();                     // readers of the segment before
        if (grp == 0) { wave_m[wave][col] = m; wave_l[wave][col] = l; }
        __syncthreads();
        float top = wave_m[0][col];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, wave_m[w][col]);
        const float f = top == -INFINITY ? 0.0f : exp2_fast(m - top);
        constexpr int PITCH = DP + 4;
        if (col < nh) {
            float *p = lds + (wave * a.gmax + col) * PITCH;
#pragma unroll
            for (int b = 0; b < VB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < VD; i += 4)
                        *(float4 *)(p + (b * 16 + grp * 4 + r) * VD + i) =
                            make_float4(acc[b][i][r] * f, acc[b][i + 1][r] * f, acc[b][i + 2][r] * f, acc[b][i + 3][r] * f);
        }
        __syncthreads();
        const bool whole = first == 0 && last == sp.units;
        const int slot = 2 * blk + (first == 0 ? 1 : 0);
        const int d4 = a.d / 4;
        for (int i = tid; i < nh * d4; i += kNT) {
            const int h = i / d4, e = (i - h * d4) * 4;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            float ls = 0.0f, mt = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                v += *(const f32x4 *)(lds + (w * a.gmax + h) * PITCH + e);
                mt = fmaxf(mt, wave_m[w][h]);
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w) ls += wave_l[w][h] * (mt == -INFINITY ? 0.0f : exp2_fast(wave_m[w][h] - mt));
            if (whole) {
                const float n = ls > 0.0f || ls != ls ? a.v_scale / ls : 0.0f;
                const int64_t to = ((int64_t)row * a.n_heads + h0 + h) * a.d + e;
                if constexpr (CT == KF32) *(f32x4 *)(a.o + to * 4) = v * n;
                else *(uint2 *)(a.o + to * 2) = make_uint2(pack_bf16(v[0] * n, v[1] * n), pack_bf16(v[2] * n, v[3] * n));
                if (e == 0 && a.lse) a.lse[(int64_t)row * a.n_heads + h0 + h] = (mt == -INFINITY ? 0.0f : mt * kLn2) + logf(ls);
            } else {
                *(f32x4 *)(a.part + ((int64_t)slot * a.gmax + h) * a.d + e) = v;
                if (e == 0) *(float2 *)(a.ml + ((int64_t)slot * a.gmax + h) * 2) = make_float2(mt, ls);
            }
        }
    }
}

// Joins the pieces of one (row, query head): piece i's share is scaled by
// 2^(m_i - max m).  Rows without tokens get o = 0, lse = -inf here.
template <bool BF16>
__global__ void __launch_bounds__(kNT) paged_attn_join_kernel(Kp a, int grid) {
    __shared__ float red[kWaves], out[kNT * 4];
    const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = a.n_kv * a.passes;
    const int kv = h / a.group, pass = (h - kv * a.group) / a.gmax, hh = h - kv * a.group - pass * a.gmax;
    const int64_t total = a.start[a.batch];
    const int nu = (a.start[row + 1] - a.start[row]) / per;
    const int64_t to = ((int64_t)row * a.n_heads + h) * a.d;
    if (nu == 0) {
        for (int e = tid; e < a.d; e += kNT) {
            if (BF16) ((uint16_t *)a.o)[to + e] = 0;
            else ((float *)a.o)[to + e] = 0.0f;
        }
        if (tid == 0 && a.lse) a.lse[(int64_t)row * a.n_heads + h] = -INFINITY;
        return;
    }
    // the blocks whose pieces hold this head's first and last unit
    const int64_t blocks = min((int64_t)grid, total), u0 = a.start[row] + (int64_t)(kv * a.passes + pass) * nu;
    const int b0 = (int)(((u0 + 1) * blocks - 1) / total), b1 = (int)(((u0 + nu) * blocks - 1) / total);
    if (b0 == b1) return;                    // written whole
    const int n = b1 - b0 + 1;
    // the first block began this head (its second place); the others go on with it (their first)
    auto place = [&](int i) { return (int64_t)(i == 0 ? 2 * b0 + 1 : 2 * (b0 + i)) * a.gmax + hh; };
    float m = -INFINITY;
    for (int i = tid; i < n; i += kNT) m = fmaxf(m, a.ml[place(i) * 2]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) red[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m_use = m == -INFINITY ? 0.0f : m;
    __syncthreads();
    float l = 0.0f;
    for (int i = tid; i < n; i += kNT) l += a.ml[place(i) * 2 + 1] * exp2_fast(a.ml[place(i) * 2] - m_use);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
    if (lane == 0) red[wave] = l;
    const int d4 = a.d / 4, slices = kNT / d4, sl = tid / d4, e = (tid - sl * d4) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (sl < slices)
        for (int i = sl; i < n; i += slices)
            v += *(const f32x4 *)(a.part + place(i) * a.d + e) * exp2_fast(a.ml[place(i) * 2] - m_use);
    *(f32x4 *)(out + tid * 4) = v;
    __syncthreads();
    l = red[0] + red[1] + red[2] + red[3];
    if (tid < d4) {
        for (int s = 1; s < slices; ++s) v += *(const f32x4 *)(out + (s * d4 + tid) * 4);
        v *= l > 0.0f || l != l ? a.v_scale / l : 0.0f;
        if (BF16) *(uint2 *)(a.o + (to + e) * 2) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else *(f32x4 *)(a.o + (to + e) * 4) = v;
    }
    if (tid == 0 && a.lse) a.lse[(int64_t)row * a.n_heads + h] = m_use * kLn2 + logf(l);
}

// ------------------------------------------------------------------ host ----
int64_t passes_of(int64_t group) { return (group + kHeads - 1) / kHeads; }
int64_t align16(int64_t n) { return (n + 15) & ~int64_t(15); }

// shared memory a block may have beyond the default needs no attribute up to 64 KiB; the
// widest case (four waves, 16 heads, 256 dims) takes 65 KiB
template <int CT, int DP, bool EXACT>
hipError_t go(const Kp &k, int grid, hipStream_t stream) {
    const size_t lds = (size_t)kWaves * k.gmax * (DP + 4) * sizeof(float);
    if (lds > 64 * 1024 - 1024) {
        const hipError_t e = hipFuncSetAttribute((const void *)paged_attn_kernel<CT, DP, EXACT>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_attn_kernel<CT, DP, EXACT>), dim3((unsigned)grid), dim3(kNT), lds, stream, k);
    return hipGetLastError();
}
template <int CT, int DP>
hipError_t go_d(const Kp &k, int grid, hipStream_t stream) {
    return k.d == DP ? go<CT, DP, true>(k, grid, stream) : go<CT, DP, false>(k, grid, stream);
}
template <int CT>
hipError_t go_type(const Kp &k, int grid, hipStream_t stream) {
    if (k.d <= 64) return go_d<CT, 64>(k, grid, stream);
    if (k.d <= 128) return go_d<CT, 128>(k, grid, stream);
    if (k.d <= 192) return go_d<CT, 192>(k, grid, stream);
    return go_d<CT, 256>(k, grid, stream);
}

}  // namespace

double paged_attn_max_units(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size) {
    const double len = (double)max_pages * (double)page_size;
    return (double)batch * (double)n_kv_heads * (double)passes_of(n_heads / n_kv_heads) * ((len + kUnit - 1) / kUnit);
}

static int64_t grid_of(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size) {
    const double most = paged_attn_max_units(batch, n_heads, n_kv_heads, max_pages, page_size);
    return most < kBlocks ? std::max<int64_t>(1, (int64_t)most) : kBlocks;
}

size_t paged_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                  int64_t max_pages, int64_t page_size) {
    const int64_t group = n_heads / n_kv_heads, gmax = std::min<int64_t>(group, kHeads);
    const int64_t places = 2 * grid_of(batch, n_heads, n_kv_heads, max_pages, page_size) * gmax;
    return (size_t)(align16((batch + 1) * 4) + align16(places * 8) + places * headdim * 4);
}

hipError_t launch_paged_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "paged_attn_kernel";
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    const int64_t grid = grid_of(a.batch, a.n_heads, a.n_kv_heads, a.max_pages, a.page_size);
    Kp k = {};
    k.q = (const char *)a.q; k.k = (const char *)a.k_cache; k.v = (const char *)a.v_cache;
    k.table = a.block_table; k.lens = a.lens; k.o = (char *)a.o; k.lse = a.lse;
    k.group = (int)(a.n_heads / a.n_kv_heads);
    k.gmax = std::min(k.group, kHeads);
    k.passes = (int)passes_of(k.group);
    char *ws = (char *)a.workspace;
    k.start = (int32_t *)ws; ws += align16((a.batch + 1) * 4);
    k.ml = (float *)ws; ws += align16(2 * grid * k.gmax * 8);
    k.part = (float *)ws;
    k.table_stride = a.table_stride; k.q_sr = a.q_sr * qe; k.q_sh = a.q_sh * qe; k.c_sh = a.c_sh * e;
    k.c_sp16 = (uint32_t)(a.c_sp * e / 16); k.c_st16 = (uint32_t)(a.c_st * e / 16);
    k.batch = (int)a.batch; k.n_heads = (int)a.n_heads; k.n_kv = (int)a.n_kv_heads;
    k.d = a.headdim; k.n_pages = (int)a.n_pages; k.page_size = (int)a.page_size;
    k.max_len = (int)(a.max_pages * a.page_size);
    k.window = a.window > 0 && a.window < k.max_len ? (int)a.window : 0;
    k.scale2 = a.scale * (a.kv_dtype == SSM_KV_F8E4M3 ? a.k_scale : 1.0f) * kLog2e;
    k.v_scale = a.kv_dtype == SSM_KV_F8E4M3 ? a.v_scale : 1.0f;
    const hipError_t rc = a.kv_dtype == SSM_KV_F32 ? go_type<KF32>(k, (int)grid, stream)
                        : a.kv_dtype == SSM_KV_BF16 ? go_type<KBF16>(k, (int)grid, stream)
                                                    : go_type<KF8>(k, (int)grid, stream);
    if (rc != hipSuccess) return rc;
    *kernel_name = "paged_attn_join_kernel";
    const dim3 g((unsigned)a.batch, (unsigned)a.n_heads);
    if (a.kv_dtype == SSM_KV_F32) hipLaunchKernelGGL((paged_attn_join_kernel<false>), g, dim3(kNT), 0, stream, k, (int)grid);
    else hipLaunchKernelGGL((paged_attn_join_kernel<true>), g, dim3(kNT), 0, stream, k, (int)grid);
    return hipGetLastError();
}

}  // namespace ssm
