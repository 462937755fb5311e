// paged_attn.hip -- attention of one new token over a paged key-value cache
// (ssm_paged_attn_decode_fwd in include/ssm_attn.h).
//
// o = sum_t p_t v_t / sum_t p_t with p_t = 2^(s_t - m), s_t = log2(e) scale q . k_t: one pass over the
// tokens with the running maximum m and sum, for any m the same o, so pieces of a row join.
//
// Every cached byte is read once, for the query heads that share it (up to 16), so the bound
// is HBM; of one request alone, latency.  The work is cut by length: a unit is a tile
// of 16 to 64 tokens for each wave of a block, of one (row, kv head), the units of
// all rows stand in one line, and each resident block takes an equal piece of it,
// whatever the rows' lengths are.  A piece that does not hold a whole (row, kv head) leaves
// its unnormalised output, maximum and sum in the workspace, and a second kernel joins those,
// in an order that the lengths alone decide.  (One row alone is cut the same way for each length, with
// pieces that may be empty.)  Where rows cannot be long (a short table, or a window), a
// block takes a whole (row, kv head) instead, and the call is one launch.
//
// Inside a block every wave walks tiles of its own with a running maximum and sum, and
// takes its operands from global memory straight into the matrix instructions' registers:
//  - scores S^T = K Q^T: a lane's 16 bytes of a K row are its operand as they
//    are.  Up to 16 query heads are the columns; unused ones are zero.
//  - output O^T = V^T P^T: a lane of the scores' result holds head lane % 16 and
//    tokens 4 (lane / 16) + {0..3} (+ 16), and that is the lane's share of P^T as an
//    operand if the contraction takes the tokens in that order.  So each lane loads
//    those V rows (its own 8 or 4 dims of them), and transposes them in registers
//    with byte permutations.  Nothing passes through LDS before a piece's end.
//  - the result's columns are heads too, so the running maximum and sum that scale
//    it are the lane's own.
// 8-bit elements widen to bf16 exactly.  Scores, maxima, sums and outputs are fp32.
//
// Measured (both kernels): 64 rows of up to 8192 tokens, 32 + 8 heads of 128, bf16, 1.06 GB of
// cache 205 us (5.2 TB/s; the counters show those bytes fetched and no others); 16 rows of 65536,
// 64 + 8 heads of 128, 8 bits, 2.15 GB 370 us (5.8 TB/s); 48 rows of up to 5000 tokens, 5 + 1
// heads of 256, fp32, 234 MB 62 us (3.8 TB/s, 6 of it the join); one row of 2047 tokens 9.9 us, two
// launches that each wait for a few loads in a chain (lengths, pages, K, V).
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

constexpr int kNT = 256;            // threads of the joining kernel's blocks
constexpr int kHeads = 16;          // query heads of a pass
constexpr int kCUs = 256;

enum { KBF16, KF8, KF32 };

struct Kp {
    const char *q; const char *k; const char *v; const int32_t *table; const int32_t *lens; char *o; float *lse;
    int32_t *start;                 // units before each row (batch + 1)
    float *part;                    // unjoined outputs: (2 blocks, heads of a pass, d)
    float *ml;                      // and their maxima and sums: (2 blocks, heads of a pass, 2)
    int64_t table_stride, q_sr, q_sh, c_sh;    // q and cache strides in bytes
    uint32_t c_sp16, c_st16;        // cache strides of page and token in 16 bytes
    int batch, n_heads, n_kv, group, passes, gmax;   // group: query heads a kv head; passes of gmax <= 16 of them
    int d, n_pages, page_size, max_len, window, unit, unit_lg;
    int wh_lg;                      // 2^wh_lg kv heads side by side (worker_of)
    bool whole;                     // a block for each (row, kv head, pass), and nothing to join
    int fixed;                      // > 0: one row, of which each (kv head, pass) has as many pieces, empty ones too
    float scale2, v_scale;          // scale2: score -> log2 units
};

// The tokens of a row: [lo, hi), in `units` units
struct Span { int lo, hi, units; };
__device__ __forceinline__ Span span_of(const Kp &a, int len) {
    Span s;
    s.hi = min(max(len, 0), a.max_len);
    s.lo = a.window > 0 ? max(0, s.hi - a.window) : 0;
    s.units = (s.hi - s.lo + a.unit - 1) >> a.unit_lg;
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
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp_i(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true); }
// inclusive sums over a wave: within rows of 16 lanes, then the rows' last lanes onward
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp_i<0x111>(v);
    v += dpp_i<0x112>(v);
    v += dpp_i<0x114>(v);
    v += dpp_i<0x118>(v);
    v += dpp_i<0x142, 0xa>(v);
    v += dpp_i<0x143, 0xc>(v);
    return v;
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

// waves on one of a compute unit's 4 SIMDs that the work is cut for, for heads of up to dp (why: Tile::PER_SIMD)
constexpr int per_simd(int dp) { return dp <= 64 ? 3 : dp <= 128 ? 2 : 1; }
// One (cache type, padded head size): register shapes of a tile
template <int CT, int DP, int W> struct Tile {
    static constexpr int E = CT == KF32 ? 4 : CT == KBF16 ? 2 : 1;
    // tokens: 4 to 16 KiB of K (and of V), 8 most often, that a wave has on its way at any time.  (8-bit heads of
    // 256 in tiles of 64 and of 32 tokens: 1 row of 600 15.8 and 11.9 us, 78 rows of up to 600 26.4 and 19.1, 10 of
    // 16000 73.3 and 76.0.)
    static constexpr int NT = CT == KF32 ? (DP <= 64 ? 32 : 16) : CT == KBF16 ? (DP <= 64 ? 64 : 32) : DP > 128 ? 32 : 64;
    static constexpr int SUB = NT / 16;                        // 16-token blocks of scores
    static constexpr int KD = 16 / E;                          // dims of a 16-byte load of K
    static constexpr int KC = DP / (4 * KD);                   // loads of a K row (four lanes each)
    static constexpr int VD = CT == KF32 || DP % 128 ? 4 : 8;  // dims of a lane's load of V
    static constexpr int VB = DP / (16 * VD);                  // loads of a V row (16 lanes each)
    static constexpr int VW = VD * E / 4;                      // dwords of one
    static constexpr int VR = NT / 4;                          // V rows of a lane
    static constexpr int QW = CT == KF8 ? 2 : 1;               // operands of q to a K load
    static constexpr int UNIT = W * NT;
    // blocks of a compute unit that the work is cut for, by the registers of a tile's K, V and output (and of q,
    // which waits in LDS where those leave it no room).
    //  - Up to 64: 3 waves a SIMD, at most 168 registers; fp32 and four-wave bf16 kernels spill 12 to 20 bytes a lane
    //    for it.  8 kv heads of 64, 16000 tokens each, us on 2 and on 3: 8 bits 222, 201; bf16 411, 360; fp32 713, 675.
    //  - Up to 128: 2.  3 spill: 64 rows of up to 16000 tokens, 8 kv heads in 8 bits 228 us on 2 and 234 on 3, of up
    //    to 2000 32 and 41; bf16 374 and 375; 59 and 60.
    //  - Above: 1.  fp32 heads of 256 would spill 250 bytes on 2 (118 us against 58), bf16 ones 170.  8-bit heads, and
    //    bf16 ones of up to 192, have room for 2 as they are compiled (202 to 256 registers), so a second block may
    //    well run beside the first, but twice the pieces gain as often as they lose: us on 1 and on 2, 8-bit heads of
    //    256 (4 kv heads), 1 row of 16000 tokens 16.5, 18.8; 78 rows of 3000 104, 108; 256 of them 290, 272; bf16
    //    heads of 192 (3 kv heads), 78 rows of 600 tokens 21.8, 31.0; 10 rows of 16000 73.7, 77.0; 8-bit ones of 192
    //    (4 kv heads), 10 rows of 3000 22.2, 21.0, 256 rows of 600 46.6, 51.6.
    static constexpr int PER_SIMD = per_simd(DP);
    static constexpr int RES = PER_SIMD * 4 / W;
    static constexpr bool QLDS = DP > 128;
    static constexpr uint64_t ALL = NT == 64 ? ~uint64_t(0) : (uint64_t(1) << NT) - 1;
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

template <int CT, int DP> struct KRows { u32x4 r[Tile<CT, DP, 1>::SUB][Tile<CT, DP, 1>::KC]; };
// K rows of a tile: lane (grp, col) takes dims grp * KD (+ 4 KD c) of tokens col (+ 16)
template <int CT, int DP, bool EXACT>
__device__ __forceinline__ void load_k(KRows<CT, DP> &kf, const char *kb, uint32_t off, int col, int grp, int d) {
    using T = Tile<CT, DP, 1>;
#pragma unroll
    for (int s = 0; s < T::SUB; ++s) {
        const char *p = kb + (uint64_t)(uint32_t)__shfl((int)off, 16 * s + col) * 16;
#pragma unroll
        for (int c = 0; c < T::KC; ++c) {
            // past headdim: the row's own first dims, and zero instead
            const bool in = EXACT || (c * 4 + grp) * T::KD < d;
            const u32x4 x = *(const u32x4 *)(p + (in ? c * 64 : -grp * 16));
            kf.r[s][c] = in ? x : (u32x4){0, 0, 0, 0};
        }
    }
}

// 2^lg kv heads side by side take the same tokens at the same time, on blocks of one XCD
// (blocks go round the 8 of them): where a row of the cache holds the heads next to
// each other and one head's part of it does not fill whole cache lines, the lines that
// two heads share then come from that XCD's L2 for the second of them.  (32 rows of up to 8192
// tokens, 8 kv heads: 8-bit heads of 64 53.5 us alone, 40.7 side by side; bf16 heads of 80 49.9 and 44.8.
// Where a head's part is whole lines, bf16 heads of 128 lose 2%; but with one wave a SIMD,
// heads of 192 and 256, all gain 5 to 18%.)  Of 8 heads instead of 4 nothing more comes.
__device__ __forceinline__ int worker_of(int blk, int lg) { return (blk >> (3 + lg)) * 8 + (blk & 7); }
__device__ __forceinline__ int side_of(int blk, int lg) { return (blk >> 3) & ((1 << lg) - 1); }
__device__ __forceinline__ int block_of(int worker, int side, int lg) {
    return lg == 0 ? worker : (((worker >> 3) << lg) + side) * 8 + (worker & 7);
}

template <int CT, int DP, bool EXACT, int W>      // EXACT: headdim == DP; W: waves of a block
__global__ void __launch_bounds__(W * 64, (Tile<CT, DP, W>::PER_SIMD)) paged_attn_kernel(Kp a) {
    using T = Tile<CT, DP, W>;
    constexpr int VD = T::VD, VB = T::VB;
    extern __shared__ float lds[];          // q, and at a piece's end the waves' outputs
    u32x4 *q_lds = (u32x4 *)lds;
    __shared__ int scan[W], found[3];
    __shared__ float wave_m[W][kHeads], wave_l[W][kHeads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 15, grp = lane >> 4;

    // ---- this block's piece [u, u_end) of the line of units, and the row that u is in
    const int per = (a.n_kv >> a.wh_lg) * a.passes;      // (kv heads side by side, pass) of a row
    const int blk = worker_of(blockIdx.x, a.wh_lg), side = side_of(blockIdx.x, a.wh_lg);
    int units = 0, u, u_end, row, row_u, row_len;
    if (a.whole) {                          // the units of its own row alone, from 0 on
        row = (int)((uint32_t)blk / (uint32_t)per);
        if (row >= a.batch) return;
        const int hp = blk - row * per;
        row_u = 0;
        row_len = a.lens[row];
        units = span_of(a, row_len).units;
        u = hp * units;
        u_end = u + units;
        if (units == 0) {                   // no token: o = 0, lse = -inf
            const int kvs = hp / a.passes, pass = hp - kvs * a.passes, kv = (kvs << a.wh_lg) + side;
            const int nh = min(a.gmax, a.group - pass * a.gmax);
            const int64_t h = (int64_t)row * a.n_heads + kv * a.group + pass * a.gmax;
            constexpr int OE = CT == KF32 ? 4 : 2;
            for (int i = tid; i < nh * a.d * OE / 16; i += W * 64) *(u32x4 *)(a.o + h * a.d * OE + i * 16) = (u32x4){0, 0, 0, 0};
            if (a.lse && tid < nh) a.lse[h + tid] = -INFINITY;
            return;
        }
    } else if (a.fixed) {
        const int hp = blk / a.fixed, i = blk - hp * a.fixed;
        if (hp >= per) return;
        row = row_u = 0;
        row_len = a.lens[0];
        units = span_of(a, row_len).units;
        u = hp * units + (int)((int64_t)i * units / a.fixed);
        u_end = hp * units + (int)((int64_t)(i + 1) * units / a.fixed);
        if (u >= u_end) {                   // weighs nothing
            if (tid < a.gmax) *(float2 *)(a.ml + ((int64_t)2 * blockIdx.x * a.gmax + tid) * 2) = make_float2(-INFINITY, 0.0f);
            return;
        }
    } else if (a.batch <= 64) {                    // each wave for itself: row `lane`
        const int len = lane < a.batch ? a.lens[lane] : 0, own_units = span_of(a, len).units * per;
        const int upto = wave_scan(own_units), before = upto - own_units;
        units = __builtin_amdgcn_readlane(upto, 63);
        if (blockIdx.x == 0 && wave == 0) {
            if (lane < a.batch) a.start[lane] = before;
            if (lane == 0) a.start[a.batch] = units;
        }
        const int blocks = min((int)gridDim.x >> a.wh_lg, units);
        if (blk >= blocks) return;
        u = (int)((int64_t)blk * units / blocks);
        u_end = (int)((int64_t)(blk + 1) * units / blocks);
        row = __builtin_ctzll(__ballot(u >= before && u < upto));
        row_u = __builtin_amdgcn_readlane(before, row);
        row_len = __builtin_amdgcn_readlane(len, row);
    } else {                                // a thread's rows: [r0, r1)
        const int mine = (a.batch + W * 64 - 1) / (W * 64), r0 = tid * mine, r1 = min(r0 + mine, a.batch);
        int own_units = 0;
        for (int r = r0; r < r1; ++r) own_units += span_of(a, a.lens[r]).units * per;
        int before = wave_scan(own_units);
        if (lane == 63) scan[wave] = before;
        __syncthreads();
        before -= own_units;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            before += w < wave ? scan[w] : 0;
            units += scan[w];
        }
        const int blocks = min((int)gridDim.x >> a.wh_lg, units);
        if (blockIdx.x > 0 && blk >= blocks) return;
        u = blocks ? (int)((int64_t)blk * units / blocks) : 0;
        u_end = blocks ? (int)((int64_t)(blk + 1) * units / blocks) : 0;
        if (blockIdx.x == 0 || (u >= before && u < before + own_units)) {
            for (int r = r0; r < r1; ++r) {
                const int len = a.lens[r], n = span_of(a, len).units * per;
                if (u >= before && u < before + n) { found[0] = r; found[1] = before; found[2] = len; }
                if (blockIdx.x == 0) a.start[r] = before;
                before += n;
            }
        }
        if (blockIdx.x == 0 && tid == 0) a.start[a.batch] = units;
        __syncthreads();
        if (u >= u_end) return;
        row = found[0];
        row_u = found[1];
        row_len = found[2];
    }
    Span sp = span_of(a, row_len);

    while (u < u_end) {
        while (u >= row_u + sp.units * per) {
            row_u += sp.units * per;
            sp = span_of(a, a.lens[++row]);
        }
        const int at = u - row_u, hp = at / sp.units, first = at - hp * sp.units;
        const int last = min(sp.units, first + (u_end - u));          // units [first, last) of this head
        const int kvs = hp / a.passes, pass = hp - kvs * a.passes, kv = (kvs << a.wh_lg) + side;
        const int nh = min(a.gmax, a.group - pass * a.gmax);          // query heads of this pass
        const int h0 = kv * a.group + pass * a.gmax;
        u += last - first;

        const char *kb = a.k + kv * a.c_sh + grp * 16, *vb = a.v + kv * a.c_sh;
        const int32_t *table = a.table + row * a.table_stride;
        const int t_end = min(sp.hi, sp.lo + last * T::UNIT);
        int t0 = sp.lo + first * T::UNIT + wave * T::NT;

        // A lane's token of a tile: its page (-1: not the row's), and its place in the cache
        // in 16 bytes.  Tokens that are not the row's read the cache's first row, and are masked.
        auto page_of = [&](int tile) {
            const int t = tile + (lane & (T::NT - 1));
            return t < sp.hi && tile < t_end ? table[(uint32_t)t / (uint32_t)a.page_size] : -1;
        };
        auto place_of = [&](int tile, int page) {
            const uint32_t t = (uint32_t)(tile + (lane & (T::NT - 1)));
            return (uint32_t)page < (uint32_t)a.n_pages ? (uint32_t)page * a.c_sp16 + t % (uint32_t)a.page_size * a.c_st16 : 0u;
        };
        auto tokens_of = [&](int page) {
            return (uint64_t)__ballot((uint32_t)page < (uint32_t)a.n_pages) & T::ALL;
        };
        // The pipeline: while a tile's scores are formed its V rows are on their way, while its
        // output is, the next tile's K rows; the page after that is asked for a tile earlier.
        int page = page_of(t0);
        uint64_t ok = tokens_of(page);
        uint32_t off = place_of(t0, page);
        KRows<CT, DP> kf;
        load_k<CT, DP, EXACT>(kf, kb, off, col, grp, a.d);
        page = page_of(t0 + T::UNIT);

        // q, as the scores' second operand
        u32x4 qf[T::QLDS ? 1 : T::KC * T::QW];
        if (T::QLDS) __syncthreads();        // readers of the piece before
#pragma unroll
        for (int i = 0; i < T::KC * T::QW; ++i) {
            if (T::QLDS && i % W != wave) continue;
            const int dim = i / T::QW * 4 * T::KD + grp * T::KD + i % T::QW * 8;
            u32x4 x = {0, 0, 0, 0};
            if (col < nh && (EXACT || dim < a.d))
                x = *(const u32x4 *)(a.q + row * a.q_sr + (h0 + col) * a.q_sh + dim * (CT == KF32 ? 4 : 2));
            if constexpr (T::QLDS) q_lds[i * 64 + lane] = x;
            else qf[i] = x;
        }
        if (T::QLDS) __syncthreads();

        float m = -INFINITY, l = 0.0f;       // of head col; l over this lane's tokens only
        f32x4 acc[VB][VD];
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
            for (int i = 0; i < VD; ++i) acc[b][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

        for (; t0 < t_end; t0 += T::UNIT) {
            const bool full = ok == T::ALL;
            Words<T::VW> vf[T::VR][VB];
#pragma unroll
            for (int j = 0; j < T::VR; ++j) {
                const int tok = (j >> 2) * 16 + grp * 4 + (j & 3);
                const char *p = vb + (uint64_t)(uint32_t)__shfl((int)off, tok) * 16;
#pragma unroll
                for (int b = 0; b < VB; ++b) {       // past headdim: the row's first dims, in rows of the result that are not kept
                    const int dim = (b * 16 + col) * VD;
                    vf[j][b] = ld_words<T::VW>(p + (EXACT || dim < a.d ? dim * T::E : 0));
                }
            }

            f32x4 s[T::SUB];
#pragma unroll
            for (int i = 0; i < T::SUB; ++i) s[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < T::KC; ++c) {
                u32x4 q[T::QW];
#pragma unroll
                for (int w = 0; w < T::QW; ++w) {
                    if constexpr (T::QLDS) q[w] = q_lds[(c * T::QW + w) * 64 + lane];
                    else q[w] = qf[c * T::QW + w];
                }
#pragma unroll
                for (int i = 0; i < T::SUB; ++i) {
                    const u32x4 k = kf.r[i][c];
                    if constexpr (CT == KBF16) {
                        s[i] = mfma_bf16(k, q[0], s[i]);
                    } else if constexpr (CT == KF8) {
                        const u32x4 k0 = {widen<false>(k[0]), widen<true>(k[0]), widen<false>(k[1]), widen<true>(k[1])};
                        const u32x4 k1 = {widen<false>(k[2]), widen<true>(k[2]), widen<false>(k[3]), widen<true>(k[3])};
                        s[i] = mfma_bf16(k0, q[0], s[i]);
                        s[i] = mfma_bf16(k1, q[T::QW - 1], s[i]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(q[0][e]), s[i], 0, 0, 0);
                    }
                }
            }
            float x[T::VR], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < T::VR; ++j) x[j] = s[j >> 2][j & 3] * a.scale2;
            if (!full) {                     // no weight, and not 0 * what stands in a row that is not the request's
                const uint32_t bits[2] = {(uint32_t)ok >> (grp * 4), (uint32_t)(ok >> 32) >> (grp * 4)};
#pragma unroll
                for (int j = 0; j < T::VR; ++j) {
                    const bool in = bits[j >> 3] >> ((j >> 2 & 1) * 16 + (j & 3)) & 1;
                    x[j] = in ? x[j] : -INFINITY;
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int w = 0; w < T::VW; ++w) vf[j][b].w[w] = in ? vf[j][b].w[w] : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < T::VR; ++j) top = fmaxf(top, x[j]);
            // the next tile's K
            ok = tokens_of(page);
            off = place_of(t0 + T::UNIT, page);
            if (t0 + T::UNIT < t_end) load_k<CT, DP, EXACT>(kf, kb, off, col, grp, a.d);
            page = page_of(t0 + 2 * T::UNIT);

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
                for (int j = 0; j < T::VR; ++j)
#pragma unroll
                    for (int b = 0; b < VB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[j][b].w[i]), x[j], acc[b][i], 0, 0, 0);
            } else {
                // p as the sum of three bf16 values, all its 24 bits.  (Two keep 16 and more: outputs a few 1e-6 off before
                // their rounding.  64 rows of up to 8192 tokens, bf16 204.4 us with two, 205.2 with three; 16 of 65536 in
                // 8 bits 368.1 and 370.0; one of 2047 9.88 and 9.96.)
#pragma unroll
                for (int g = 0; g < T::VR; g += 8) {     // 32 tokens at a time
                    u32x4 ph, pm, pl;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ph[j] = pack_bf16(x[g + 2 * j], x[g + 2 * j + 1]);
                        const float r0 = x[g + 2 * j] - lo_f(ph[j]), r1 = x[g + 2 * j + 1] - hi_f(ph[j]);
                        pm[j] = pack_bf16(r0, r1);
                        pl[j] = pack_bf16(r0 - lo_f(pm[j]), r1 - hi_f(pm[j]));
                    }
#pragma unroll
                    for (int b = 0; b < VB; ++b) {
                        if constexpr (CT == KBF16) {
#pragma unroll
                            for (int i = 0; i < VD; ++i) {
                                u32x4 vt;
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    vt[j] = perm(vf[g + 2 * j + 1][b].w[i / 2], vf[g + 2 * j][b].w[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
                                acc[b][i] = mfma_bf16(vt, ph, acc[b][i]);
                                acc[b][i] = mfma_bf16(vt, pm, acc[b][i]);
                                acc[b][i] = mfma_bf16(vt, pl, acc[b][i]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < VD; i += 2) {
                                u32x4 v0, v1;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint32_t w = perm(vf[g + 2 * j + 1][b].w[i / 4], vf[g + 2 * j][b].w[i / 4], i & 2 ? 0x07030602u : 0x05010400u);
                                    v0[j] = widen<false>(w);
                                    v1[j] = widen<true>(w);
                                }
                                acc[b][i] = mfma_bf16(v0, ph, acc[b][i]);
                                acc[b][i] = mfma_bf16(v0, pm, acc[b][i]);
                                acc[b][i] = mfma_bf16(v0, pl, acc[b][i]);
                                acc[b][i + 1] = mfma_bf16(v1, ph, acc[b][i + 1]);
                                acc[b][i + 1] = mfma_bf16(v1, pm, acc[b][i + 1]);
                                acc[b][i + 1] = mfma_bf16(v1, pl, acc[b][i + 1]);
                            }
                        }
                    }
                }
            }
        }

        // ---- join the block's waves
        l = head_sum(l);
        __syncthreads();                     // readers of the segment before
        if (grp == 0) { wave_m[wave][col] = m; wave_l[wave][col] = l; }
        __syncthreads();
        float top = wave_m[0][col];
#pragma unroll
        for (int w = 1; w < W; ++w) top = fmaxf(top, wave_m[w][col]);
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
        const bool whole = first == 0 && last == sp.units && !a.fixed;
        const int slot = 2 * (int)blockIdx.x + (first == 0 && !a.fixed ? 1 : 0);
        const int d4 = a.d / 4;
        for (int i = tid; i < nh * d4; i += W * 64) {
            const int h = i / d4, e = (i - h * d4) * 4;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            float ls = 0.0f, mt = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                v += *(const f32x4 *)(lds + (w * a.gmax + h) * PITCH + e);
                mt = fmaxf(mt, wave_m[w][h]);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) ls += wave_l[w][h] * (mt == -INFINITY ? 0.0f : exp2_fast(wave_m[w][h] - mt));
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

// Joins the pieces of a (row, query head): piece i's share is scaled by
// 2^(m_i - max m).  Rows without tokens get o = 0, lse = -inf here.  A block has HB heads of
// a row.  Where a head has few pieces, a wave joins it alone; else the whole block does,
// d / gridDim.z dims of it, head after head.
template <bool BF16, int HB>
__global__ void __launch_bounds__(kNT) paged_attn_join_kernel(Kp a, int grid) {
    __shared__ f32x4 out[kNT];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.n_kv >> a.wh_lg) * a.passes;
    const int64_t total = a.fixed ? 1 : a.start[a.batch];
    const int row_u = a.fixed ? 0 : a.start[row], nu = a.fixed ? 1 : (a.start[row + 1] - row_u) / per;
    const int64_t blocks = min((int64_t)(grid >> a.wh_lg), total);
    const int d4 = a.d / 4;
    auto store = [&](int h, int e, f32x4 v) {
        const int64_t to = ((int64_t)row * a.n_heads + h) * a.d + e;
        if constexpr (BF16) *(uint2 *)(a.o + to * 2) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else *(f32x4 *)(a.o + to * 4) = v;
    };
    // The threads of a head: slice sl of its pieces, dims e..e+3; the caller adds up the slices.
    // Every wave forms the maximum and the sum for itself: lane i has pieces i, i + 64, ...
    // n: pieces (1: the head was written whole); scale, lse: of the sum
    struct Joined { f32x4 v; int n; float scale, lse; };
    auto join = [&](int h, int sl, int slices, int e) {
        Joined r = {{0.0f, 0.0f, 0.0f, 0.0f}, 1, 0.0f, -INFINITY};
        const int kv = h / a.group, side = kv & ((1 << a.wh_lg) - 1), pass = (h - kv * a.group) / a.gmax;
        const int hh = h - kv * a.group - pass * a.gmax;
        // the blocks whose pieces hold this head's first and last unit
        const int hp = (kv >> a.wh_lg) * a.passes + pass;
        const int64_t u0 = row_u + (int64_t)hp * nu;
        const int b0 = a.fixed ? hp * a.fixed : (int)(((u0 + 1) * blocks - 1) / total);
        const int n = a.fixed ? a.fixed : (int)(((u0 + nu) * blocks - 1) / total) - b0 + 1;
        if (n == 1) return r;
        r.n = n;
        // the first block began this head (its second place); the others go on with it (their first)
        auto place = [&](int i) { return ((int64_t)block_of(b0 + i, side, a.wh_lg) * 2 + (i == 0 && !a.fixed ? 1 : 0)) * a.gmax + hh; };
        f32x4 part0 = r.v, part1 = r.v;
        // the first two shares of a slice need not wait for the maximum
        const bool in0 = sl < slices && sl < n, in1 = sl < slices && sl + slices < n;
        if (in0) part0 = *(const f32x4 *)(a.part + place(sl) * a.d + e);
        if (in1) part1 = *(const f32x4 *)(a.part + place(sl + slices) * a.d + e);
        float2 own = make_float2(-INFINITY, 0.0f);
        if (lane < n) own = *(const float2 *)(a.ml + place(lane) * 2);
        float m = own.x;
        for (int i = lane + 64; i < n; i += 64) m = fmaxf(m, a.ml[place(i) * 2]);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        m = m == -INFINITY ? 0.0f : m;
        const float scale = exp2_fast(own.x - m);
        float l = own.y * scale;
        for (int i = lane + 64; i < n; i += 64) {
            const float2 w = *(const float2 *)(a.ml + place(i) * 2);
            l += w.y * exp2_fast(w.x - m);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
        const float s0 = __shfl(scale, sl & 63), s1 = __shfl(scale, (sl + slices) & 63);
        // (what weighs nothing may never have been written)
        auto add = [&](f32x4 part, float w) { r.v += w > 0.0f ? part * w : (f32x4){0.0f, 0.0f, 0.0f, 0.0f}; };
        if (in0) add(part0, sl < 64 ? s0 : exp2_fast(a.ml[place(sl) * 2] - m));
        if (in1) add(part1, sl + slices < 64 ? s1 : exp2_fast(a.ml[place(sl + slices) * 2] - m));
        if (sl < slices) {
#pragma unroll 4
            for (int i = sl + 2 * slices; i < n; i += slices)
                add(*(const f32x4 *)(a.part + place(i) * a.d + e), exp2_fast(a.ml[place(i) * 2] - m));
        }
        r.scale = l > 0.0f || l != l ? a.v_scale / l : 0.0f;
        r.lse = m * kLn2 + logf(l);
        return r;
    };
    const int h0 = (int)blockIdx.y * HB, h1 = min(h0 + HB, a.n_heads);
    // (a head's pieces lie within nu units, a block's share is total / blocks of them)
    if (HB > 1 && (nu == 0 || nu * blocks / total + 2 <= 16)) {
        const int h = h0 + wave, slices = 64 / d4, sl = lane / d4, e = (lane - sl * d4) * 4;
        if (h >= h1) return;
        Joined r = {{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0.0f, -INFINITY};
        if (nu > 0) r = join(h, sl, slices, e);
        if (r.n == 1) return;
        f32x4 v = r.v;
        for (int s = 1; s < min(slices, r.n); ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += __shfl(r.v[i], lane + s * d4);
        if (sl == 0) store(h, e, v * r.scale);
        if (lane == 0 && a.lse) a.lse[(int64_t)row * a.n_heads + h] = r.lse;
        return;
    }
    const int cols = d4 / gridDim.z, slices = kNT / cols, sl = tid / cols, e = ((int)blockIdx.z * cols + tid - sl * cols) * 4;
    for (int h = h0; h < h1; ++h) {
        Joined r = {{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0.0f, -INFINITY};
        if (nu > 0) r = join(h, sl, slices, e);
        if (r.n == 1) continue;                  // the same in the whole block
        out[tid] = r.v;
        __syncthreads();
        if (sl == 0) {
            f32x4 v = r.v;
            for (int s = 1; s < min(slices, r.n); ++s) v += out[s * cols + tid];
            store(h, e, v * r.scale);
        }
        if (tid == 0 && blockIdx.z == 0 && a.lse) a.lse[(int64_t)row * a.n_heads + h] = r.lse;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host ----
int64_t passes_of(int64_t group) { return (group + kHeads - 1) / kHeads; }
int64_t align16(int64_t n) { return (n + 15) & ~int64_t(15); }

// (row, kv head)s that occupy the chip with a wave each, by the waves that the work is cut for
int64_t waves_of(int64_t d) { return (d <= 128 ? 2 : 1) * 4 * kCUs; }

template <int CT, int DP, bool EXACT, int W>
hipError_t go_w(Kp &k, int &grid, hipStream_t stream) {
    using T = Tile<CT, DP, W>;
    k.unit = T::UNIT;
    k.unit_lg = __builtin_ctz(T::UNIT);
    while (k.wh_lg < 2 && (T::PER_SIMD == 1 || (k.c_sh << k.wh_lg) % 128 != 0) && (k.n_kv >> k.wh_lg) % 2 == 0) ++k.wh_lg;
    // the blocks that are resident at once, or one a unit if there are fewer; whole groups of heads side by side
    const double units = (double)k.batch * k.n_kv * k.passes * ((k.max_len + T::UNIT - 1) / T::UNIT);
    grid = k.whole ? k.batch * k.n_kv * k.passes : (int)std::max(1.0, std::min(units, (double)(T::RES * kCUs)));
    const int group = 8 << k.wh_lg, per = (k.n_kv >> k.wh_lg) * k.passes;
    // One row is cut evenly by the sizes alone, and its pieces join without a look at its length: 32 + 8
    // heads of 128, bf16, 1000 tokens 10.2 us by lengths, 9.7 by sizes; 32000 34.1 and 33.6
    if (k.batch == 1 && !k.whole && grid >> k.wh_lg >= 2 * per) k.fixed = (grid >> k.wh_lg) / per;
    if (k.wh_lg > 0) grid = (grid + group - 1) / group * group;
    const size_t lds = std::max((size_t)W * k.gmax * (DP + 4) * sizeof(float), T::QLDS ? (size_t)T::KC * T::QW * 1024 : 0);
    if (lds > 32 * 1024) {               // more than a block has unasked, from 64 KiB on
        const hipError_t e = hipFuncSetAttribute((const void *)paged_attn_kernel<CT, DP, EXACT, W>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_attn_kernel<CT, DP, EXACT, W>), dim3((unsigned)grid), dim3(W * 64), lds, stream, k);
    return hipGetLastError();
}
// Blocks of one wave or of four, and whole (row, kv head)s or equal pieces.  A whole one saves the second
// launch and the search for a piece, and makes a block work for as long as its row is, so it is taken
// where rows reach few tiles, more of them if there are many rows to even the blocks out.  One wave
// takes a head where every wave of the chip has one or nearly so.  us, bf16 heads of 128, 8 kv heads, all rows
// of the length (whole in one wave, whole in four, pieces):
//   1 row of 32 tokens 5.7, 5.7, 8.2; 300: 12.0, 7.7, 9.6; 600: 19.8, 10.5, 10.0; 2400: 67, 28, 10.6
//   64 rows of 128 tokens 10.3, 9.2, 12.1; 600: 36.9, 29.6, 32.9; up to 1200: 59, 39, 39; up to 2400: 118, 78, 71
//   256 rows of 128 tokens 24.4, 29.0, 30.2; up to 300: 32.8, 38.9, 43.5; up to 1200: 132, 130, 136; up to 2400: 255, 248, 244
// and of 4 and 3 kv heads in 8 and 32 bits, heads of 64 and 256 the same way: above 128, with more heads than a
// quarter of waves_of, 78 rows of 90 tokens, 4 heads of 256 in 8 bits 11.7, 15.7; 150 rows, 2 heads of 256 in bf16
// 12.1, 16.7 (one block of four a compute unit in bf16; in 8 bits two fit, and four waves still idle on rows of 3
// tiles).  In pieces, four waves share the tokens of one, and fewer pieces are left to join; one row of 100000
// tokens 32.8 us by waves, 23.1 by fours.  (Taken with weights in two bf16 parts; three are up to 3% slower either way.)
template <int CT, int DP, bool EXACT>
hipError_t go(Kp &k, int &grid, hipStream_t stream) {
    using T = Tile<CT, DP, 1>;
    const int64_t heads = (int64_t)k.batch * k.n_kv * k.passes, waves = waves_of(DP);
    const int tiles = ((k.window > 0 ? k.window : k.max_len) + T::NT - 1) / T::NT;
    const bool by_wave = tiles <= 1 || (heads > waves / 4 && tiles <= (heads >= waves ? 32 : heads >= waves / 2 ? 16 : 8));
    const bool by_block = tiles <= (heads >= waves / 4 ? 40 : heads >= waves / 8 ? 20 : 12);
    k.whole = (by_wave || by_block) && heads < (1 << 22);      // (a grid's threads are counted in 32 bits)
    return (k.whole ? by_wave : heads >= waves) ? go_w<CT, DP, EXACT, 1>(k, grid, stream) : go_w<CT, DP, EXACT, 4>(k, grid, stream);
}
template <int CT, int DP>
hipError_t go_d(Kp &k, int &grid, hipStream_t stream) {
    return k.d == DP ? go<CT, DP, true>(k, grid, stream) : go<CT, DP, false>(k, grid, stream);
}
template <int CT>
hipError_t go_type(Kp &k, int &grid, hipStream_t stream) {
    if (k.d <= 64) return go_d<CT, 64>(k, grid, stream);
    if (k.d <= 128) return go_d<CT, 128>(k, grid, stream);
    if (k.d <= 192) return go_d<CT, 192>(k, grid, stream);
    return go_d<CT, 256>(k, grid, stream);
}

}  // namespace

// (of the smallest unit, a tile of one wave)
double paged_attn_max_units(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t max_pages, int64_t page_size) {
    const double len = (double)max_pages * (double)page_size;
    return (double)batch * (double)n_kv_heads * (double)passes_of(n_heads / n_kv_heads) * (len / 16 + 1.0);
}

// blocks of the largest grid that any cache type gives these sizes
static int64_t most_blocks(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim, int64_t max_pages,
                           int64_t page_size) {
    const bool one = batch * n_kv_heads * passes_of(n_heads / n_kv_heads) >= waves_of(headdim);
    const double units = paged_attn_max_units(batch, n_heads, n_kv_heads, max_pages, page_size) + 32;
    return (int64_t)std::min(units, (double)(per_simd((int)std::min<int64_t>(headdim, 256)) * kCUs * (one ? 4 : 1)));
}

size_t paged_attn_workspace_bytes(int64_t batch, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                  int64_t max_pages, int64_t page_size) {
    const int64_t group = n_heads / n_kv_heads, gmax = std::min<int64_t>(group, kHeads);
    const int64_t places = 2 * most_blocks(batch, n_heads, n_kv_heads, headdim, max_pages, page_size) * gmax;
    return (size_t)(align16((batch + 1) * 4) + align16(places * 8) + places * headdim * 4);
}

hipError_t launch_paged_attn(const PagedAttnArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "paged_attn_kernel";
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    Kp k = {};
    k.q = (const char *)a.q; k.k = (const char *)a.k_cache; k.v = (const char *)a.v_cache;
    k.table = a.block_table; k.lens = a.lens; k.o = (char *)a.o; k.lse = a.lse;
    k.group = (int)(a.n_heads / a.n_kv_heads);
    k.gmax = std::min(k.group, kHeads);
    k.passes = (int)passes_of(k.group);
    char *ws = (char *)a.workspace;
    k.start = (int32_t *)ws; ws += align16((a.batch + 1) * 4);
    k.ml = (float *)ws; ws += align16(2 * most_blocks(a.batch, a.n_heads, a.n_kv_heads, a.headdim, a.max_pages, a.page_size) * k.gmax * 8);
    k.part = (float *)ws;
    k.table_stride = a.table_stride; k.q_sr = a.q_sr * qe; k.q_sh = a.q_sh * qe; k.c_sh = a.c_sh * e;
    k.c_sp16 = (uint32_t)(a.c_sp * e / 16); k.c_st16 = (uint32_t)(a.c_st * e / 16);
    k.batch = (int)a.batch; k.n_heads = (int)a.n_heads; k.n_kv = (int)a.n_kv_heads;
    k.d = a.headdim; k.n_pages = (int)a.n_pages; k.page_size = (int)a.page_size;
    k.max_len = (int)(a.max_pages * a.page_size);
    k.window = a.window > 0 && a.window < k.max_len ? (int)a.window : 0;
    k.scale2 = a.scale * (a.kv_dtype == SSM_KV_F8E4M3 ? a.k_scale : 1.0f) * kLog2e;
    k.v_scale = a.kv_dtype == SSM_KV_F8E4M3 ? a.v_scale : 1.0f;
    int grid = 0;
    const hipError_t rc = a.kv_dtype == SSM_KV_F32 ? go_type<KF32>(k, grid, stream)
                        : a.kv_dtype == SSM_KV_BF16 ? go_type<KBF16>(k, grid, stream)
                                                    : go_type<KF8>(k, grid, stream);
    if (rc != hipSuccess || k.whole) return rc;
    *kernel_name = "paged_attn_join_kernel";
    // Where a head has many pieces, a block joins it, or several of 32 dims each; else its waves a head
    // each.  One row of 100000 tokens 22.7 us with, 46 without the split; 256 rows of up to 60
    // tokens 20.9 us by waves, 32 by blocks; one row of 4096, 32 heads 11.7 us by blocks, 16.2 by waves.
    const int64_t pieces = (grid >> k.wh_lg) / (a.batch * (a.n_kv_heads >> k.wh_lg) * k.passes);
    const int split = pieces >= 64 && a.headdim % 32 == 0 ? a.headdim / 32 : 1, hb = pieces >= 8 ? 1 : 4;
    const dim3 g((unsigned)a.batch, (unsigned)((a.n_heads + hb - 1) / hb), (unsigned)split);
    const bool bf16 = a.kv_dtype != SSM_KV_F32;
    if (hb == 1 && bf16) hipLaunchKernelGGL((paged_attn_join_kernel<true, 1>), g, dim3(kNT), 0, stream, k, grid);
    else if (hb == 1) hipLaunchKernelGGL((paged_attn_join_kernel<false, 1>), g, dim3(kNT), 0, stream, k, grid);
    else if (bf16) hipLaunchKernelGGL((paged_attn_join_kernel<true, 4>), g, dim3(kNT), 0, stream, k, grid);
    else hipLaunchKernelGGL((paged_attn_join_kernel<false, 4>), g, dim3(kNT), 0, stream, k, grid);
    return hipGetLastError();
}

}  // namespace ssm
