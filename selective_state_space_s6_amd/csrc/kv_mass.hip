// kv_mass.hip -- the softmax weight that each cached token gathers from a step's queries
// (ssm_kv_mass_update in include/ssm_longctx.h).
//
// w_j = sum over rows and heads of 2^(log2(e) (scale q . k_j - lse)): given lse, no maximum and no second pass.  log2(e) lse is
// a float and a rest, whose power of two is the column's factor: a multiply-add in place of an addition, and without it
// all weights of a column are off by up to u log2(e) |lse| the same way.
// (row, head) pairs are columns of the matrix products, 16 tokens or more their rows; a lane adds up its columns'
// exponentials, and the 16 lanes of a token are joined once at the end.  Two forms, and in both one writer a token:
//   step: a wave has tiles of 16 to 64 tokens from one line of all requests' tiles, cut into equal pieces, the next
//     tile's keys on their way while one is worked on, and walks the request's columns, 16 at a time.
//     Bound: HBM, the keys.  64 requests of up to 8192 tokens, 8 kv heads of 128, bf16: 176 us for 819 MB, 4.7 TB/s.
//   prompt: a block has 64 tokens, their keys in shared memory, and its 8 waves columns of their own from the first row on
//     that sees the tile; requests go to XCDs in turn.  Bound: the way of q from the L2s, 64 bytes of each of 16 columns a load,
//     beside one exponential a (row, head, token).  4 prompts of up to 2048 tokens, 32 + 8 heads of 128, bf16: 54 us,
//     13.9 GFLOP and 54 million exponentials.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <type_traits>

#include "attn_device.hpp"
#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

constexpr int kW = 4;               // waves of a block that share nothing
constexpr int kShare = 8;           // waves of a block that share their tokens
constexpr int kCUs = 256;

struct Mp {
    const char *q; const char *k; const float *lse; float *mass;
    const int32_t *table; const int32_t *starts; const int32_t *positions; const int32_t *len_old; const int32_t *lens;
    int64_t table_stride, q_sr, q_sh, c_sp, c_st, c_sh;              // q and cache strides in bytes
    int batch, n_tokens, n_heads, n_kv, group, d, n_pages, page_size, row_len, blocks;   // blocks: of a (request, kv head)
    float scale2;
};

template <int CT, int DP> struct MTile {
    static constexpr int E = CT == KF32 ? 4 : CT == KBF16 ? 2 : 1;
    static constexpr int KD = 16 / E, KC = DP / (4 * KD);            // dims of a load of K, loads of a row (four lanes each)
    static constexpr int QW = CT == KF8 ? 2 : 1;                     // operands of q to a load of K
    static constexpr int QR = KC * QW * 4;                           // registers of a column's q
    // a step's tile: 16-token blocks, 8 KiB of keys that a wave has on its way
    static constexpr int SUB = KC <= 2 ? 4 : KC <= 4 ? 2 : 1;
    static constexpr int NT = SUB * 16;
    static constexpr int HELD = KC * SUB * 8 + QR * 2;               // registers of two tiles' keys and columns
    // waves on a SIMD (8-bit keys widen in registers of their own: on three, heads of 128 spilled, 207 us for 64 requests of up
    // to 8192 tokens, 99 on two; 108 on three with tiles of 32 tokens)
    static constexpr int OCC = HELD <= (CT == KF8 ? 64 : 112) ? 3 : HELD <= 192 ? 2 : 1;
    // a prompt's tile, in shared memory, and 16-column groups of a wave in a round
    static constexpr int PSUB = 4, PNT = 64;
    // (two where both fit the registers: of heads of 128 in fp32 and of 256 in bf16 two spilled, 73 us instead of 60 and 229
    // instead of 128; tiles of 128 tokens 66 us for 4 prompts of up to 2048 tokens, 56 with 64, and blocks of 16 columns a wave
    // two a compute unit 86)
    static constexpr int NC = QR <= 24 ? 2 : 1;
};

// A lane's token of a tile
struct Token {
    int page;                       // -1: none
    int64_t at;                     // its place in mass
    uint64_t off;                   // and among the keys, in bytes
};
__device__ __forceinline__ Token token_of(const Mp &a, const PageSize &ps, int r, int g, int tok, int len) {
    Token t;
    const int pj = ps.of(tok), place = ps.place(tok, pj);
    t.page = tok < len ? a.table[(int64_t)r * a.table_stride + pj] : -1;
    if ((uint32_t)t.page >= (uint32_t)a.n_pages) t.page = -1;
    t.at = ((int64_t)max(t.page, 0) * a.n_kv + g) * a.page_size + place;
    t.off = t.page >= 0 ? (uint64_t)t.page * (uint64_t)a.c_sp + (uint64_t)place * (uint64_t)a.c_st : 0;
    return t;
}

// A tile's keys, as the scores' first operand
template <int CT, int DP> struct Keys { u32x4 r[MTile<CT, DP>::SUB][MTile<CT, DP>::KC]; };
template <int CT, int DP, bool EXACT>
__device__ __forceinline__ void load_keys(Keys<CT, DP> &k, const char *kb, uint64_t off, int lane, int d) {
    using T = MTile<CT, DP>;
    const int col = lane & 15, grp = lane >> 4;
#pragma unroll
    for (int s = 0; s < T::SUB; ++s) {
        const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, 16 * s + col), hi = (uint32_t)__shfl((int)(off >> 32), 16 * s + col);
        const char *p = kb + ((uint64_t)hi << 32 | lo) + grp * 16;
#pragma unroll
        for (int c = 0; c < T::KC; ++c) {
            // past headdim: the row's own first dims, and zero instead
            const bool in = EXACT || (c * 4 + grp) * T::KD < d;
            const u32x4 x = *(const u32x4 *)(p + (in ? c * 64 : -grp * 16));
            k.r[s][c] = in ? x : (u32x4){0, 0, 0, 0};
        }
    }
}

// 16 columns of the scores: a lane's part of their queries, the last token that its column sees
// (-1: none), log2(e) lse, and 2^-(what that is short of)
template <int CT, int DP> struct Column {
    u32x4 q[MTile<CT, DP>::KC * MTile<CT, DP>::QW];
    int pos;
    float lse2, rest;
};
template <int CT, int DP, bool EXACT>
__device__ __forceinline__ void load_column(const Mp &a, Column<CT, DP> &x, const char *qp, float lse, int pos, int grp) {
    using T = MTile<CT, DP>;
    x.pos = lse == -INFINITY ? -1 : pos;
    x.lse2 = lse * kLog2e;
    // (log2(e) is kLog2e + 1.925963033e-8; of an infinite lse there is no rest)
    const float low = fmaf(lse, 1.925963033e-8f, fmaf(lse, kLog2e, -x.lse2));
    x.rest = fabsf(lse) < INFINITY ? exp2_fast(-low) : 1.0f;
#pragma unroll
    for (int k = 0; k < T::KC; ++k)
#pragma unroll
        for (int y = 0; y < T::QW; ++y) {
            const int dim = (k * 4 + grp) * T::KD + y * 8;
            u32x4 v = {0, 0, 0, 0};
            if (EXACT || dim < a.d) v = *(const u32x4 *)(qp + k * 64 * T::QW + y * 16);
            x.q[k * T::QW + y] = v;
        }
}

// scores of a 16-token block (its keys in k) and 16 columns
template <int CT, int DP>
__device__ __forceinline__ f32x4 scores(const u32x4 (&k)[MTile<CT, DP>::KC], const Column<CT, DP> &x) {
    using T = MTile<CT, DP>;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < T::KC; ++c) {
        const u32x4 y = k[c];
        if constexpr (CT == KBF16) {
            s = mfma_bf16(y, x.q[c], s);
        } else if constexpr (CT == KF8) {
            const u32x4 k0 = {widen<false>(y[0]), widen<true>(y[0]), widen<false>(y[1]), widen<true>(y[1])};
            const u32x4 k1 = {widen<false>(y[2]), widen<true>(y[2]), widen<false>(y[3]), widen<true>(y[3])};
            s = mfma_bf16(k0, x.q[c * T::QW], s);
            s = mfma_bf16(k1, x.q[c * T::QW + T::QW - 1], s);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y[e]), __uint_as_float(x.q[c][e]), s, 0, 0, 0);
        }
    }
    return s;
}
// adds a column's weights to w; t: the first of the lane's four tokens, ALL: the column sees them all
template <bool ALL>
__device__ __forceinline__ void weigh(float (&w)[4], f32x4 s, float scale2, float lse2, float rest, int t, int pos) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float p = exp2_fast(fmaf(s[e], scale2, -lse2));
        w[e] = fmaf(ALL || t + e <= pos ? p : 0.0f, rest, w[e]);
    }
}

// the 16 columns of each token joined, into sums[token of the tile]
template <int SUB>
__device__ __forceinline__ void join_columns(const float (&w)[SUB][4], float *sums, int lane) {
#pragma unroll
    for (int b = 0; b < SUB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = w[b][e];
            v += dpp_f<0x111>(v);                 // up to each lane of a row of 16
            v += dpp_f<0x112>(v);
            v += dpp_f<0x114>(v);
            v += dpp_f<0x118>(v);
            if ((lane & 15) == 15) sums[b * 16 + (lane >> 4) * 4 + e] = v;
        }
}

// Few columns a request (a decode step): the tiles of all requests and kv heads stand in one line, each
// wave takes an equal piece of it, and has the next keys and columns on their way while it weighs one tile's.
template <int CT, int DP, bool EXACT>
__global__ void __launch_bounds__(kW * 64, (MTile<CT, DP>::OCC)) kv_mass_step_kernel(Mp a) {
    using T = MTile<CT, DP>;
    extern __shared__ int upto[];                 // tiles of the requests up to each
    __shared__ int scan[kW];
    __shared__ float sums[kW][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    const PageSize ps(a.page_size);
    const int mine = (a.batch + kW * 64 - 1) / (kW * 64), r0 = tid * mine, r1 = min(r0 + mine, a.batch);
    int own = 0;
    for (int r = r0; r < r1; ++r) upto[r] = own += (min(max(a.lens[r], 0), a.row_len) + T::NT - 1) / T::NT;
    int before = wave_scan(own);
    if (lane == 63) scan[wave] = before;
    before -= own;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) before += w < wave ? scan[w] : 0;
    for (int r = r0; r < r1; ++r) upto[r] += before;
    __syncthreads();
    const int units = upto[a.batch - 1] * a.n_kv;
    // (a wave's piece is in order, so that it looks a tile up once for all of its kv heads)
    const int64_t wv = (int64_t)blockIdx.x * kW + wave, waves = (int64_t)gridDim.x * kW;
    const int u_end = (int)((wv + 1) * units / waves);
    int u = (int)(wv * units / waves);
    if (u >= u_end) return;
    // A tile: its request, and what does not depend on the kv head.  The next one is asked for a tile ahead.
    struct Tile { int t0, len, s0, cols, page, place, pos; bool kept; };
    int r = 0;                                    // of the tile that is looked up next
    {
        int end = a.batch - 1;                    // the first request with upto > it
        while (r < end) {
            const int mid = (r + end) >> 1;
            if (upto[mid] > u / a.n_kv) end = mid; else r = mid + 1;
        }
    }
    int col_row, col_head;                        // the first 16 columns: row of the request and head
    col_row = col / a.group;
    col_head = col - col_row * a.group;
    auto look_up = [&](int tile) {
        Tile n;
        while (r < a.batch - 1 && upto[r] <= tile) ++r;
        n.t0 = (tile - (r > 0 ? upto[r - 1] : 0)) * T::NT;
        n.len = min(max(a.lens[r], 0), a.row_len);
        n.s0 = min(max(a.starts[r], 0), a.n_tokens);
        n.cols = (min(max(a.starts[r + 1], n.s0), a.n_tokens) - n.s0) * a.group;
        const int t = n.t0 + (lane & (T::NT - 1)), pj = ps.of(t);
        n.place = ps.place(t, pj);
        n.page = t < n.len ? a.table[(int64_t)r * a.table_stride + pj] : -1;
        n.kept = t < a.len_old[r];
        n.pos = col < n.cols ? a.positions[n.s0 + col_row] : -1;
        return n;
    };
    // A (tile, kv head): keys and first columns on their way
    struct Unit { float was; int64_t at; Keys<CT, DP> k; Column<CT, DP> x; };
    auto ask = [&](const Tile &n, int g) {
        Unit x;
        const bool is = (uint32_t)n.page < (uint32_t)a.n_pages;
        x.at = is ? ((int64_t)n.page * a.n_kv + g) * a.page_size + n.place : -1;
        x.was = 0.0f;
        if (is && n.kept) x.was = a.mass[x.at];
        if (n.cols > 0) {
            const bool has = col < n.cols;
            const int64_t t = n.s0 + (has ? col_row : 0), h = (int64_t)g * a.group + (has ? col_head : 0);
            const float lse = a.lse[t * a.n_heads + h];
            load_column<CT, DP, EXACT>(a, x.x, a.q + t * a.q_sr + h * a.q_sh + grp * (CT == KF8 ? 32 : 16), lse, n.pos < n.len ? n.pos : -1, grp);
            const uint64_t off = is ? (uint64_t)n.page * (uint64_t)a.c_sp + (uint64_t)n.place * (uint64_t)a.c_st : 0;
            load_keys<CT, DP, EXACT>(x.k, a.k + (int64_t)g * a.c_sh, off, lane, a.d);
        }
        return x;
    };
    int tile = u / a.n_kv, g = u - tile * a.n_kv;
    const int last = (u_end - 1) / a.n_kv;
    Tile now = look_up(tile), then = now;
    if (tile < last) then = look_up(tile + 1);
    Unit next = ask(now, g);
    for (; u < u_end; ++u) {
        const Tile here = now;
        Unit x = next;
        const int gu = g;
        if (u + 1 < u_end) {
            if (++g == a.n_kv) {
                g = 0;
                ++tile;
                now = then;
                if (tile < last) then = look_up(tile + 1);
            }
            next = ask(now, g);
        }
        float w[T::SUB][4];
#pragma unroll
        for (int s = 0; s < T::SUB; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[s][i] = 0.0f;
        for (int c0 = 0; c0 < here.cols; c0 += 16) {
            if (c0 > 0) {                         // columns behind the first 16: not asked for ahead
                const int c = c0 + col, i = c / a.group;
                const bool is = c < here.cols;
                const int64_t t = here.s0 + (is ? i : 0), h = (int64_t)gu * a.group + (is ? c - i * a.group : 0);
                const int pos = a.positions[t];
                const float lse = a.lse[t * a.n_heads + h];
                load_column<CT, DP, EXACT>(a, x.x, a.q + t * a.q_sr + h * a.q_sh + grp * (CT == KF8 ? 32 : 16), lse,
                                           is && pos < here.len ? pos : -1, grp);
            }
            if (!__any(x.x.pos >= here.t0)) continue;
#pragma unroll
            for (int b = 0; b < T::SUB; ++b) {
                weigh<false>(w[b], scores<CT, DP>(x.k.r[b], x.x), a.scale2, x.x.lse2, x.x.rest, here.t0 + b * 16 + grp * 4, x.x.pos);
                if constexpr (CT == KF8) __builtin_amdgcn_sched_barrier(0);      // (widened keys of one block at a time)
            }
        }
        join_columns<T::SUB>(w, sums[wave], lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float got = sums[wave][lane & (T::NT - 1)];
        if (x.at >= 0 && lane < T::NT) a.mass[x.at] = got + x.was;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Many columns a request (prompts): a block has one tile of keys, in shared memory as the operands that
// they are, and its waves take 16 or 32 columns each in rounds, the next round's columns on their way.  A lane keeps its
// head from round to round.
template <int CT, int DP, bool EXACT>
__global__ void __launch_bounds__(kShare * 64, 2) kv_mass_prompt_kernel(Mp a) {
    using T = MTile<CT, DP>;
    extern __shared__ u32x4 keys[];               // (16-token block, load of a row, lane)
    __shared__ float sums[kShare][T::PNT];
    __shared__ int early;                         // a row before the guessed first one sees a token
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    // Early tiles, which most rows see, first; requests go round the XCDs (as blocks do, 8 of them) and on by one
    // each time, so that no XCD has the long ones alone.
    const int j = blockIdx.x >> 3, q8 = j / a.n_kv, pair = q8 * 8 + ((blockIdx.x + q8) & 7), g = j - q8 * a.n_kv;
    const int blk = pair / a.batch, r = pair - blk * a.batch;
    if (blk >= a.blocks) return;
    const PageSize ps(a.page_size);
    const int len = min(max(a.lens[r], 0), a.row_len), old = a.len_old[r];
    const int s0 = min(max(a.starts[r], 0), a.n_tokens), s1 = min(max(a.starts[r + 1], s0), a.n_tokens);
    // columns of a round: whole rows, so that heads stay (of more heads than columns: one row and a part of its heads
    // each time)
    constexpr int NC = T::NC, COLS = kShare * 16 * NC;
    const int whole = COLS / a.group, step = max(whole, 1), parts = whole > 0 ? 1 : (a.group + COLS - 1) / COLS;
    int crow[NC], head0[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int c = (wave * NC + n) * 16 + col;
        crow[n] = whole > 0 ? c / a.group : 0;
        head0[n] = c - crow[n] * a.group;
    }
    for (int t0 = blk * T::PNT; t0 < len; t0 += a.blocks * T::PNT) {
        const Token tok = token_of(a, ps, r, g, t0 + lane, len);
        // Rows at rising places, as a page step numbers them, see the tile from row b0 on.  Other orders are right too:
        // if a row before it sees a token, all rows are taken.
        int b0 = s0;
        if (s1 > s0) b0 = min(max((int64_t)s0 + t0 - a.positions[s0], (int64_t)s0), (int64_t)s1);
        const char *kb = a.k + (int64_t)g * a.c_sh + grp * 16;
        if (tid == 0) early = 0;
        for (int i = wave; i < T::PSUB * T::KC; i += kShare) {
            const int s = i / T::KC, x = i - s * T::KC;
            const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)tok.off, 16 * s + col), hi = (uint32_t)__shfl((int)(tok.off >> 32), 16 * s + col);
            // past headdim: the row's own first dims, and zero instead
            const bool in = EXACT || (x * 4 + grp) * T::KD < a.d;
            const u32x4 v = *(const u32x4 *)(kb + ((uint64_t)hi << 32 | lo) + (in ? x * 64 : -grp * 16));
            keys[i * 64 + lane] = in ? v : (u32x4){0, 0, 0, 0};
        }
        __syncthreads();
        for (int t = s0 + tid; t < b0; t += kShare * 64) {
            const int pos = a.positions[t];
            if (pos >= t0 && pos < len) early = 1;
        }
        const float was = tok.page >= 0 && t0 + lane < old ? a.mass[tok.at] : 0.0f;
        float w[T::PSUB][4];
#pragma unroll
        for (int s = 0; s < T::PSUB; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[s][i] = 0.0f;
        __syncthreads();
        if (early) b0 = s0;

        struct Round { Column<CT, DP> x[NC]; };
        auto round = [&](Round &r) {
            bool any = false, all = true;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if (r.x[n].pos >= len) r.x[n].pos = -1;
                any = any || r.x[n].pos >= t0;
                all = all && r.x[n].pos >= t0 + T::PNT - 1;
            }
            if (!__any(any)) return;
            auto go = [&](auto every) {
#pragma unroll
                for (int b = 0; b < T::PSUB; ++b) {
                    u32x4 k[T::KC];
#pragma unroll
                    for (int y = 0; y < T::KC; ++y) k[y] = keys[(b * T::KC + y) * 64 + lane];
#pragma unroll
                    for (int n = 0; n < NC; ++n)
                        weigh<decltype(every)::value>(w[b], scores<CT, DP>(k, r.x[n]), a.scale2, r.x[n].lse2, r.x[n].rest, t0 + b * 16 + grp * 4, r.x[n].pos);
                }
            };
            if (__all(all)) go(std::true_type{});
            else go(std::false_type{});
        };
        for (int part = 0; part < parts; ++part) {
            bool mine[NC], has = false;
            int row[NC];
            const char *qp[NC], *qs[NC];
            const float *lp[NC], *ls[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int head = head0[n] + part * COLS;
                mine[n] = whole > 0 ? crow[n] < whole : head < a.group;       // (columns left over by whole rows have none)
                has = has || mine[n];
                row[n] = b0 + crow[n];
                const int h = g * a.group + (mine[n] ? head : 0);
                qs[n] = a.q + (int64_t)s0 * a.q_sr + h * a.q_sh + grp * (CT == KF8 ? 32 : 16);
                qp[n] = qs[n] + (int64_t)(row[n] - s0) * a.q_sr;
                ls[n] = a.lse + (int64_t)s0 * a.n_heads + h;
                lp[n] = ls[n] + (int64_t)(row[n] - s0) * a.n_heads;
            }
            if (!__any(has)) continue;
            const int64_t q_on = step * a.q_sr, l_on = (int64_t)step * a.n_heads;
            auto ask = [&](Round &r) {
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const bool is = mine[n] && row[n] < s1;   // (else: the request's first row, and not counted)
                    const int pos = a.positions[is ? row[n] : s0];
                    load_column<CT, DP, EXACT>(a, r.x[n], is ? qp[n] : qs[n], is ? *lp[n] : *ls[n], is ? pos : -1, grp);
                    row[n] += step;
                    qp[n] += q_on;
                    lp[n] += l_on;
                }
            };
            // the first row of the wave's columns in this round; two rounds at a time
            int first = b0 + (whole > 0 ? wave * 16 * NC / a.group : 0);
            Round x, y;
            if (first < s1) ask(x);
            while (first < s1) {
                if (first + step < s1) ask(y);
                round(x);
                first += step;
                if (first >= s1) break;
                if (first + step < s1) ask(x);
                round(y);
                first += step;
            }
        }
        join_columns<T::PSUB>(w, sums[wave], lane);
        __syncthreads();
        if (wave == 0 && tok.page >= 0) {
            float got = sums[0][lane];
#pragma unroll
            for (int x = 1; x < kShare; ++x) got += sums[x][lane];
            a.mass[tok.at] = got + was;
        }
        __syncthreads();                          // readers of keys, sums and early
    }
}

template <int CT, int DP>
hipError_t go_d(Mp &k, bool prompt, hipStream_t stream) {
    using T = MTile<CT, DP>;
    const int64_t heads = (int64_t)k.batch * k.n_kv;
    if (prompt) {
        const int64_t tiles = (k.row_len + T::PNT - 1) / T::PNT;
        k.blocks = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, 65536 / heads));
        const dim3 grid((unsigned)(((int64_t)k.batch * k.blocks + 7) / 8 * 8 * k.n_kv));
        const int lds = T::PSUB * T::KC * 1024;
        const void *f = k.d == DP ? (const void *)kv_mass_prompt_kernel<CT, DP, true> : (const void *)kv_mass_prompt_kernel<CT, DP, false>;
        if (lds > 32 * 1024) {               // more than a block has unasked, from 64 KiB on
            const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        if (k.d == DP) hipLaunchKernelGGL((kv_mass_prompt_kernel<CT, DP, true>), grid, dim3(kShare * 64), lds, stream, k);
        else hipLaunchKernelGGL((kv_mass_prompt_kernel<CT, DP, false>), grid, dim3(kShare * 64), lds, stream, k);
        return hipGetLastError();
    }
    // the blocks that are resident at once, or a wave a tile if those are fewer
    const int64_t tiles = (k.row_len + T::NT - 1) / T::NT;
    const dim3 grid((unsigned)std::min<int64_t>((heads * tiles + kW - 1) / kW, T::OCC * kCUs));
    const size_t lds = (size_t)k.batch * sizeof(int);
    if (k.d == DP) hipLaunchKernelGGL((kv_mass_step_kernel<CT, DP, true>), grid, dim3(kW * 64), lds, stream, k);
    else hipLaunchKernelGGL((kv_mass_step_kernel<CT, DP, false>), grid, dim3(kW * 64), lds, stream, k);
    return hipGetLastError();
}
template <int CT>
hipError_t go(Mp &k, bool prompt, hipStream_t stream) {
    if (k.d <= 64) return go_d<CT, 64>(k, prompt, stream);
    if (k.d <= 128) return go_d<CT, 128>(k, prompt, stream);
    if (k.d <= 192) return go_d<CT, 192>(k, prompt, stream);
    return go_d<CT, 256>(k, prompt, stream);
}

}  // namespace

hipError_t launch_kv_mass(const KvMassArgs &a, hipStream_t stream, const char **kernel_name) {
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    Mp k = {};
    k.q = (const char *)a.q; k.k = (const char *)a.k_cache; k.lse = a.lse; k.mass = a.mass;
    k.table = a.block_table; k.starts = a.starts; k.positions = a.positions; k.len_old = a.len_old; k.lens = a.lens;
    k.table_stride = a.table_stride; k.q_sr = a.q_st * qe; k.q_sh = a.q_sh * qe;
    k.c_sp = a.c_sp * e; k.c_st = a.c_st * e; k.c_sh = a.c_sh * e;
    k.n_tokens = (int)a.n_tokens; k.n_heads = (int)a.n_heads; k.n_kv = (int)a.n_kv_heads; k.group = (int)(a.n_heads / a.n_kv_heads);
    k.d = a.headdim; k.n_pages = (int)a.n_pages; k.page_size = (int)a.page_size; k.row_len = (int)(a.max_pages * a.page_size);
    k.scale2 = a.scale * (a.kv_dtype == SSM_KV_F8E4M3 ? a.k_scale : 1.0f) * kLog2e;
    // by columns a request on average (rows of q that each tile of tokens meets), and from a quarter as many on where a block a
    // tile is resident at once and the step's form would leave the chip idle.  us (step, prompt):
    //   16 requests of 2000 tokens, 4 kv heads of 128, bf16:  16 columns 10.9, 32.0;  61: 22.1, 34.3;  123: 39.5, 38.5;  248: 70, 50
    //   16 of 4000, 4 of 128, fp32:  122: 235, 138;   32 of 2000, 4 of 256, bf16:  38: 78, 75
    //   2 of 4000, 4 of 128, fp32:  20: 9.5, 13.4;  80: 20.0, 16.7;  160: 33.4, 23.0
    //   4 of 1000, 4 of 64, 8 bits:  43: 9.2, 5.9;  86: 13.0, 6.6;  172: 20.9, 7.7
    //   8 of 2000, 1 of 256, bf16:  35: 8.9, 6.9;  75: 14.8, 7.9;  155: 26.3, 11.0
    const bool idle = k.row_len <= 64 * (2 * kCUs / (a.batch * a.n_kv_heads));
    const bool prompt = a.n_tokens * k.group >= (idle ? 32 : 128) * a.batch;
    k.batch = (int)a.batch;
    *kernel_name = prompt ? "kv_mass_prompt_kernel" : "kv_mass_step_kernel";
    return a.kv_dtype == SSM_KV_F32 ? go<KF32>(k, prompt, stream) : a.kv_dtype == SSM_KV_BF16 ? go<KBF16>(k, prompt, stream)
                                                                                             : go<KF8>(k, prompt, stream);
}

}  // namespace ssm
