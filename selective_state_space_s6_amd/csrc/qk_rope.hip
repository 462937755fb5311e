// qk_rope.hip -- RMS norm of each q and k head with the position rotation in the
// same pass, its gradients, and its form that writes k and v into a paged cache
// (ssm_qk_norm_rope_* in include/ssm_attn.h).
//
// Forward: n = x r w with r = 1 / sqrt(mean x^2 + eps), and each pair (a, b) of the first
// rot_dim elements turned by its angle, position * inv_freq: (a c - b s, b c + a s).
// Backward: g = dy turned back, dx = r (w g - x r^2 mean(x w g)), dw = sum of g x r.
//
// All of them move every element once and are bound by HBM.  A wave takes a token at
// a time (of few heads, several) of one side, q, k or v.  Its 64 lanes form the
// token's cosines and sines, one or two each, and hand them round through a part of
// LDS of their own; the heads of the token share them.  Then groups of lanes take one
// head each: a lane holds 2 V elements of it, chosen so that both halves of each rotated
// pair are its own, and only the norm's sums cross lanes.  The next heads' elements are
// asked for before the present ones are worked on, and no wave waits for another.
//
// Measured, us a call, 16384 tokens of 16 + 4 heads of 128 in bf16: forward 168 MB 36.4 (4.6 TB/s; a strided
// copy 35 to 37), backward 252 MB 58 (4.3 TB/s), 4 of it to join dw.  8192 tokens of 32 + 8 + 8 heads into an
// 8-bit cache 185 MB 46.  64 tokens into a cache 5.1, 1021 fp32 tokens of 6 + 3 heads of 72 5.4: a chain
// of loads.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kCUs = 256;
constexpr int kFwdWaves = 4;        // waves of a block, forward: one on each SIMD
// Forward: blocks of a compute unit, as many as registers let run at once: up to 66 of them without a
// cache in bf16, 79 in fp32, 80 with a cache.  (16k tokens of 16 + 4 heads of 128, us: bf16 on 6, 7 and 8 blocks, where
// they spill, 34.6, 33.9, 36.1; fp32 on 5, 6 and 8 71.2, 69.9, 77.5; into an 8-bit cache on 6, 7 and 8 42.5, 51.6, 59.6.
// 16 bf16 elements a lane in place of 8, which leave room for 4 blocks: 37.5.)
constexpr int fwd_blocks(int esize, bool cache) { return esize == 2 && !cache ? 7 : 6; }
// Backward: up to 110 registers, 4 waves on a SIMD, in two blocks of 8: one block of 16 starts and ends
// together and leaves half the shares of dw (16k tokens of 16 + 4 heads of 128, bf16 60.6 against 57.8 us, fp32 111.5
// against 106.6), blocks of 4 leave twice as many (4k tokens 20.7 against 20.4 us).  16 bf16 elements a
// lane take 149 registers and 3 waves (16k tokens of 8 + 2 heads of 256 67.5 against 58.6 us, of 8 + 8 heads of 192
// 68.7 against 73.5).
constexpr int kBwdWaves = 8;
constexpr int kBwdBlocks = 2 * kCUs;
constexpr int kOneWaves = 16;       // of the only block of a side
constexpr int kChain = 32;          // heads of a lane whose shares of dw are added up in fp32 before they go on in fp64

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);   // to nearest even
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// V consecutive elements: as loaded, widened to fp32, and rounded back
template <typename T, int V> struct Row;
template <> struct Row<float, 4> {
    typedef float4 Raw;
    __device__ __forceinline__ static void get(Raw u, float *v) { v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w; }
    __device__ __forceinline__ static void st(float *p, const float *v) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Row<float, 1> {
    typedef float Raw;
    __device__ __forceinline__ static void get(Raw u, float *v) { v[0] = u; }
    __device__ __forceinline__ static void st(float *p, const float *v) { *p = v[0]; }
};
template <> struct Row<uint16_t, 4> {
    typedef uint2 Raw;
    __device__ __forceinline__ static void get(Raw u, float *v) {
        v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
    }
    __device__ __forceinline__ static void st(uint16_t *p, const float *v) {
        *(uint2 *)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
};
template <> struct Row<uint16_t, 1> {
    typedef uint16_t Raw;
    __device__ __forceinline__ static void get(Raw u, float *v) { v[0] = lo_f(u); }
    __device__ __forceinline__ static void st(uint16_t *p, const float *v) { *p = (uint16_t)pack_bf16(v[0], v[0]); }
};

// V elements into an 8-bit cache: divided by the scale, clamped to the type's range, and
// rounded once.  The comparisons leave a NaN as it is.
template <int V>
__device__ __forceinline__ void st_f8(uint8_t *p, const float *v, float scale) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = i < V ? v[i] / scale : 0.0f;
        const float y = x > 448.0f ? 448.0f : x;
        c[i] = y < -448.0f ? -448.0f : y;
    }
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    const uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    if constexpr (V == 4) *(uint32_t *)p = w;
    else *p = (uint8_t)w;
}

// cos and sin of position * inv_freq.  The angle is formed and reduced in fp64, as turns:
// a quarter-turn count and a rest of at most 1/8 turn, whose Taylor series (sine to the
// 9th, cosine to the 10th power of at most pi/4: below 2e-9) run in fp32.
constexpr double kTurn = 0.15915494309189533577;       // 1 / (2 pi)
__device__ __forceinline__ float2 cos_sin(int position, double turns) {     // turns: inv_freq / (2 pi)
    const double t = (double)position * turns;
    const double f = t - rint(t);
    const double q = rint(4.0 * f);                     // -2 .. 2
    const float y = (float)((f - 0.25 * q) * 6.28318530717958647692);
    const float z = y * y;
    const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 2.75573192e-6f, -1.98412698e-4f), 8.33333333e-3f), -1.66666667e-1f), y);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.75573192e-7f, 2.48015873e-5f), -1.38888889e-3f), 4.16666667e-2f), -0.5f), 1.0f);
    const int n = (int)q & 3;
    const float cc = (n & 1) ? s : c, ss = (n & 1) ? c : s;
    return make_float2((n == 1 || n == 2) ? -cc : cc, n >= 2 ? -ss : ss);
}

// 1 / sqrt(v): the instruction, within an ulp, on a v that it does not flush to zero; for
// fp32 elements with a Newton step (bf16 rounds to 2^-9 afterwards), which leaves an
// infinite v's 0 and a zero's infinity alone
template <typename T>
__device__ __forceinline__ float inv_sqrt(float v) {
    const bool tiny = v < 0x1p-96f;
    const float u = tiny ? v * 0x1p96f : v;
    float r = __builtin_amdgcn_rsqf(u);
    if constexpr (sizeof(T) == 4) {
        const float e = fmaf(-u * r, r, 1.0f);
        r = fabsf(e) < 0.5f ? fmaf(0.5f * r, e, r) : r;
    }
    return r * (tiny ? 0x1p48f : 1.0f);
}

// sum over the 2^lg lanes of a group (lg is the same in the whole launch); every lane
// gets it
__device__ __forceinline__ float group_sum(float v, int lg) {
    if (lg > 0) v += dpp_f<0xb1>(v);                    // lane ^ 1
    if (lg > 1) v += dpp_f<0x4e>(v);                    // lane ^ 2
    if (lg > 2) v += dpp_f<0x141>(v);                   // the other quad of 8 lanes
    if (lg > 3) v += dpp_f<0x140>(v);                   // the other half of 16 lanes
    if (lg > 4) v += __shfl_xor(v, 16);
    if (lg > 5) v += __shfl_xor(v, 32);
    return v;
}

// Places of a lane's 2 V elements in its head: V at o1, V at o2, and its first pair.  The
// first rot/2/V units rotate, the others hold what follows rot_dim.
struct Unit {
    int o1, o2, pair;
    bool turn, in1, in2;
};
template <int V, bool IL>
__device__ __forceinline__ Unit unit_of(int u, int rot, int d) {
    const int half = rot >> 1, nr = half / V;
    Unit n;
    n.turn = u < nr;
    n.pair = u * V;
    n.o1 = n.turn ? (IL ? 2 * u * V : u * V) : rot + 2 * (u - nr) * V;
    n.o2 = n.turn && !IL ? half + u * V : n.o1 + V;
    n.in1 = n.o1 < d;
    n.in2 = n.o2 < d;
    return n;
}

// What a wave works on: one of q, k, v.  Its tokens stand in groups of `tokens` (1 where the
// heads fill a wave's lane groups, then in `passes` steps of which a wave does `each`).
struct Side {
    const void *x; const void *dy; void *y; const float *w; float *part;
    int64_t st, sh, dst, dsh;      // strides of x and dy: token, head
    int heads, tokens, passes, each, splits;
    int64_t parts;                 // (token group, split) pairs
    int blocks, stride, groups_on, splits_on;      // waves of the side, and what they add to a part
    bool rotate, cache;            // normed and rotated, or copied; y is a cache
};
struct Kp {
    Side side[3];
    const float *inv_freq; const int32_t *positions; const int64_t *slots;
    int64_t n_tokens, c_sp, c_st, c_sh;
    uint32_t page_size, n_slots;
    int d, rot, units, lg;         // units of a head, log2 of its lanes
    float eps, inv_d, k_scale, v_scale;
    bool norm;
    int sums;                      // backward, FOLD: where the sums in fp64 begin in LDS, in floats
};

// LDS of a wave is read by its own lanes: its instructions are in order, the compiler's
// have to be told
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A lane's place in its wave's work, and the cosines and sines of the present token group
template <typename T, int V, bool IL> struct Lane {
    static constexpr int NU = V == 1 ? 2 : 1;    // units (2 only for V = 1, where 64 lanes may be too few)
    typedef typename Row<T, V>::Raw Raw;
    const Kp &a;
    const Side &s;
    float *tab;                                  // this wave's part of LDS: cosines, then sines
    int lane, half, tok, head;                   // token of the group, head of the first pass
    Unit un[NU];
    float freq[2];                               // of angles lane and lane + 64 where the group is one token
    float cs[NU][V], sn[NU][V];

    __device__ __forceinline__ Lane(const Kp &a_, const Side &s_, float *tab_) : a(a_), s(s_), tab(tab_) {
        lane = threadIdx.x & 63;
        half = a.rot >> 1;
        const int lanes = 1 << a.lg, group = lane >> a.lg, u0 = lane & (lanes - 1);
        tok = s.tokens > 1 ? group / s.heads : 0;
        head = group - tok * s.heads;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = u0 + n * lanes;
            un[n] = unit_of<V, IL>(u, a.rot, a.d);
            un[n].in1 &= u < a.units;
            un[n].in2 &= u < a.units;
            un[n].turn &= u < a.units;
#pragma unroll
            for (int i = 0; i < V; ++i) cs[n][i] = sn[n][i] = 0.0f;     // of lanes without a token, too
        }
    }
    // loads that the first elements need not wait for
    __device__ __forceinline__ void frequencies() {
        if (half == 0) return;
#pragma unroll
        for (int k = 0; k < 2; ++k) freq[k] = a.inv_freq[min(lane + 64 * k, half - 1)];
    }
    // token and head of a pass; on: there is such a one
    struct At { int t, h; bool on; };
    __device__ __forceinline__ At at(int64_t group, int pass) const {
        At p;
        p.t = (int)group * s.tokens + tok;
        p.h = head + pass * (64 >> a.lg);
        p.on = tok < s.tokens && p.t < a.n_tokens && p.h < s.heads;
        return p;
    }
    __device__ __forceinline__ void load(Raw (*r)[2], const void *x, int64_t st, int64_t sh, const At &p) const {
        const T *xp = (const T *)x + (int64_t)p.t * st + (int64_t)p.h * sh;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            r[n][0] = Raw{};
            r[n][1] = Raw{};
            if (p.on && un[n].in1) r[n][0] = *(const Raw *)(xp + un[n].o1);
            if (p.on && un[n].in2) r[n][1] = *(const Raw *)(xp + un[n].o2);
        }
    }
    __device__ __forceinline__ int position(const At &p) const {
        return half > 0 && p.t < a.n_tokens && tok < s.tokens ? a.positions[p.t] : 0;
    }
    // cosines and sines of the group's tokens; pos: the position of this lane's own token
    __device__ __forceinline__ void angles(int pos) {
        if (half == 0) return;
        const int n = s.tokens * half;
        wave_sync();                             // readers of the group before
        if (s.tokens == 1) {
            pos = __builtin_amdgcn_readfirstlane(pos);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (lane + 64 * k < n) {
                    const float2 v = cos_sin(pos, (double)freq[k] * kTurn);
                    tab[lane + 64 * k] = v.x;
                    tab[n + lane + 64 * k] = v.y;
                }
        } else {
            for (int i0 = 0; i0 < n; i0 += 64) {
                const int i = i0 + lane, t = min(i / half, s.tokens - 1), j = i - t * half;
                const int p = __shfl(pos, (t * s.heads) << a.lg);
                if (i < n) {
                    const float2 v = cos_sin(p, (double)a.inv_freq[j] * kTurn);
                    tab[i] = v.x;
                    tab[n + i] = v.y;
                }
            }
        }
        wave_sync();
#pragma unroll
        for (int k = 0; k < NU; ++k)
            if (un[k].turn && tok < s.tokens) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    cs[k][i] = tab[tok * half + un[k].pair + i];
                    sn[k][i] = tab[n + tok * half + un[k].pair + i];
                }
            }
    }
    __device__ __forceinline__ void weights(float (*w)[2 * V]) const {
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = h ? un[n].in2 : un[n].in1;
                const float *p = s.w + (in ? (h ? un[n].o2 : un[n].o1) : 0);
                if constexpr (V == 1) {
                    const float u = *p;
                    w[n][h] = in ? u : 0.0f;
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        const float4 u = *(const float4 *)(p + i);
                        w[n][h * V + i] = in ? u.x : 0.0f;
                        w[n][h * V + i + 1] = in ? u.y : 0.0f;
                        w[n][h * V + i + 2] = in ? u.z : 0.0f;
                        w[n][h * V + i + 3] = in ? u.w : 0.0f;
                    }
                }
            }
    }
};

// The parts of a wave: (token group, split) pairs, as many apart as the side has waves, and
// the passes of the group's heads that a split has.
struct Walk {
    int64_t part, group;
    int split, pass0, pass1;
    __device__ __forceinline__ Walk(const Side &s, uint32_t first) : part(first) {
        const uint32_t g = first / (uint32_t)s.splits;
        group = g;
        split = (int)(first - g * (uint32_t)s.splits);
        passes(s);
    }
    __device__ __forceinline__ void passes(const Side &s) {
        pass0 = split * s.each;
        pass1 = min(pass0 + s.each, s.passes);
    }
    __device__ __forceinline__ bool next(const Side &s) {
        part += s.stride;
        group += s.groups_on;
        split += s.splits_on;
        if (split >= s.splits) { split -= s.splits; ++group; }
        passes(s);
        return part < s.parts;
    }
};

// the side of a block and the block's number in it
__device__ __forceinline__ int side_of(const Kp &a, int &blk) {
    int i = 0;
    while (blk >= a.side[i].blocks) blk -= a.side[i++].blocks;
    return i;
}

// turns the pairs of a lane's 2 V elements; SIGN -1 turns them back
template <int V, bool IL, int SIGN>
__device__ __forceinline__ void turn(float *x, const float *cs, const float *sn) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float &a = x[IL ? 2 * i : i], &b = x[IL ? 2 * i + 1 : V + i];
        const float c = cs[i], s = SIGN * sn[i], u = a, v = b;
        a = fmaf(u, c, -v * s);
        b = fmaf(v, c, u * s);
    }
}

template <typename T, int V, bool IL, int KV>      // KV: 0 no cache, 1 a cache of type T, 2 an 8-bit cache
__global__ void __launch_bounds__(kFwdWaves * 64, fwd_blocks(sizeof(T), KV != 0)) qk_rope_kernel(Kp a) {
    typedef Lane<T, V, IL> L;
    constexpr int NU = L::NU;
    extern __shared__ float tab[];
    int blk = blockIdx.x;
    const Side &s = a.side[side_of(a, blk)];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    L me(a, s, tab + wave * s.tokens * a.rot);
    const bool norm = s.rotate && a.norm;
    float w[NU][2 * V];
    Walk at(s, (uint32_t)(blk * kFwdWaves + wave));
    if (at.part >= s.parts) return;
    int pass = at.pass0;

    typename L::Raw raw[NU][2], ahead[NU][2];
    typename L::At p = me.at(at.group, pass);
    me.load(raw, s.x, s.st, s.sh, p);
    int pos = s.rotate ? me.position(p) : 0;
    bool turn_group = true;             // the present step is the first of its group
    if (norm) me.weights(w);
    if (s.rotate) me.frequencies();
    while (true) {
        // what comes next is asked for first
        const bool new_group = turn_group;
        const int64_t group = at.group;
        const int pass_now = pass;
        turn_group = pass + 1 >= at.pass1;
        const bool more = turn_group ? at.next(s) : true;
        pass = turn_group ? at.pass0 : pass + 1;
        int pos_n = 0;
        if (more) {
            const typename L::At p_n = me.at(at.group, pass);
            me.load(ahead, s.x, s.st, s.sh, p_n);
            if (turn_group && s.rotate) pos_n = me.position(p_n);
        }
        p = me.at(group, pass_now);
        int64_t slot = 0;
        if (KV != 0 && s.cache && p.on) slot = a.slots[p.t];
        if (s.rotate && new_group) me.angles(pos);

        float x[NU][2 * V], ss = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            Row<T, V>::get(raw[n][0], x[n]);
            Row<T, V>::get(raw[n][1], x[n] + V);
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) ss = fmaf(x[n][i], x[n][i], ss);
        }
        if (norm) {
            const float r = inv_sqrt<T>(fmaf(group_sum(ss, a.lg), a.inv_d, a.eps));
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) x[n][i] = x[n][i] * r * w[n][i];
        }
        int64_t row = ((int64_t)p.t * s.heads + p.h) * a.d;
        bool keep = p.on;
        if (KV != 0 && s.cache) {
            keep = keep && slot >= 0 && slot < (int64_t)a.n_slots;
            const uint32_t sl = keep ? (uint32_t)slot : 0u, page = sl / a.page_size;
            row = page * a.c_sp + (sl - page * a.page_size) * a.c_st + p.h * a.c_sh;
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (s.rotate && me.un[n].turn) turn<V, IL, 1>(x[n], me.cs[n], me.sn[n]);
            if (KV == 2 && s.cache) {
                const float scale = s.rotate ? a.k_scale : a.v_scale;
                uint8_t *yp = (uint8_t *)s.y + row;
                if (keep && me.un[n].in1) st_f8<V>(yp + me.un[n].o1, x[n], scale);
                if (keep && me.un[n].in2) st_f8<V>(yp + me.un[n].o2, x[n] + V, scale);
            } else {
                T *yp = (T *)s.y + row;
                if (keep && me.un[n].in1) Row<T, V>::st(yp + me.un[n].o1, x[n]);
                if (keep && me.un[n].in2) Row<T, V>::st(yp + me.un[n].o2, x[n] + V);
            }
        }
        if (!more) break;
        if (turn_group) pos = pos_n;
#pragma unroll
        for (int n = 0; n < NU; ++n) { raw[n][0] = ahead[n][0]; raw[n][1] = ahead[n][1]; }
    }
}

// The gradients.  A wave keeps its share of dw in registers (a lane's elements are the same
// in every head); the shares of its lane groups are joined across lanes at the end, those of
// the block's waves in LDS.  FOLD: where a lane has more than kChain heads, what it has goes to a sum in
// fp64 each time that it has so many, in its own part of LDS: the error of dw does not grow with the tokens.
// (Tokens of 16 + 4 heads of 128, us without and with: 65536 in bf16 203.4, 203.7, in fp32 402.2, 403.7; of 3 + 1 heads
// of 90, one element a lane, 300000 in bf16 580, 588.  The same tests in one kernel cost those that need none 1%.)
template <typename T, int V, bool IL, int WAVES, bool FOLD>
__global__ void __launch_bounds__(WAVES * 64, 4) qk_rope_bwd_kernel(Kp a) {
    typedef Lane<T, V, IL> L;
    constexpr int NU = L::NU;
    extern __shared__ float tab[];
    int blk = blockIdx.x;
    const Side &s = a.side[side_of(a, blk)];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    L me(a, s, tab + wave * s.tokens * a.rot);
    float w[NU][2 * V], dw[NU][2 * V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) dw[n][i] = 0.0f;
    double *sums = (double *)(tab + a.sums) + wave * (64 * NU * 2 * V) + me.lane;
    if constexpr (FOLD) {
#pragma unroll
        for (int i = 0; i < NU * 2 * V; ++i) sums[i * 64] = 0.0;
    }
    int chain = 0;
    Walk at(s, (uint32_t)(blk * WAVES + wave));
    if (at.part < s.parts) {
        int pass = at.pass0;
        typename L::Raw raw[NU][2], raw_g[NU][2], ahead[NU][2], ahead_g[NU][2];
        typename L::At p = me.at(at.group, pass);
        me.load(raw_g, s.dy, s.dst, s.dsh, p);
        if (a.norm) me.load(raw, s.x, s.st, s.sh, p);
        int pos = me.position(p);
        bool turn_group = true;         // the present step is the first of its group
        if (a.norm) me.weights(w);
        me.frequencies();
        while (true) {
            const bool new_group = turn_group;
            const int64_t group = at.group;
            const int pass_now = pass;
            turn_group = pass + 1 >= at.pass1;
            const bool more = turn_group ? at.next(s) : true;
            pass = turn_group ? at.pass0 : pass + 1;
            int pos_n = 0;
            if (more) {
                const typename L::At p_n = me.at(at.group, pass);
                me.load(ahead_g, s.dy, s.dst, s.dsh, p_n);
                if (a.norm) me.load(ahead, s.x, s.st, s.sh, p_n);
                if (turn_group) pos_n = me.position(p_n);
            }
            p = me.at(group, pass_now);
            if (new_group) me.angles(pos);

            float x[NU][2 * V], g[NU][2 * V], ss = 0.0f, sg = 0.0f;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                Row<T, V>::get(raw_g[n][0], g[n]);
                Row<T, V>::get(raw_g[n][1], g[n] + V);
                if (me.un[n].turn) turn<V, IL, -1>(g[n], me.cs[n], me.sn[n]);
                if (a.norm) {
                    Row<T, V>::get(raw[n][0], x[n]);
                    Row<T, V>::get(raw[n][1], x[n] + V);
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        ss = fmaf(x[n][i], x[n][i], ss);
                        sg = fmaf(x[n][i], w[n][i] * g[n][i], sg);
                    }
                }
            }
            if (a.norm) {
                // (lanes without a head: with eps = 0 their 1/0 would turn all of dw into NaN)
                const float mean = fmaf(group_sum(ss, a.lg), a.inv_d, a.eps);
                const float r = p.on ? inv_sqrt<T>(mean) : 0.0f;
                const float c = group_sum(sg, a.lg) * a.inv_d * r * r;
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        dw[n][i] = fmaf(g[n][i], x[n][i] * r, dw[n][i]);
                        g[n][i] = r * fmaf(w[n][i], g[n][i], -x[n][i] * c);
                    }
                if (FOLD && ++chain == kChain) {
                    chain = 0;
#pragma unroll
                    for (int i = 0; i < NU * 2 * V; ++i) {
                        float &v = dw[i / (2 * V)][i % (2 * V)];
                        sums[i * 64] += (double)v;
                        v = 0.0f;
                    }
                }
            }
            T *yp = (T *)s.y + ((int64_t)p.t * s.heads + p.h) * a.d;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (p.on && me.un[n].in1) Row<T, V>::st(yp + me.un[n].o1, g[n]);
                if (p.on && me.un[n].in2) Row<T, V>::st(yp + me.un[n].o2, g[n] + V);
            }
            if (!more) break;
            if (turn_group) pos = pos_n;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) { raw[n][i] = ahead[n][i]; raw_g[n][i] = ahead_g[n][i]; }
        }
    }
    if (!a.norm) return;
    if constexpr (FOLD) {
#pragma unroll
        for (int i = 0; i < NU * 2 * V; ++i) {
            float &v = dw[i / (2 * V)][i % (2 * V)];
            v = (float)(sums[i * 64] + (double)v);
        }
    }
    __syncthreads();                             // the angles' last readers
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i)
            for (int o = 1 << a.lg; o < 64; o <<= 1) dw[n][i] += __shfl_xor(dw[n][i], o);
    if (me.lane < 1 << a.lg) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (me.un[n].in1) tab[wave * a.d + me.un[n].o1 + i] = dw[n][i];
                if (me.un[n].in2) tab[wave * a.d + me.un[n].o2 + i] = dw[n][V + i];
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += WAVES * 64) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) v += tab[k * a.d + e];
        s.part[(int64_t)blk * a.d + e] = v;
    }
}

// dw = sum of the blocks' shares in fp64: 8 elements a block, 32 slices of the shares, all asked for at once
__global__ void __launch_bounds__(256) qk_rope_dw_kernel(const float *pq, const float *pk, float *dwq, float *dwk,
                                                         int nq, int nk, int d) {
    __shared__ double sum[32][9];
    const int i = threadIdx.x & 7, e = blockIdx.x * 8 + i, sl = threadIdx.x >> 3;
    const float *p = (blockIdx.y ? pk : pq) + min(e, d - 1);
    const int n = blockIdx.y ? nk : nq;
    double v = 0.0;
    if (n > 0) {
        float share[kBwdBlocks / 32];
#pragma unroll
        for (int k = 0; k < kBwdBlocks / 32; ++k) share[k] = p[min(sl + 32 * k, n - 1) * d];
#pragma unroll
        for (int k = 0; k < kBwdBlocks / 32; ++k) v += sl + 32 * k < n ? (double)share[k] : 0.0;
    }
    sum[sl][i] = v;
    __syncthreads();
    if (sl == 0 && e < d) {
#pragma unroll
        for (int k = 1; k < 32; ++k) v += sum[k][i];
        (blockIdx.y ? dwk : dwq)[e] = (float)v;
    }
}

// ------------------------------------------------------------------ host ----
// 4 where units of 2 x 4 elements fit the rotation's halves, what follows it, and every
// address; else 1, which fits everything
int pick_v(const void *const *ptr, const int64_t *stride, int np, int ns, int d, int rot, int esize,
           const float *wq, const float *wk) {
    bool ok = (((uintptr_t)wq | (uintptr_t)wk) & 15) == 0;         // weights are loaded by fours
    ok &= rot / 2 % 4 == 0 && (d - rot) % 8 == 0;
    for (int i = 0; i < np; ++i) ok &= ((uintptr_t)ptr[i] & (uintptr_t)(4 * esize - 1)) == 0;
    for (int i = 0; i < ns; ++i) ok &= stride[i] % 4 == 0;
    return ok ? 4 : 1;
}

void set_geometry(Kp &k, int v, int d, int rot) {
    k.d = d;
    k.rot = rot;
    k.units = rot / 2 / v + (d - rot + 2 * v - 1) / (2 * v);
    k.lg = 0;
    while ((1 << k.lg) < k.units && k.lg < 6) ++k.lg;
    k.inv_d = 1.0f / (float)d;
}

// blocks that a side may have: its share of the launch's, by heads
int blocks_of(int64_t heads, int64_t all_heads, int most) {
    return (int)std::max<int64_t>(1, most * heads / all_heads);
}

// Parts of a side's work, (token group, split of its passes) pairs dealt to the waves that
// the chip holds at once.  A group is split where that evens the waves' steps out, or gives more of
// them one (4096 tokens of 64 + 8 heads of 128: 34.3 us in whole groups, 30.7 split); a part costs
// about half a step more, for its angles.
void set_work(Side &s, const Kp &k, int64_t n_tokens, int64_t all_heads, int waves, int blocks) {
    const int groups = 64 >> k.lg;
    s.tokens = std::max(1, groups / s.heads);
    s.passes = (s.heads + groups - 1) / groups;
    const int64_t token_groups = (n_tokens + s.tokens - 1) / s.tokens;
    const int64_t most = (int64_t)blocks_of(s.heads, all_heads, blocks) * waves;
    int64_t best = INT64_MAX;
    for (int t = 1; t <= std::min(s.passes, 64); ++t) {
        const int each = (s.passes + t - 1) / t, splits = (s.passes + each - 1) / each;
        const int64_t steps = (token_groups * splits + most - 1) / most * (2 * each + 1);
        if (steps >= best) continue;
        best = steps;
        s.each = each;
        s.splits = splits;
    }
    s.parts = token_groups * s.splits;
    s.blocks = (int)((std::min(s.parts, most) + waves - 1) / waves);
    s.stride = s.blocks * waves;
    s.groups_on = s.stride / s.splits;
    s.splits_on = s.stride % s.splits;
}

size_t table_bytes(const Kp &k, int waves) {
    size_t most = 0;
    for (const Side &s : k.side)
        if (s.blocks > 0 && s.rotate) most = std::max(most, (size_t)waves * s.tokens * k.rot * sizeof(float));
    return most;
}

template <typename T, int V, int KV>
void fwd_go(const Kp &k, unsigned blocks, size_t lds, bool il, hipStream_t stream) {
    if (il) hipLaunchKernelGGL((qk_rope_kernel<T, V, true, KV>), dim3(blocks), dim3(kFwdWaves * 64), lds, stream, k);
    else hipLaunchKernelGGL((qk_rope_kernel<T, V, false, KV>), dim3(blocks), dim3(kFwdWaves * 64), lds, stream, k);
}
template <int KV>
void fwd_type(const Kp &k, unsigned blocks, size_t lds, bool bf16, int v, bool il, hipStream_t stream) {
    if (bf16) {
        if (v == 4) fwd_go<uint16_t, 4, KV>(k, blocks, lds, il, stream);
        else fwd_go<uint16_t, 1, KV>(k, blocks, lds, il, stream);
    } else if constexpr (KV != 2) {
        if (v == 4) fwd_go<float, 4, KV>(k, blocks, lds, il, stream);
        else fwd_go<float, 1, KV>(k, blocks, lds, il, stream);
    }
}

template <typename T, int V, int WAVES, bool FOLD>
void bwd_waves_go(const Kp &k, unsigned blocks, bool il, size_t lds, hipStream_t stream) {
    if (il) hipLaunchKernelGGL((qk_rope_bwd_kernel<T, V, true, WAVES, FOLD>), dim3(blocks), dim3(WAVES * 64), lds, stream, k);
    else hipLaunchKernelGGL((qk_rope_bwd_kernel<T, V, false, WAVES, FOLD>), dim3(blocks), dim3(WAVES * 64), lds, stream, k);
}
template <typename T, int V>
void bwd_go(const Kp &k, unsigned blocks, bool one, bool il, size_t lds, hipStream_t stream) {
    if (one) bwd_waves_go<T, V, kOneWaves, false>(k, blocks, il, lds, stream);
    else if (k.sums) bwd_waves_go<T, V, kBwdWaves, true>(k, blocks, il, lds, stream);
    else bwd_waves_go<T, V, kBwdWaves, false>(k, blocks, il, lds, stream);
}

}  // namespace

hipError_t launch_qk_rope(const QkRopeArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "qk_rope_kernel";
    const bool cache = a.slots != nullptr, f8 = cache && a.kv_dtype == SSM_KV_F8E4M3;
    const int esize = a.bf16 ? 2 : 4;
    const void *ptr[] = {a.q, a.q_out, a.k, a.k_out, a.v};
    const int64_t stride[] = {a.q_st, a.q_sh, a.k_st, a.k_sh, a.v_st, a.v_sh, (int64_t)a.headdim};
    int v = pick_v(ptr, stride, cache ? 5 : a.n_kv_heads > 0 ? 4 : 2, 7, a.headdim, a.rot_dim, esize, a.wq, a.wk);
    if (cache) {   // the cache's own addresses: V elements of 1, 2 or 4 bytes
        const void *cp[] = {a.k_out, a.v_cache};
        const int64_t cs[] = {a.c_sp, a.c_st, a.c_sh};
        const int ce = f8 ? 1 : esize;
        bool ok = true;
        for (const void *p : cp) ok &= ((uintptr_t)p & (uintptr_t)(v * ce - 1)) == 0;
        for (int64_t st : cs) ok &= st % v == 0;
        if (!ok) v = 1;
    }
    Kp k = {};
    set_geometry(k, v, a.headdim, a.rot_dim);
    k.inv_freq = a.inv_freq; k.positions = a.positions; k.slots = a.slots;
    k.n_tokens = a.n_tokens; k.c_sp = a.c_sp; k.c_st = a.c_st; k.c_sh = a.c_sh;
    k.page_size = (uint32_t)a.page_size; k.n_slots = (uint32_t)(a.n_pages * a.page_size);
    k.eps = a.eps; k.k_scale = a.k_scale; k.v_scale = a.v_scale;
    k.norm = (a.flags & SSM_QK_NO_NORM) == 0;
    auto side = [&](int i, const void *x, void *y, const float *w, int64_t st, int64_t sh, int64_t heads, bool rotate, bool to_cache) {
        Side &s = k.side[i];
        s.x = x; s.y = y; s.w = w; s.st = st; s.sh = sh;
        s.heads = (int)heads; s.rotate = rotate; s.cache = to_cache;
        set_work(s, k, a.n_tokens, a.n_heads + (cache ? 2 : 1) * a.n_kv_heads, kFwdWaves,
                 kCUs * fwd_blocks(esize, cache));
    };
    side(0, a.q, a.q_out, a.wq, a.q_st, a.q_sh, a.n_heads, true, false);
    if (a.n_kv_heads > 0) side(1, a.k, a.k_out, a.wk, a.k_st, a.k_sh, a.n_kv_heads, true, cache);
    if (cache) side(2, a.v, a.v_cache, nullptr, a.v_st, a.v_sh, a.n_kv_heads, false, true);
    const unsigned blocks = (unsigned)(k.side[0].blocks + k.side[1].blocks + k.side[2].blocks);
    const size_t lds = table_bytes(k, kFwdWaves);
    const bool il = (a.flags & SSM_ROPE_INTERLEAVED) != 0;
    if (f8) fwd_type<2>(k, blocks, lds, a.bf16, v, il, stream);
    else if (cache) fwd_type<1>(k, blocks, lds, a.bf16, v, il, stream);
    else fwd_type<0>(k, blocks, lds, a.bf16, v, il, stream);
    return hipGetLastError();
}

size_t qk_rope_bwd_workspace_bytes(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                   uint32_t flags) {
    if (flags & SSM_QK_NO_NORM) return 0;
    const int64_t all = n_heads + n_kv_heads;
    auto blocks = [&](int64_t heads) {           // each wave has a (token, head) at least
        return std::min<int64_t>(n_tokens * heads / kBwdWaves + 1, blocks_of(heads, all, kBwdBlocks));
    };
    return (size_t)(blocks(n_heads) + (n_kv_heads > 0 ? blocks(n_kv_heads) : 0)) * (size_t)headdim * sizeof(float);
}

hipError_t launch_qk_rope_bwd(const QkRopeBwdArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "qk_rope_bwd_kernel";
    const int esize = a.bf16 ? 2 : 4;
    const void *ptr[] = {a.q, a.dq_out, a.dq, a.k, a.dk_out, a.dk};
    const int64_t stride[] = {a.q_st, a.q_sh, a.dq_st, a.dq_sh, (int64_t)a.headdim, a.k_st, a.k_sh, a.dk_st, a.dk_sh};
    const bool has_k = a.n_kv_heads > 0, norm = (a.flags & SSM_QK_NO_NORM) == 0;
    const int v = pick_v(ptr, stride, has_k ? 6 : 3, has_k ? 9 : 5, a.headdim, a.rot_dim, esize, a.wq, a.wk);
    Kp k = {};
    set_geometry(k, v, a.headdim, a.rot_dim);
    k.inv_freq = a.inv_freq; k.positions = a.positions;
    k.n_tokens = a.n_tokens; k.eps = a.eps; k.norm = norm;
    auto side = [&](int i, const void *x, const void *dy, void *y, const float *w, int64_t st, int64_t sh, int64_t dst,
                    int64_t dsh, int64_t heads) {
        Side &s = k.side[i];
        s.x = x; s.dy = dy; s.y = y; s.w = w; s.st = st; s.sh = sh; s.dst = dst; s.dsh = dsh;
        s.heads = (int)heads; s.rotate = true;
    };
    // steps of a wave, where the sides have `blocks` blocks together, and one each at least
    auto deal = [&](int blocks, int waves) {
        int64_t most = 0;
        for (int i = 0; i < (has_k ? 2 : 1); ++i) {
            Side &s = k.side[i];
            set_work(s, k, a.n_tokens, a.n_heads + a.n_kv_heads, waves, blocks);
            if (s.blocks > 0) most = std::max(most, (s.parts + s.stride - 1) / s.stride * s.each);
        }
        return most;
    };
    side(0, a.q, a.dq_out, a.dq, a.wq, a.q_st, a.q_sh, a.dq_st, a.dq_sh, a.n_heads);
    if (has_k) side(1, a.k, a.dk_out, a.dk, a.wk, a.k_st, a.k_sh, a.dk_st, a.dk_sh, a.n_kv_heads);
    // Few heads: a block a side, whose share of dw is dw, and no second launch.  (16 + 4 heads of 128, us a
    // call in one launch and in two: 4 tokens, 1 step 6.4 and 9.3; 8 tokens, 2 steps 7.6 and 9.2; 16 tokens, 4
    // steps 10.3 and 9.3.)
    const bool one = norm && a.n_tokens > 0 && deal(1, kOneWaves) <= 2;
    const bool fold = !one && deal(kBwdBlocks, kBwdWaves) > kChain && norm;
    const int waves = one ? kOneWaves : kBwdWaves;
    float *ws = (float *)a.workspace;
    k.side[0].part = one ? a.dwq : ws;
    k.side[1].part = one ? a.dwk : norm ? ws + (int64_t)k.side[0].blocks * a.headdim : nullptr;
    size_t lds = std::max(table_bytes(k, waves), norm ? (size_t)waves * a.headdim * sizeof(float) : 0);
    if (fold) {                        // and at most 32 KiB of sums behind at most 16 KiB
        lds = (lds + 15) / 16 * 16;
        k.sums = (int)(lds / sizeof(float));
        lds += (size_t)waves * 64 * (v == 4 ? 8 : 4) * sizeof(double);
    }
    const unsigned blocks = (unsigned)(k.side[0].blocks + k.side[1].blocks);
    const bool il = (a.flags & SSM_ROPE_INTERLEAVED) != 0;
    if (blocks > 0) {
        if (a.bf16) v == 4 ? bwd_go<uint16_t, 4>(k, blocks, one, il, lds, stream) : bwd_go<uint16_t, 1>(k, blocks, one, il, lds, stream);
        else v == 4 ? bwd_go<float, 4>(k, blocks, one, il, lds, stream) : bwd_go<float, 1>(k, blocks, one, il, lds, stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !norm || one) return e;
    *kernel_name = "qk_rope_dw_kernel";
    hipLaunchKernelGGL(qk_rope_dw_kernel, dim3((unsigned)((a.headdim + 7) / 8), has_k ? 2 : 1), dim3(256), 0, stream,
                       k.side[0].part, k.side[1].part, a.dwq, a.dwk, k.side[0].blocks, k.side[1].blocks, a.headdim);
    return hipGetLastError();
}

}  // namespace ssm
