// qk_rope.hip -- RMS norm of each q and k head with the position rotation in the
// same pass, its gradients, and its form that writes k and v into a paged cache
// (ssm_qk_norm_rope_* in include/ssm_attn.h).
//
// All of them move every element once and are bound by HBM.  A block takes some
// tokens of one side (q, k or v).  It first forms the tokens' cosines and sines
// once, into LDS (the heads of a token share them), then its lane groups take one
// (token, head) each: a lane holds 2 V elements of the head, chosen so that both
// halves of each rotated pair are its own, and only the norm's sums cross lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kNT = 256;
constexpr int kTabMax = 2048;       // angles of a block: 16 KiB of cosines and sines

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);   // to nearest even
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// V consecutive elements, widened to fp32 and rounded back
template <typename T, int V> struct Row;
template <> struct Row<float, 4> {
    __device__ __forceinline__ static void ld(const float *p, float *v) {
        const float4 u = *(const float4 *)p;
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    __device__ __forceinline__ static void st(float *p, const float *v) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Row<float, 1> {
    __device__ __forceinline__ static void ld(const float *p, float *v) { v[0] = *p; }
    __device__ __forceinline__ static void st(float *p, const float *v) { *p = v[0]; }
};
template <> struct Row<uint16_t, 8> {
    __device__ __forceinline__ static void ld(const uint16_t *p, float *v) {
        const uint4 u = *(const uint4 *)p;
        v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
        v[4] = lo_f(u.z); v[5] = hi_f(u.z); v[6] = lo_f(u.w); v[7] = hi_f(u.w);
    }
    __device__ __forceinline__ static void st(uint16_t *p, const float *v) {
        *(uint4 *)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
};
template <> struct Row<uint16_t, 4> {
    __device__ __forceinline__ static void ld(const uint16_t *p, float *v) {
        const uint2 u = *(const uint2 *)p;
        v[0] = lo_f(u.x); v[1] = hi_f(u.x); v[2] = lo_f(u.y); v[3] = hi_f(u.y);
    }
    __device__ __forceinline__ static void st(uint16_t *p, const float *v) {
        *(uint2 *)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
};
template <> struct Row<uint16_t, 1> {
    __device__ __forceinline__ static void ld(const uint16_t *p, float *v) { v[0] = lo_f(*p); }
    __device__ __forceinline__ static void st(uint16_t *p, const float *v) { *p = (uint16_t)pack_bf16(v[0], v[0]); }
};

// V elements into an 8-bit cache: divided by the scale, clamped to the type's range, and
// rounded once.  The comparisons leave a NaN as it is.
template <int V>
__device__ __forceinline__ void st_f8(uint8_t *p, const float *v, float scale) {
    float c[V < 4 ? 4 : V];
#pragma unroll
    for (int i = 0; i < (V < 4 ? 4 : V); ++i) {
        const float x = i < V ? v[i] / scale : 0.0f;
        const float y = x > 448.0f ? 448.0f : x;
        c[i] = y < -448.0f ? -448.0f : y;
    }
    uint32_t w[V < 4 ? 1 : V / 4];
#pragma unroll
    for (int i = 0; i < (V < 4 ? 1 : V / 4); ++i) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], u, true);
    }
    if constexpr (V == 8) *(uint2 *)p = make_uint2(w[0], w[1]);
    else if constexpr (V == 4) *(uint32_t *)p = w[0];
    else *p = (uint8_t)w[0];
}

// cos and sin of position * inv_freq.  The angle is formed and reduced in fp64, as turns:
// a quarter-turn count and a rest of at most 1/8 turn, whose Taylor series (sine to the
// 9th, cosine to the 10th power of at most pi/4: below 2e-9) run in fp32.
__device__ __forceinline__ float2 cos_sin(int position, float inv_freq) {
    constexpr double kTurn = 0.15915494309189533577;   // 1 / (2 pi)
    const double t = (double)position * ((double)inv_freq * kTurn);
    const double f = t - rint(t);
    const double q = rint(4.0 * f);                     // -2 .. 2
    const float y = (float)(f - 0.25 * q) * 6.28318530717958647692f;
    const float z = y * y;
    const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 2.75573192e-6f, -1.98412698e-4f), 8.33333333e-3f), -1.66666667e-1f), y);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.75573192e-7f, 2.48015873e-5f), -1.38888889e-3f), 4.16666667e-2f), -0.5f), 1.0f);
    const int n = (int)q & 3;
    const float cc = (n & 1) ? s : c, ss = (n & 1) ? c : s;
    return make_float2((n == 1 || n == 2) ? -cc : cc, n >= 2 ? -ss : ss);
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

// what a block works on: one of q, k, v
struct Side {
    const void *x; const void *dy; void *y; const float *w; float *part;
    int64_t st, sh, dst, dsh;      // strides of x and dy: token, head
    int heads, tb, blocks;         // tb: tokens a block takes at a time
    uint32_t magic;                // ceil(2^32 / heads): i / heads = i * magic >> 32
    int kind;                      // 0: normed and rotated, 1: copied
    bool cache;                    // y is a cache
};
struct Kp {
    Side side[3];
    const float *inv_freq; const int32_t *positions; const int64_t *slots;
    int64_t n_tokens, c_sp, c_st, c_sh;
    uint32_t page_size, n_slots;
    int d, rot, units, lg;         // units of a head, log2 of its lanes
    float eps, inv_d, k_scale, v_scale;
    bool norm;
};

__device__ __forceinline__ int div_heads(int i, const Side &s) {
    return s.heads == 1 ? i : (int)__umulhi((uint32_t)i, s.magic);
}

// cosines and sines of tb tokens from t0 on into cs[0 .. tb*half) and sn = cs + tb*half
__device__ __forceinline__ void fill_table(const Kp &a, int64_t t0, int tb, float *cs) {
    const int half = a.rot >> 1, n = tb * half;
    for (int i = threadIdx.x; i < n; i += kNT) {
        const int t = i / half, j = i - t * half;
        if (t0 + t >= a.n_tokens) break;
        const float2 v = cos_sin(a.positions[t0 + t], a.inv_freq[j]);
        cs[i] = v.x;
        cs[n + i] = v.y;
    }
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

// NU units a lane (2 only for V = 1, where 64 lanes may be too few for a head)
template <typename T, int V, bool IL, int KV>      // KV: 0 no cache, 1 a cache of type T, 2 an 8-bit cache
__global__ void __launch_bounds__(kNT) qk_rope_kernel(Kp a) {
    constexpr int NU = V == 1 ? 2 : 1;
    extern __shared__ float tab[];
    int blk = blockIdx.x, si = 0;
    while (blk >= a.side[si].blocks) blk -= a.side[si++].blocks;     // uniform
    const Side &s = a.side[si];
    const int64_t t0 = (int64_t)blk * s.tb;
    const int half = a.rot >> 1, lanes = 1 << a.lg, ng = kNT >> a.lg;
    const int u0 = threadIdx.x & (lanes - 1);
    const bool work = s.kind == 0, norm = work && a.norm;
    if (work) fill_table(a, t0, s.tb, tab);
    Unit un[NU];
    float w[NU][2 * V];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = u0 + n * lanes;
        un[n] = unit_of<V, IL>(u, a.rot, a.d);
        un[n].in1 &= u < a.units;
        un[n].in2 &= u < a.units;
        if (norm) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                w[n][i] = un[n].in1 ? s.w[un[n].o1 + i] : 0.0f;
                w[n][V + i] = un[n].in2 ? s.w[un[n].o2 + i] : 0.0f;
            }
        }
    }
    __syncthreads();
    const int items = s.tb * s.heads;
    for (int it = threadIdx.x >> a.lg; it < items; it += ng) {
        const int tok = div_heads(it, s), h = it - tok * s.heads;
        const int64_t t = t0 + tok;
        if (t >= a.n_tokens) break;
        const T *xp = (const T *)s.x + t * s.st + h * s.sh;
        float x[NU][2 * V];
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) x[n][i] = 0.0f;
            if (un[n].in1) Row<T, V>::ld(xp + un[n].o1, x[n]);
            if (un[n].in2) Row<T, V>::ld(xp + un[n].o2, x[n] + V);
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) ss = fmaf(x[n][i], x[n][i], ss);
        }
        if (norm) {
            const float r = 1.0f / sqrtf(fmaf(group_sum(ss, a.lg), a.inv_d, a.eps));
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) x[n][i] = x[n][i] * r * w[n][i];
        }
        int64_t row;
        bool keep = true;
        if (KV != 0 && s.cache) {
            const int64_t slot = a.slots[t];
            keep = slot >= 0 && slot < (int64_t)a.n_slots;
            const uint32_t sl = keep ? (uint32_t)slot : 0u, page = sl / a.page_size;
            row = page * a.c_sp + (sl - page * a.page_size) * a.c_st + h * a.c_sh;
        } else {
            row = (t * s.heads + h) * a.d;
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (work && un[n].turn && un[n].in1)
                turn<V, IL, 1>(x[n], tab + tok * half + un[n].pair, tab + (s.tb + tok) * half + un[n].pair);
            if (KV == 2 && s.cache) {
                const float scale = work ? a.k_scale : a.v_scale;
                uint8_t *yp = (uint8_t *)s.y + row;
                if (keep && un[n].in1) st_f8<V>(yp + un[n].o1, x[n], scale);
                if (keep && un[n].in2) st_f8<V>(yp + un[n].o2, x[n] + V, scale);
            } else {
                T *yp = (T *)s.y + row;
                if (keep && un[n].in1) Row<T, V>::st(yp + un[n].o1, x[n]);
                if (keep && un[n].in2) Row<T, V>::st(yp + un[n].o2, x[n] + V);
            }
        }
    }
}

// The gradients.  A block walks its side's token groups blk, blk + blocks, ... and keeps
// its share of dw in registers (a lane's elements are the same in every head); the
// shares of its lane groups are joined in LDS at the end.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kNT) qk_rope_bwd_kernel(Kp a) {
    constexpr int NU = V == 1 ? 2 : 1;
    extern __shared__ float tab[];
    int blk = blockIdx.x, si = 0;
    while (blk >= a.side[si].blocks) blk -= a.side[si++].blocks;     // uniform
    const Side &s = a.side[si];
    const int half = a.rot >> 1, lanes = 1 << a.lg, ng = kNT >> a.lg;
    const int u0 = threadIdx.x & (lanes - 1);
    Unit un[NU];
    float w[NU][2 * V], dw[NU][2 * V];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = u0 + n * lanes;
        un[n] = unit_of<V, IL>(u, a.rot, a.d);
        un[n].in1 &= u < a.units;
        un[n].in2 &= u < a.units;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[n][i] = a.norm && un[n].in1 ? s.w[un[n].o1 + i] : 0.0f;
            w[n][V + i] = a.norm && un[n].in2 ? s.w[un[n].o2 + i] : 0.0f;
            dw[n][i] = 0.0f;
            dw[n][V + i] = 0.0f;
        }
    }
    const int items = s.tb * s.heads;
    const int64_t step = (int64_t)s.blocks * s.tb;
    for (int64_t t0 = (int64_t)blk * s.tb; t0 < a.n_tokens; t0 += step) {
        __syncthreads();                               // the table's last readers
        fill_table(a, t0, s.tb, tab);
        __syncthreads();
        for (int it = threadIdx.x >> a.lg; it < items; it += ng) {
            const int tok = div_heads(it, s), h = it - tok * s.heads;
            const int64_t t = t0 + tok;
            if (t >= a.n_tokens) break;
            const T *xp = (const T *)s.x + t * s.st + h * s.sh;
            const T *gp = (const T *)s.dy + t * s.dst + h * s.dsh;
            T *yp = (T *)s.y + (t * s.heads + h) * a.d;
            float x[NU][2 * V], g[NU][2 * V];
            float ss = 0.0f, sg = 0.0f;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) { x[n][i] = 0.0f; g[n][i] = 0.0f; }
                if (un[n].in1) Row<T, V>::ld(gp + un[n].o1, g[n]);
                if (un[n].in2) Row<T, V>::ld(gp + un[n].o2, g[n] + V);
                if (a.norm && un[n].in1) Row<T, V>::ld(xp + un[n].o1, x[n]);
                if (a.norm && un[n].in2) Row<T, V>::ld(xp + un[n].o2, x[n] + V);
                if (un[n].turn && un[n].in1)
                    turn<V, IL, -1>(g[n], tab + tok * half + un[n].pair, tab + (s.tb + tok) * half + un[n].pair);
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    ss = fmaf(x[n][i], x[n][i], ss);
                    sg = fmaf(x[n][i], w[n][i] * g[n][i], sg);
                }
            }
            if (a.norm) {
                const float r = 1.0f / sqrtf(fmaf(group_sum(ss, a.lg), a.inv_d, a.eps));
                const float c = group_sum(sg, a.lg) * a.inv_d * r * r;
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        dw[n][i] = fmaf(g[n][i], x[n][i] * r, dw[n][i]);
                        g[n][i] = r * fmaf(w[n][i], g[n][i], -x[n][i] * c);
                    }
            }
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (un[n].in1) Row<T, V>::st(yp + un[n].o1, g[n]);
                if (un[n].in2) Row<T, V>::st(yp + un[n].o2, g[n] + V);
            }
        }
    }
    if (!a.norm) return;
    __syncthreads();
    const int group = threadIdx.x >> a.lg;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (un[n].in1) tab[group * a.d + un[n].o1 + i] = dw[n][i];
            if (un[n].in2) tab[group * a.d + un[n].o2 + i] = dw[n][V + i];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += kNT) {
        float v = 0.0f;
        for (int k = 0; k < ng; ++k) v += tab[k * a.d + e];
        s.part[(int64_t)blk * a.d + e] = v;
    }
}

// dw = sum of the blocks' shares in fp64: 16 elements a block, 16 slices of the shares
__global__ void __launch_bounds__(kNT) qk_rope_dw_kernel(const float *pq, const float *pk, float *dwq, float *dwk,
                                                         int nq, int nk, int d) {
    __shared__ double sum[16][17];
    const int e = blockIdx.x * 16 + (threadIdx.x & 15), sl = threadIdx.x >> 4;
    const float *p = blockIdx.y ? pk : pq;
    const int n = blockIdx.y ? nk : nq;
    double v = 0.0;
    if (e < d)
        for (int i = sl; i < n; i += 16) v += (double)p[(int64_t)i * d + e];
    sum[sl][threadIdx.x & 15] = v;
    __syncthreads();
    if (sl == 0 && e < d) {
        for (int i = 1; i < 16; ++i) v += sum[i][threadIdx.x & 15];
        (blockIdx.y ? dwk : dwq)[e] = (float)v;
    }
}

// ------------------------------------------------------------------ host ----
// Widest V whose unit of 2 V elements fits the rotation's halves, what follows it, and
// every address: 16 bytes where possible.  V = 1 fits everything.
int pick_v(const void *const *ptr, const int64_t *stride, int np, int ns, int d, int rot, int esize) {
    for (int v = 16 / esize; v >= 4; v >>= 1) {
        bool ok = (rot / 2) % v == 0 && (d - rot) % (2 * v) == 0;
        for (int i = 0; i < np; ++i) ok &= ((uintptr_t)ptr[i] & (uintptr_t)(v * esize - 1)) == 0;
        for (int i = 0; i < ns; ++i) ok &= stride[i] % v == 0;
        if (ok) return v;
    }
    return 1;
}

void set_geometry(Kp &k, int v, int d, int rot) {
    k.d = d;
    k.rot = rot;
    k.units = rot / 2 / v + (d - rot + 2 * v - 1) / (2 * v);
    k.lg = 0;
    while ((1 << k.lg) < k.units && k.lg < 6) ++k.lg;
    k.inv_d = 1.0f / (float)d;
}

// tokens of a block: two (token, head) items a lane group, fewer where that leaves the
// chip's 256 compute units without a block, and no more angles than the table holds
void set_tokens(Side &s, const Kp &k, int64_t n_tokens) {
    const int ng = kNT >> k.lg, half = k.rot / 2;
    int64_t tb = 2 * ng / s.heads;
    if (tb > n_tokens / 256) tb = n_tokens / 256;
    if (half > 0 && tb > kTabMax / half) tb = kTabMax / half;
    s.tb = (int)(tb < 1 ? 1 : tb);
    s.blocks = (int)((n_tokens + s.tb - 1) / s.tb);
    s.magic = s.heads > 1 ? (uint32_t)(((uint64_t(1) << 32) + s.heads - 1) / s.heads) : 0;
}

size_t table_bytes(const Kp &k) {
    size_t most = 0;
    for (const Side &s : k.side)
        if (s.blocks > 0) most = std::max(most, (size_t)s.tb * k.rot * sizeof(float));
    return most;
}

template <typename T, int V, int KV>
void fwd_go(const Kp &k, unsigned blocks, size_t lds, bool il, hipStream_t stream) {
    if (il) hipLaunchKernelGGL((qk_rope_kernel<T, V, true, KV>), dim3(blocks), dim3(kNT), lds, stream, k);
    else hipLaunchKernelGGL((qk_rope_kernel<T, V, false, KV>), dim3(blocks), dim3(kNT), lds, stream, k);
}
template <int KV>
void fwd_type(const Kp &k, unsigned blocks, size_t lds, bool bf16, int v, bool il, hipStream_t stream) {
    if (bf16) {
        if (v == 8) fwd_go<uint16_t, 8, KV>(k, blocks, lds, il, stream);
        else if (v == 4) fwd_go<uint16_t, 4, KV>(k, blocks, lds, il, stream);
        else fwd_go<uint16_t, 1, KV>(k, blocks, lds, il, stream);
    } else if constexpr (KV != 2) {
        if (v == 4) fwd_go<float, 4, KV>(k, blocks, lds, il, stream);
        else fwd_go<float, 1, KV>(k, blocks, lds, il, stream);
    }
}

// blocks of the backward's sides: at most 1024 in all, in proportion to the heads
void bwd_blocks(int64_t n_tokens, int64_t nq, int64_t nk, int &bq, int &bk) {
    const double share = 1024.0 / (double)(nq + nk);
    bq = (int)std::min<int64_t>(n_tokens, std::max<int64_t>(1, (int64_t)(share * (double)nq)));
    bk = nk > 0 ? (int)std::min<int64_t>(n_tokens, std::max<int64_t>(1, (int64_t)(share * (double)nk))) : 0;
}

}  // namespace

hipError_t launch_qk_rope(const QkRopeArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "qk_rope_kernel";
    const bool cache = a.slots != nullptr, f8 = cache && a.kv_dtype == SSM_KV_F8E4M3;
    const int esize = a.bf16 ? 2 : 4;
    const void *ptr[] = {a.q, a.q_out, a.k, a.k_out, a.v};
    const int64_t stride[] = {a.q_st, a.q_sh, a.k_st, a.k_sh, a.v_st, a.v_sh, (int64_t)a.headdim};
    int v = pick_v(ptr, stride, cache ? 5 : a.n_kv_heads > 0 ? 4 : 2, 7, a.headdim, a.rot_dim, esize);
    if (cache) {   // the cache's own addresses: V elements of 1, 2 or 4 bytes
        const void *cp[] = {a.k_out, a.v_cache};
        const int64_t cs[] = {a.c_sp, a.c_st, a.c_sh};
        const int ce = f8 ? 1 : esize;
        for (; v > 1; v = v > 4 ? v / 2 : 1) {
            bool ok = (a.rot_dim / 2) % v == 0 && (a.headdim - a.rot_dim) % (2 * v) == 0;
            for (const void *p : cp) ok &= ((uintptr_t)p & (uintptr_t)(v * ce - 1)) == 0;
            for (int64_t st : cs) ok &= st % v == 0;
            if (ok) break;
        }
    }
    Kp k = {};
    set_geometry(k, v, a.headdim, a.rot_dim);
    k.inv_freq = a.inv_freq; k.positions = a.positions; k.slots = a.slots;
    k.n_tokens = a.n_tokens; k.c_sp = a.c_sp; k.c_st = a.c_st; k.c_sh = a.c_sh;
    k.page_size = (uint32_t)a.page_size; k.n_slots = (uint32_t)(a.n_pages * a.page_size);
    k.eps = a.eps; k.k_scale = a.k_scale; k.v_scale = a.v_scale;
    k.norm = (a.flags & SSM_QK_NO_NORM) == 0;
    k.side[0] = {a.q, nullptr, a.q_out, a.wq, nullptr, a.q_st, a.q_sh, 0, 0, (int)a.n_heads, 0, 0, 0, 0, false};
    k.side[1] = {a.k, nullptr, a.k_out, a.wk, nullptr, a.k_st, a.k_sh, 0, 0, (int)a.n_kv_heads, 0, 0, 0, 0, cache};
    k.side[2] = {a.v, nullptr, a.v_cache, nullptr, nullptr, a.v_st, a.v_sh, 0, 0, (int)a.n_kv_heads, 0, 0, 0, 1, cache};
    set_tokens(k.side[0], k, a.n_tokens);
    if (a.n_kv_heads > 0) set_tokens(k.side[1], k, a.n_tokens);
    if (cache) set_tokens(k.side[2], k, a.n_tokens);
    const unsigned blocks = (unsigned)(k.side[0].blocks + k.side[1].blocks + k.side[2].blocks);
    const size_t lds = table_bytes(k);
    const bool il = (a.flags & SSM_ROPE_INTERLEAVED) != 0;
    if (f8) fwd_type<2>(k, blocks, lds, a.bf16, v, il, stream);
    else if (cache) fwd_type<1>(k, blocks, lds, a.bf16, v, il, stream);
    else fwd_type<0>(k, blocks, lds, a.bf16, v, il, stream);
    return hipGetLastError();
}

size_t qk_rope_bwd_workspace_bytes(int64_t n_tokens, int64_t n_heads, int64_t n_kv_heads, int64_t headdim,
                                   uint32_t flags) {
    if (flags & SSM_QK_NO_NORM) return 0;
    int bq, bk;
    bwd_blocks(n_tokens, n_heads, n_kv_heads, bq, bk);
    return (size_t)(bq + bk) * (size_t)headdim * sizeof(float);
}

hipError_t launch_qk_rope_bwd(const QkRopeBwdArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "qk_rope_bwd_kernel";
    const int esize = a.bf16 ? 2 : 4;
    const void *ptr[] = {a.q, a.dq_out, a.dq, a.k, a.dk_out, a.dk};
    const int64_t stride[] = {a.q_st, a.q_sh, a.dq_st, a.dq_sh, (int64_t)a.headdim, a.k_st, a.k_sh, a.dk_st, a.dk_sh};
    const bool has_k = a.n_kv_heads > 0, norm = (a.flags & SSM_QK_NO_NORM) == 0;
    const int v = pick_v(ptr, stride, has_k ? 6 : 3, has_k ? 9 : 5, a.headdim, a.rot_dim, esize);
    Kp k = {};
    set_geometry(k, v, a.headdim, a.rot_dim);
    k.inv_freq = a.inv_freq; k.positions = a.positions;
    k.n_tokens = a.n_tokens; k.eps = a.eps; k.norm = norm;
    k.side[0] = {a.q, a.dq_out, a.dq, a.wq, nullptr, a.q_st, a.q_sh, a.dq_st, a.dq_sh, (int)a.n_heads, 0, 0, 0, 0, false};
    k.side[1] = {a.k, a.dk_out, a.dk, a.wk, nullptr, a.k_st, a.k_sh, a.dk_st, a.dk_sh, (int)a.n_kv_heads, 0, 0, 0, 0, false};
    int bq, bk;
    bwd_blocks(a.n_tokens, a.n_heads, a.n_kv_heads, bq, bk);
    set_tokens(k.side[0], k, a.n_tokens);
    k.side[0].blocks = std::min(k.side[0].blocks, bq);
    if (has_k) {
        set_tokens(k.side[1], k, a.n_tokens);
        k.side[1].blocks = std::min(k.side[1].blocks, bk);
    }
    float *ws = (float *)a.workspace;
    k.side[0].part = ws;
    k.side[1].part = norm ? ws + (int64_t)k.side[0].blocks * a.headdim : nullptr;
    // the joining of dw takes 2 V floats of every thread
    const size_t lds = std::max(table_bytes(k), norm ? (size_t)kNT * (size_t)(v == 1 ? 4 : 2 * v) * sizeof(float) : 0);
    const unsigned blocks = (unsigned)(k.side[0].blocks + k.side[1].blocks);
    const bool il = (a.flags & SSM_ROPE_INTERLEAVED) != 0;
#define SSM_BWD(T, V)                                                                                           \
    do {                                                                                                        \
        if (il) hipLaunchKernelGGL((qk_rope_bwd_kernel<T, V, true>), dim3(blocks), dim3(kNT), lds, stream, k);  \
        else hipLaunchKernelGGL((qk_rope_bwd_kernel<T, V, false>), dim3(blocks), dim3(kNT), lds, stream, k);    \
    } while (0)
    if (blocks > 0) {
        if (a.bf16) {
            if (v == 8) SSM_BWD(uint16_t, 8);
            else if (v == 4) SSM_BWD(uint16_t, 4);
            else SSM_BWD(uint16_t, 1);
        } else {
            if (v == 4) SSM_BWD(float, 4);
            else SSM_BWD(float, 1);
        }
    }
#undef SSM_BWD
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !norm) return e;
    *kernel_name = "qk_rope_dw_kernel";
    hipLaunchKernelGGL(qk_rope_dw_kernel, dim3((unsigned)((a.headdim + 15) / 16), has_k ? 2 : 1), dim3(kNT), 0, stream,
                       k.side[0].part, k.side[1].part, a.dwq, a.dwk, k.side[0].blocks, k.side[1].blocks, a.headdim);
    return hipGetLastError();
}

}  // namespace ssm
