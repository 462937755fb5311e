// kv_mass.hip -- the softmax weight that each cached token gathers from a step's queries
// (ssm_kv_mass_update in include/ssm_longctx.h).
//
// w_j = sum over rows and heads of 2^(log2(e) (scale q . k_j - lse)): given lse, no maximum and no second pass.
// A wave has 16 to 64 tokens of a (request, kv head), their keys in registers for as long as it takes to walk
// the request's (row, head) pairs, 16 at a time, as columns of the matrix products; a lane adds up its
// column's exponentials, and the 16 lanes of a token are joined once at the end.  No two waves add to one token.
// Bound: for one row a request HBM, the keys; for prompts the exponentials, one a
// (row, head, token), with 2 headdim operations on the matrix cores beside each.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_device.hpp"
#include "attn_launchers.hpp"
#include "device_common.hpp"

namespace ssm {
namespace {

constexpr int kW = 4;               // waves of a block

struct Mp {
    const char *q; const char *k; const float *lse; float *mass;
    const int32_t *table; const int32_t *starts; const int32_t *positions; const int32_t *len_old; const int32_t *lens;
    int64_t table_stride, q_sr, q_sh, c_sp, c_st, c_sh;              // q and cache strides in bytes
    int n_tokens, n_heads, n_kv, group, d, n_pages, page_size, row_len, blocks;   // blocks: of a (request, kv head)
    float scale2;
};

template <int CT, int DP> struct MTile {
    static constexpr int E = CT == KF32 ? 4 : CT == KBF16 ? 2 : 1;
    static constexpr int KD = 16 / E, KC = DP / (4 * KD);            // dims of a load of K, loads of a row (four lanes each)
    static constexpr int QW = CT == KF8 ? 2 : 1;                     // operands of q to a load of K
    static constexpr int SUB = KC <= 4 ? 4 : KC <= 8 ? 2 : 1;        // 16-token blocks: 64 registers of keys
    static constexpr int NT = SUB * 16;
};

template <int CT, int DP, bool EXACT>
__global__ void __launch_bounds__(kW * 64) kv_mass_kernel(Mp a) {
    using T = MTile<CT, DP>;
    __shared__ float sums[kW][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    const int hr = blockIdx.x / a.blocks, blk = blockIdx.x - hr * a.blocks;
    const int r = hr / a.n_kv, g = hr - r * a.n_kv;
    const PageSize ps(a.page_size);
    const int len = min(max(a.lens[r], 0), a.row_len), old = a.len_old[r];
    const int s0 = min(max(a.starts[r], 0), a.n_tokens), s1 = min(max(a.starts[r + 1], s0), a.n_tokens);
    const int cols = (s1 - s0) * a.group;
    const char *kb = a.k + (int64_t)g * a.c_sh + grp * 16;
    const char *qb = a.q + (int64_t)g * a.group * a.q_sh + grp * (CT == KF32 ? 16 : CT == KBF16 ? 16 : 32);
    const float *lb = a.lse + (int64_t)g * a.group;
    for (int t0 = (blk * kW + wave) * T::NT; t0 < len; t0 += a.blocks * kW * T::NT) {
        // a lane's token: its page (-1: none), its place among the keys, what it gathered before
        const int tok = t0 + (lane & (T::NT - 1)), pj = ps.of(tok);
        int page = tok < len ? a.table[(int64_t)r * a.table_stride + pj] : -1;
        if ((uint32_t)page >= (uint32_t)a.n_pages) page = -1;
        const int place = ps.place(tok, pj);
        const int64_t at = ((int64_t)max(page, 0) * a.n_kv + g) * a.page_size + place;
        const float was = page >= 0 && tok < old ? a.mass[at] : 0.0f;
        const uint64_t off = page >= 0 ? (uint64_t)page * (uint64_t)a.c_sp + (uint64_t)place * (uint64_t)a.c_st : 0;
        u32x4 kf[T::SUB][T::KC];
        if (cols > 0) {
#pragma unroll
            for (int s = 0; s < T::SUB; ++s) {
                const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, 16 * s + col), hi = (uint32_t)__shfl((int)(off >> 32), 16 * s + col);
                const char *p = kb + ((uint64_t)hi << 32 | lo);
#pragma unroll
                for (int c = 0; c < T::KC; ++c) {
                    // past headdim: the row's own first dims, and zero instead
                    const bool in = EXACT || (c * 4 + grp) * T::KD < a.d;
                    const u32x4 x = *(const u32x4 *)(p + (in ? c * 64 : -grp * 16));
                    kf[s][c] = in ? x : (u32x4){0, 0, 0, 0};
                }
            }
        }
        float w[T::SUB][4];
#pragma unroll
        for (int s = 0; s < T::SUB; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[s][i] = 0.0f;

        for (int c0 = 0; c0 < cols; c0 += 16) {
            const int c = c0 + col, i = c / a.group, h = c - i * a.group;
            const int64_t t = s0 + (c < cols ? i : 0);
            int pos = c < cols ? a.positions[t] : -1;         // the last token that this column sees
            if (pos >= len) pos = -1;
            const float lse = c < cols ? lb[t * a.n_heads + h] : 0.0f;
            if (lse == -INFINITY) pos = -1;
            if (!__any(pos >= t0)) continue;
            const float lse2 = lse * kLog2e;
            const char *qp = qb + t * a.q_sr + (c < cols ? h : 0) * a.q_sh;
            f32x4 s[T::SUB];
#pragma unroll
            for (int b = 0; b < T::SUB; ++b) s[b] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < T::KC; ++k) {
                u32x4 q[T::QW];
#pragma unroll
                for (int x = 0; x < T::QW; ++x) {
                    const int dim = (k * 4 + grp) * T::KD + x * 8;
                    q[x] = (u32x4){0, 0, 0, 0};
                    if (EXACT || dim < a.d) q[x] = *(const u32x4 *)(qp + k * 64 * T::QW + x * 16);
                }
#pragma unroll
                for (int b = 0; b < T::SUB; ++b) {
                    const u32x4 x = kf[b][k];
                    if constexpr (CT == KBF16) {
                        s[b] = mfma_bf16(x, q[0], s[b]);
                    } else if constexpr (CT == KF8) {
                        const u32x4 k0 = {widen<false>(x[0]), widen<true>(x[0]), widen<false>(x[1]), widen<true>(x[1])};
                        const u32x4 k1 = {widen<false>(x[2]), widen<true>(x[2]), widen<false>(x[3]), widen<true>(x[3])};
                        s[b] = mfma_bf16(k0, q[0], s[b]);
                        s[b] = mfma_bf16(k1, q[T::QW - 1], s[b]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[e]), __uint_as_float(q[0][e]), s[b], 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < T::SUB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = exp2_fast(fmaf(s[b][e], a.scale2, -lse2));
                    w[b][e] += t0 + b * 16 + grp * 4 + e <= pos ? p : 0.0f;
                }
        }
        // the 16 columns of a token, and the token's sum to the lane that has its place
#pragma unroll
        for (int b = 0; b < T::SUB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = w[b][e];
                v += __shfl_xor(v, 1);
                v += __shfl_xor(v, 2);
                v += __shfl_xor(v, 4);
                v += __shfl_xor(v, 8);
                if (col == 0) sums[wave][b * 16 + grp * 4 + e] = v;
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float got = sums[wave][lane & (T::NT - 1)];
        if (page >= 0 && lane < T::NT) a.mass[at] = got + was;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int CT, int DP>
void go_d(Mp &k, int64_t heads, hipStream_t stream) {
    const int64_t tiles = (k.row_len + kW * MTile<CT, DP>::NT - 1) / (kW * MTile<CT, DP>::NT);
    // a block a tile of each wave up to a limit, since most tables have room for more tokens than they hold
    k.blocks = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, 32768 / heads));
    const dim3 grid((unsigned)(heads * k.blocks));
    if (k.d == DP) hipLaunchKernelGGL((kv_mass_kernel<CT, DP, true>), grid, dim3(kW * 64), 0, stream, k);
    else hipLaunchKernelGGL((kv_mass_kernel<CT, DP, false>), grid, dim3(kW * 64), 0, stream, k);
}
template <int CT>
void go(Mp &k, int64_t heads, hipStream_t stream) {
    if (k.d <= 64) go_d<CT, 64>(k, heads, stream);
    else if (k.d <= 128) go_d<CT, 128>(k, heads, stream);
    else if (k.d <= 192) go_d<CT, 192>(k, heads, stream);
    else go_d<CT, 256>(k, heads, stream);
}

}  // namespace

hipError_t launch_kv_mass(const KvMassArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "kv_mass_kernel";
    const int e = a.kv_dtype == SSM_KV_F32 ? 4 : a.kv_dtype == SSM_KV_BF16 ? 2 : 1, qe = a.kv_dtype == SSM_KV_F32 ? 4 : 2;
    Mp k = {};
    k.q = (const char *)a.q; k.k = (const char *)a.k_cache; k.lse = a.lse; k.mass = a.mass;
    k.table = a.block_table; k.starts = a.starts; k.positions = a.positions; k.len_old = a.len_old; k.lens = a.lens;
    k.table_stride = a.table_stride; k.q_sr = a.q_st * qe; k.q_sh = a.q_sh * qe;
    k.c_sp = a.c_sp * e; k.c_st = a.c_st * e; k.c_sh = a.c_sh * e;
    k.n_tokens = (int)a.n_tokens; k.n_heads = (int)a.n_heads; k.n_kv = (int)a.n_kv_heads; k.group = (int)(a.n_heads / a.n_kv_heads);
    k.d = a.headdim; k.n_pages = (int)a.n_pages; k.page_size = (int)a.page_size; k.row_len = (int)(a.max_pages * a.page_size);
    k.scale2 = a.scale * (a.kv_dtype == SSM_KV_F8E4M3 ? a.k_scale : 1.0f) * kLog2e;
    const int64_t heads = a.batch * a.n_kv_heads;
    if (a.kv_dtype == SSM_KV_F32) go<KF32>(k, heads, stream);
    else if (a.kv_dtype == SSM_KV_BF16) go<KBF16>(k, heads, stream);
    else go<KF8>(k, heads, stream);
    return hipGetLastError();
}

}  // namespace ssm
