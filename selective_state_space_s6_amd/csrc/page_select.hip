// page_select.hip -- the pages of a row's cache that attention is to look at, by the largest product
// that a page's keys can have with the row's queries (ssm_kv_page_select_fwd in include/ssm_longctx.h).
//
// Two launches: the scores of every page as 32-bit keys into the workspace, and the choice, a block for
// each (row, kv head).  Products in 64 bits because the result is an order: sums in 32 bits would differ with the order of
// their terms in the last places, and with them which of two close pages is taken.
// Four lanes have a page, 16 bytes of its bounds each, read once for up to 8 query heads; max(q, 0) and min(q, 0) wait in shared
// memory in 64 bits and are read once for the two pages of a lane (for four 46 us, more registers than two blocks
// leave; q in registers and exchanged between lanes 42 to 65; two 37).
// Bound: the shared memory's reads of q, 16 bytes a dim and head, beside 2 headdim multiply-adds in 64 bits; HBM would take
// 25.  32 rows of up to 2048 pages, 32 + 8 heads of 128, bf16 (127 MB): 37 us, and 7.6 for the choice, 12 passes or so over keys
// in shared memory.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_launchers.hpp"
#include "topk.hpp"

namespace ssm {
namespace {

constexpr int kNT = 256;            // threads of a scoring block
constexpr int kPages = 2;           // pages of a lane
constexpr int kStep = kNT / 4 * kPages;      // pages of a block
constexpr int kBlocks = 2048;       // scoring blocks: twice what is resident at once, since rows' lengths differ (37 us above; 41 with half)
constexpr int kKept = 8192;         // keys that the choice keeps in shared memory

template <int CT> struct Wide {
    static constexpr int N = CT == KF32 ? 4 : CT == KBF16 ? 8 : 16;
    __device__ __forceinline__ static double at(u32x4 w, int i) {
        if constexpr (CT == KF32) return (double)__uint_as_float(w[i]);
        else if constexpr (CT == KBF16) return (double)(i & 1 ? hi_f(w[i / 2]) : lo_f(w[i / 2]));
        else {
            const f32x2 p = (i & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i / 4], true)
                                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i / 4], false);
            return (double)p[i & 1];
        }
    }
};

// GH: query heads of a round
template <int CT, int GH>
__global__ void __launch_bounds__(kNT) page_score_kernel(PageSelectArgs a, int chunks) {
    constexpr int N = Wide<CT>::N;
    extern __shared__ double2 qs[];               // (16-byte chunk of dims, dim, head): max(q, 0) and min(q, 0)
    const int tid = threadIdx.x, l = tid & 3;
    const int hr = blockIdx.x / chunks, chunk = blockIdx.x - hr * chunks;
    const int row = hr / a.n_kv, g = hr - row * a.n_kv;
    const PageSize ps(a.page_size);
    const int n = ps.to_hold(min(max(a.lens[row], 0), a.max_pages * a.page_size));
    if (n <= a.top_k) return;                     // all of them: no score is asked for
    const int lo = a.first, hi = n - a.last;      // what scores decide about
    if (lo + chunk * kStep >= hi) return;
    const int group = a.n_heads / a.n_kv, dims = a.d / N;            // chunks of 16 bytes
    const int64_t row_bytes = (int64_t)dims * 16;
    uint32_t *keys = a.keys + (int64_t)hr * a.max_pages;
    const int32_t *table = a.table + (int64_t)row * a.table_stride;
    constexpr int PITCH = N * GH + 1;             // (a chunk further is another bank)
    auto page_at = [&](int i) { return i < hi ? table[i] : -1; };
    auto load_q = [&](int h0) {
        for (int i = tid; i < a.d * GH; i += kNT) {
            const int dim = i / GH, h = i - dim * GH;
            double v = 0.0;
            if (h0 + h < group) {
                const int64_t at = row * a.q_sr + (int64_t)(g * group + h0 + h) * a.q_sh + dim;
                v = a.bf16 ? (double)lo_f(((const uint16_t *)a.q)[at]) : (double)((const float *)a.q)[at];
            }
            // (a NaN stays one)
            qs[dim / N * PITCH + dim % N * GH + h] = make_double2(v > 0.0 || v != v ? v : 0.0, v < 0.0 || v != v ? v : 0.0);
        }
    };
    int next[kPages];
#pragma unroll
    for (int u = 0; u < kPages; ++u) next[u] = page_at(lo + chunk * kStep + u * (kNT / 4) + (tid >> 2));
    if (group <= GH) {
        load_q(0);
        __syncthreads();
    }
    for (int p0 = lo + chunk * kStep; p0 < hi; p0 += chunks * kStep) {
        uint32_t best[kPages];
        int page[kPages];
        const char *b[kPages];
#pragma unroll
        for (int u = 0; u < kPages; ++u) {
            page[u] = next[u];
            next[u] = page_at(p0 + chunks * kStep + u * (kNT / 4) + (tid >> 2));
            best[u] = 0;
            b[u] = a.bounds + ((int64_t)((uint32_t)page[u] < (uint32_t)a.n_pages ? page[u] : 0) * a.n_kv + g) * 2 * row_bytes + l * 16;
        }
        for (int h0 = 0; h0 < group; h0 += GH) {
            if (group > GH) {
                __syncthreads();
                load_q(h0);
                __syncthreads();
            }
            double acc[kPages][GH];
#pragma unroll
            for (int u = 0; u < kPages; ++u)
#pragma unroll
                for (int h = 0; h < GH; ++h) acc[u][h] = 0.0;
            u32x4 low[kPages], high[kPages];
            auto load = [&](int c) {
#pragma unroll
                for (int u = 0; u < kPages; ++u) {
                    low[u] = *(const u32x4 *)(b[u] + (c - l) * 16);
                    high[u] = *(const u32x4 *)(b[u] + row_bytes + (c - l) * 16);
                }
            };
            if (l < dims) load(l);
            for (int c = l; c < dims; c += 4) {
                u32x4 x0[kPages], y0[kPages];
#pragma unroll
                for (int u = 0; u < kPages; ++u) { x0[u] = low[u]; y0[u] = high[u]; }
                if (c + 4 < dims) load(c + 4);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    double x[kPages], y[kPages];
#pragma unroll
                    for (int u = 0; u < kPages; ++u) {
                        x[u] = Wide<CT>::at(x0[u], e);
                        y[u] = Wide<CT>::at(y0[u], e);
                    }
#pragma unroll
                    for (int h = 0; h < GH; ++h) {
                        const double2 q = qs[c * PITCH + e * GH + h];
#pragma unroll
                        for (int u = 0; u < kPages; ++u) acc[u][h] = fma(q.x, y[u], fma(q.y, x[u], acc[u][h]));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kPages; ++u)
#pragma unroll
                for (int h = 0; h < GH; ++h) {
                    double s = acc[u][h];
                    s += __shfl_xor(s, 1);
                    s += __shfl_xor(s, 2);
                    if (h0 + h < group) best[u] = max(best[u], key_of((float)s));
                }
        }
        if (l == 0) {
#pragma unroll
            for (int u = 0; u < kPages; ++u) {
                const int i = p0 + u * (kNT / 4) + (tid >> 2);
                if (i < hi) keys[i] = (uint32_t)page[u] < (uint32_t)a.n_pages ? best[u] : kKeyLowest;
            }
        }
    }
}

template <int NT>                   // threads
__global__ void __launch_bounds__(NT) page_select_kernel(PageSelectArgs a) {
    __shared__ TopKShared<NT> sh;
    __shared__ uint32_t kept[kKept];
    const int tid = threadIdx.x;
    const int row = blockIdx.x / a.n_kv;
    const PageSize ps(a.page_size);
    const int n = ps.to_hold(min(max(a.lens[row], 0), a.max_pages * a.page_size));
    int32_t *out = a.selected + (int64_t)blockIdx.x * a.top_k;
    if (n <= a.top_k) {
        for (int i = tid; i < a.top_k; i += NT) out[i] = i < n ? i : -1;
        return;
    }
    const int m = n - a.first - a.last, want = a.top_k - a.first - a.last;
    for (int i = tid; i < a.first; i += NT) out[i] = i;
    for (int i = tid; i < a.last; i += NT) out[a.top_k - a.last + i] = n - a.last + i;
    if (want == 0) return;
    const uint32_t *keys = a.keys + (int64_t)blockIdx.x * a.max_pages + a.first;
    for (int i = tid; i < min(m, kKept); i += NT) kept[i] = keys[i];
    __syncthreads();
    auto key = [&](int i) { return i < kKept ? kept[i] : keys[i]; };
    const Cut cut = find_cut<NT>(sh, m, want, key);
    put_chosen<NT>(sh, m, cut, key, [&](int place, int i) { out[a.first + place] = a.first + i; });
}

template <int CT>
void go(const PageSelectArgs &a, hipStream_t stream) {
    const int group = a.n_heads / a.n_kv;
    // blocks that share the pages of a (row, kv head)
    const int64_t heads = (int64_t)a.batch * a.n_kv;
    const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((a.max_pages + kStep - 1) / kStep, kBlocks / heads));
    const dim3 grid((unsigned)(heads * chunks));
    const int gh = group >= 5 ? 8 : group >= 3 ? 4 : group;
    const size_t lds = (size_t)(a.d / Wide<CT>::N) * (Wide<CT>::N * gh + 1) * sizeof(double2);
    switch (gh) {
        case 8: hipLaunchKernelGGL((page_score_kernel<CT, 8>), grid, dim3(kNT), lds, stream, a, (int)chunks); break;
        case 4: hipLaunchKernelGGL((page_score_kernel<CT, 4>), grid, dim3(kNT), lds, stream, a, (int)chunks); break;
        case 2: hipLaunchKernelGGL((page_score_kernel<CT, 2>), grid, dim3(kNT), lds, stream, a, (int)chunks); break;
        default: hipLaunchKernelGGL((page_score_kernel<CT, 1>), grid, dim3(kNT), lds, stream, a, (int)chunks); break;
    }
}

}  // namespace

size_t page_select_workspace_bytes(int64_t batch, int64_t n_kv_heads, int64_t max_pages, int64_t top_k) {
    return max_pages <= top_k ? 0 : (size_t)((batch * n_kv_heads * max_pages * 4 + 15) & ~int64_t(15));
}

hipError_t launch_page_select(const PageSelectArgs &a, hipStream_t stream, const char **kernel_name) {
    if (a.max_pages > a.top_k && a.top_k > a.first + a.last) {
        *kernel_name = "page_score_kernel";
        if (a.kv_dtype == SSM_KV_F32) go<KF32>(a, stream);
        else if (a.kv_dtype == SSM_KV_BF16) go<KBF16>(a, stream);
        else go<KF8>(a, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    *kernel_name = "page_select_kernel";
    // (16 waves where that is one block a compute unit at most, else 8: 256 choices among up to 2048 pages 7.6 us with 16, 8.4
    // with 8, 12 with 4)
    const int64_t heads = (int64_t)a.batch * a.n_kv;
    if (heads <= 256) hipLaunchKernelGGL((page_select_kernel<1024>), dim3((unsigned)heads), dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((page_select_kernel<512>), dim3((unsigned)heads), dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ssm
