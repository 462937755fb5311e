// kv_bounds.hip -- smallest and largest keys of the pages that new tokens stand on
// (ssm_kv_page_bounds_update in include/ssm_longctx.h).
//
// Each new key is read once and each page's bounds written once, so prompts are bound by HBM; a
// decode step (one key and one page a request) by the latency of a chain of loads: lengths, page,
// keys.  How many pages are touched is known on the device alone: every block forms the running sum
// of them over the requests in shared memory, and its waves take (page, kv head)s from that line.  A
// wave has 16 bytes of a key a lane and as many tokens side by side as fit, and joins those at the end.
// 256 requests of one new token, 8 kv heads of 128, bf16: 5 us.  8 prompts of up to 8192 tokens on pages of 64, 8 bits: 10.3 us
// for 34 MB, 3.3 TB/s; on pages of 16 20.3, by the search for a page and the join of its lanes, of a few loads each.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_device.hpp"
#include "attn_launchers.hpp"

namespace ssm {
namespace {

constexpr int kNT = 256, kWaves = kNT / 64;
constexpr int kAhead = 4;           // tokens of a lane that are on their way at once

// smaller and larger of two, NaN if one is
__device__ __forceinline__ float lesser(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float greater(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// the values of 16 bytes of a cache, and back (exact)
template <int CT> struct Chunk {
    static constexpr int N = CT == KF32 ? 4 : CT == KBF16 ? 8 : 16;
    __device__ __forceinline__ static void get(u32x4 w, float *x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (CT == KF32) {
                x[i] = __uint_as_float(w[i]);
            } else if constexpr (CT == KBF16) {
                x[2 * i] = lo_f(w[i]);
                x[2 * i + 1] = hi_f(w[i]);
            } else {
                const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
                x[4 * i] = a[0]; x[4 * i + 1] = a[1]; x[4 * i + 2] = b[0]; x[4 * i + 3] = b[1];
            }
        }
    }
    __device__ __forceinline__ static u32x4 put(const float *x) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (CT == KF32) w[i] = __float_as_uint(x[i]);
            else if constexpr (CT == KBF16) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            else w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3],
                                                                   __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false), true);
        }
        return w;
    }
};

template <int CT>
__global__ void __launch_bounds__(kNT) kv_bounds_kernel(KvBoundsArgs a) {
    constexpr int N = Chunk<CT>::N;
    extern __shared__ int upto[];   // touched pages of the requests up to each
    __shared__ int sums[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const PageSize ps(a.page_size);
    const int room = a.max_pages * a.page_size;

    const int mine = (a.batch + kNT - 1) / kNT, r0 = tid * mine, r1 = min(r0 + mine, a.batch);
    int own = 0;
    for (int r = r0; r < r1; ++r) {
        const int lo = min(max(a.len_old[r], 0), room), hi = min(max(a.lens[r], 0), room);
        own += hi > lo ? ps.to_hold(hi) - ps.of(lo) : 0;
        upto[r] = own;
    }
    int before = wave_scan(own);
    if (lane == 63) sums[wave] = before;
    before -= own;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before += w < wave ? sums[w] : 0;
    for (int r = r0; r < r1; ++r) upto[r] += before;
    __syncthreads();
    const int items = upto[a.batch - 1] * a.n_kv;

    const int chunks = a.row_bytes / 16;
    int side = 1;                   // tokens side by side
    while (2 * side * chunks <= 64) side *= 2;
    const int sub = lane / chunks, c = lane - sub * chunks;
    const bool works = sub < side;
    // (items are fewer than 2^31, and a step behind the last of them may pass that)
    for (uint32_t item = blockIdx.x * kWaves + wave; item < (uint32_t)items; item += gridDim.x * kWaves) {
        const int touch = (int)item / a.n_kv, g = (int)item - touch * a.n_kv;
        int r = 0, end = a.batch - 1;             // the first request with upto > touch
        while (r < end) {
            const int mid = (r + end) >> 1;
            if (upto[mid] > touch) end = mid; else r = mid + 1;
        }
        const int lo = min(max(a.len_old[r], 0), room), hi = min(max(a.lens[r], 0), room);
        const int i = ps.of(lo) + touch - (r > 0 ? upto[r - 1] : 0);
        const int page = a.table[(int64_t)r * a.table_stride + i];
        if ((uint32_t)page >= (uint32_t)a.n_pages || !works) continue;
        const int first = max(lo - i * a.page_size, 0), last = min(hi - i * a.page_size, a.page_size);
        char *b = a.bounds + ((int64_t)page * a.n_kv + g) * 2 * a.row_bytes + c * 16;
        const char *k = a.k + (int64_t)page * a.c_sp + (int64_t)g * a.c_sh + c * 16;
        float low[N], high[N];
        if (first > 0) {                          // what the page had
            Chunk<CT>::get(*(const u32x4 *)b, low);
            Chunk<CT>::get(*(const u32x4 *)(b + a.row_bytes), high);
        } else {
#pragma unroll
            for (int x = 0; x < N; ++x) { low[x] = INFINITY; high[x] = -INFINITY; }
        }
        for (int t = first + sub; t - sub < last; t += kAhead * side) {
            u32x4 w[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) w[u] = *(const u32x4 *)(k + (int64_t)min(t + u * side, last - 1) * a.c_st);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {    // (the last token more than once changes nothing)
                float x[N];
                Chunk<CT>::get(w[u], x);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    low[e] = lesser(low[e], x[e]);
                    high[e] = greater(high[e], x[e]);
                }
            }
        }
        for (int s = side / 2; s > 0; s >>= 1) {
            // (as the cache stores them, which is exact, since every lane that is joined has had a key: 8 dwords in place of 32
            // floats in 8 bits, 24.0 -> 20.3 us for 8 prompts of up to 8192 tokens, 8 heads of 128 on pages of 16)
            u32x4 l = Chunk<CT>::put(low), h = Chunk<CT>::put(high);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l[i] = (uint32_t)__shfl((int)l[i], lane + s * chunks);
                h[i] = (uint32_t)__shfl((int)h[i], lane + s * chunks);
            }
            float x[N];
            Chunk<CT>::get(l, x);
#pragma unroll
            for (int e = 0; e < N; ++e) low[e] = lesser(low[e], x[e]);
            Chunk<CT>::get(h, x);
#pragma unroll
            for (int e = 0; e < N; ++e) high[e] = greater(high[e], x[e]);
        }
        if (sub == 0) {
            *(u32x4 *)b = Chunk<CT>::put(low);
            *(u32x4 *)(b + a.row_bytes) = Chunk<CT>::put(high);
        }
    }
}

}  // namespace

hipError_t launch_kv_bounds(const KvBoundsArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "kv_bounds_kernel";
    const int64_t most = (int64_t)a.batch * a.max_pages * a.n_kv;
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>((most + kWaves - 1) / kWaves, 2048)));
    const size_t lds = (size_t)a.batch * sizeof(int);
    if (a.kv_dtype == SSM_KV_F32) hipLaunchKernelGGL((kv_bounds_kernel<KF32>), grid, dim3(kNT), lds, stream, a);
    else if (a.kv_dtype == SSM_KV_BF16) hipLaunchKernelGGL((kv_bounds_kernel<KBF16>), grid, dim3(kNT), lds, stream, a);
    else hipLaunchKernelGGL((kv_bounds_kernel<KF8>), grid, dim3(kNT), lds, stream, a);
    return hipGetLastError();
}

}  // namespace ssm
