// kv_evict.hip -- eviction from a paged key-value cache by the attention weight that tokens gathered
// (ssm_kv_evict in include/ssm_longctx.h).
//
// Two launches.  The choice: a block for each (request, kv head), keys in shared memory (topk.hpp).  The
// move: kept tokens go forward in their order, in place.  Token i comes from place kept[i] >= i, and
// both rise with i, so a run of tokens whose old values are all in registers may be stored: what it
// overwrites are places below the run's end, which no later token comes from.  One block takes such runs one
// after the other, the next run's places looked up while one is loaded; for more blocks at once, a (request, kv head)'s
// rows are cut along headdim, which are moves of their own, as are k, v and mass.
//
// Bound: HBM, the moved rows read and written.  64 requests of 8 kv heads of 128, bf16, 4160 tokens cut to 4096 of random
// mass: 499 us on a new cache, 15 of them the choice, for 2.1 GB (418 us at the rate of a large copy); 91 where the evicted ones
// are the newest that may go.  One request of 30000 tokens cut to 29000: 113, of one kv head of 64, by the chain of its runs.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>

#include "attn_launchers.hpp"
#include "topk.hpp"

namespace ssm {
namespace {

constexpr int kRun = 8;             // 16-byte pieces of a thread in a run
constexpr int kMostKept = 32768;    // keys that the choice keeps in shared memory at most

template <int kPick>                // threads
__global__ void __launch_bounds__(kPick) evict_pick_kernel(KvEvictArgs a, int room) {
    __shared__ TopKShared<kPick> sh;
    extern __shared__ uint32_t own[];
    const int tid = threadIdx.x;
    const int row = blockIdx.x / a.n_kv, g = blockIdx.x - row * a.n_kv;
    const PageSize ps(a.page_size);
    const int n = min(max(a.lens[row], 0), a.max_pages * a.page_size);
    int32_t *kept = a.kept + (int64_t)blockIdx.x * a.budget;
    if (g == 0 && tid == 0) a.len_out[row] = min(n, a.budget);
    if (n <= a.budget) {
        for (int i = tid; i < a.budget; i += kPick) kept[i] = i < n ? i : -1;
        return;
    }
    const int want = a.budget - a.recent, m = n - a.recent;
    for (int i = tid; i < a.recent; i += kPick) kept[want + i] = m + i;
    if (want == 0) return;
    const int32_t *table = a.table + (int64_t)row * a.table_stride;
    auto load = [&](int i) {
        const int p = ps.of(i), page = table[p];
        if ((uint32_t)page >= (uint32_t)a.n_pages) return kKeyLowest;
        return key_of(a.mass[((int64_t)page * a.n_kv + g) * a.page_size + ps.place(i, p)]);
    };
    constexpr int U = 8;                          // keys of a thread on their way at once
    for (int i0 = tid; i0 < min(m, room); i0 += U * kPick) {
        int page[U], p[U];
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) page[u] = table[p[u] = ps.of(min(i0 + u * kPick, m - 1))];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = (uint32_t)page[u] < (uint32_t)a.n_pages ? page[u] : 0;
            x[u] = a.mass[((int64_t)at * a.n_kv + g) * a.page_size + ps.place(min(i0 + u * kPick, m - 1), p[u])];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kPick < min(m, room)) own[i0 + u * kPick] = (uint32_t)page[u] < (uint32_t)a.n_pages ? key_of(x[u]) : kKeyLowest;
    }
    __syncthreads();
    auto key = [&](int i) { return i < room ? own[i] : load(i); };
    const Cut cut = find_cut<kPick>(sh, m, want, key);
    put_chosen<kPick>(sh, m, cut, key, [&](int place, int i) { kept[place] = i; });
}

// the first i < n with kept[i] != i (n if none): once one is, all later ones are
template <int kMove>                // threads
__device__ __forceinline__ int first_moved(const int32_t *kept, int n) {
    __shared__ int at;
    const int step = (n + kMove - 1) / kMove;
    int lo = 0;
    for (int s = step, count = kMove; ; s = 1, count = step) {       // in steps, then one by one within a step
        __syncthreads();
        if (threadIdx.x == 0) at = n;
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kMove) {
            const int x = lo + i * s;
            if (x < n && kept[x] != x && (i == 0 || kept[x - s] == x - s)) at = x;      // of one x at most
        }
        __syncthreads();
        const int got = at;
        if (s == 1) return got;
        lo = got < n ? max(0, got - s + 1) : (n - 1) / s * s;
    }
}

// slices: parts of a row's 16-byte pieces for k and for v; block 2 * slices of a head moves mass
template <int kMove>                // threads
__global__ void __launch_bounds__(kMove) evict_move_kernel(KvEvictArgs a, int slices) {
    const int tid = threadIdx.x;
    const int hr = blockIdx.x / (2 * slices + 1), part = blockIdx.x - hr * (2 * slices + 1);
    const int row = hr / a.n_kv, g = hr - row * a.n_kv;
    const PageSize ps(a.page_size);
    const int n = min(max(a.lens[row], 0), a.max_pages * a.page_size);
    if (n <= a.budget) return;
    const int32_t *kept = a.kept + (int64_t)hr * a.budget, *table = a.table + (int64_t)row * a.table_stride;
    // Runs of tokens.  Where a token comes from and goes to is looked up a run ahead, and stays unmoved where both are
    // one or have no page.
    const bool is_mass = part == 2 * slices;
    const int pieces = a.row_bytes / 16, s = part >> 1;
    const int c0 = is_mass ? 0 : s * pieces / slices, cs = is_mass ? 1 : (s + 1) * pieces / slices - c0;
    const int side = kMove / cs;                  // tokens side by side
    const int sub = tid / cs, c = c0 + tid - sub * cs;
    const bool works = sub < side;
    const int run = side * kRun;
    // (the look costs 1 to 2 us, and saves the way through what stays: 128 requests of 2000 tokens cut to 1000 with the
    // evicted ones last 85 us without, 56 with)
    const int from = first_moved<kMove>(kept, a.budget);
    struct Move { int src, dst; };                // token places among all (page * page_size + place); src < 0: none
    Move now[kRun], next[kRun];
    auto look_up = [&](Move (&m)[kRun], int base) {
        int j[kRun], src[kRun], dst[kRun];
        // (without branches: all of a run's loads on their way together)
#pragma unroll
        for (int u = 0; u < kRun; ++u) j[u] = kept[min(base + u * side + sub, a.budget - 1)];
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            src[u] = table[ps.of(j[u])];
            dst[u] = table[ps.of(min(base + u * side + sub, a.budget - 1))];
        }
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const int i = base + u * side + sub;
            const bool is = works && i < a.budget && j[u] != i && (uint32_t)src[u] < (uint32_t)a.n_pages && (uint32_t)dst[u] < (uint32_t)a.n_pages;
            m[u].src = is ? src[u] * a.page_size + ps.place(j[u], ps.of(j[u])) : -1;
            m[u].dst = is ? dst[u] * a.page_size + ps.place(i, ps.of(i)) : -1;
        }
    };
    look_up(next, from);
    char *cache = (part & 1 ? a.v : a.k) + (int64_t)g * a.c_sh + c * 16;
    auto row_of = [&](int t) {
        const int page = ps.of(t);
        return cache + (int64_t)page * a.c_sp + (int64_t)ps.place(t, page) * a.c_st;
    };
    auto mass_of = [&](int t) {
        const int page = ps.of(t);
        return a.mass + ((int64_t)page * a.n_kv + g) * a.page_size + ps.place(t, page);
    };
    for (int base = from; base < a.budget; base += run) {
#pragma unroll
        for (int u = 0; u < kRun; ++u) now[u] = next[u];
        u32x4 x[kRun];
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            x[u] = (u32x4){0, 0, 0, 0};
            if (now[u].src < 0) continue;
            if (is_mass) x[u][0] = __float_as_uint(*mass_of(now[u].src));
            else x[u] = *(const u32x4 *)row_of(now[u].src);
        }
        if (base + run < a.budget) look_up(next, base + run);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // every value of the run is in a register
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if (now[u].src < 0) continue;
            if (is_mass) *mass_of(now[u].dst) = __uint_as_float(x[u][0]);
            else *(u32x4 *)row_of(now[u].dst) = x[u];
        }
    }
}

}  // namespace

hipError_t launch_kv_evict(const KvEvictArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "evict_pick_kernel";
    const int64_t heads = (int64_t)a.batch * a.n_kv, most = (int64_t)a.max_pages * a.page_size;
    const int room = (int)std::min<int64_t>(most, kMostKept);
    // 16 waves where that is one block a compute unit at most, else 8 (us with 16, with 8: 12 heads of up to 16001 tokens
    // 37.6, 42.5; one of 30000 163, 177; 600 of 300 50.6, 47.8; 1024 of 2000 259, 250)
    const bool wide = heads <= 256;
    if (room > 8192) {                   // more than a block has unasked
        const hipError_t e = hipFuncSetAttribute(wide ? (const void *)evict_pick_kernel<1024> : (const void *)evict_pick_kernel<512>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, room * 4);
        if (e != hipSuccess) return e;
    }
    if (wide) hipLaunchKernelGGL((evict_pick_kernel<1024>), dim3((unsigned)heads), dim3(1024), (size_t)room * 4, stream, a, room);
    else hipLaunchKernelGGL((evict_pick_kernel<512>), dim3((unsigned)heads), dim3(512), (size_t)room * 4, stream, a, room);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || most <= a.budget) return e;
    *kernel_name = "evict_move_kernel";
    // slices of 32 bytes and more of a row, until there are 512 moves of k (on blocks of 4 waves): 256 heads of 2900 tokens of 256 bytes 162 us whole, 179 in
    // halves, 215 in quarters; 512 heads of 4096 532 whole and 476 in halves; 32 heads of 500 within 10% of one another
    int slices = 1;
    while (slices * 4 <= a.row_bytes / 16 && heads * slices < 512) slices *= 2;
    const dim3 grid((unsigned)(heads * (2 * slices + 1)));
    // 16 waves where requests keep many runs of 4 (us with 4, with 16: 64 requests of 8 heads, 4160 -> 4096 tokens 529, 479 (of random mass, from a new cache); one of
    // 8192 -> 8000 79, 68; one head of 30000 -> 29000 163, 113; 16 requests of 2000 -> 1900 90, 88; 8 of 2000 -> 1000 54, 58;
    // 300 of 300 -> 256 49, 61)
    if (a.budget >= 2048) hipLaunchKernelGGL((evict_move_kernel<1024>), grid, dim3(1024), 0, stream, a, slices);
    else hipLaunchKernelGGL((evict_move_kernel<256>), grid, dim3(256), 0, stream, a, slices);
    return hipGetLastError();
}

}  // namespace ssm
