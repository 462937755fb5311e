// kv_pages.hip -- one scheduling step of a paged key-value cache on the device:
// pages taken from and given back to a ring of free pages, and each new token's
// request, position and slot (ssm_kv_pages_step in include/ssm_attn.h).
//
// Everything follows from three running sums over the requests (pages needed,
// pages given back, tokens), and the pages a request takes are consecutive
// entries of the ring.  So every block forms the sums for itself (a few thousand
// additions at most, out of cache) and then works on its own share of the
// tokens and moved pages: one launch, no workspace, and no order between
// blocks.  Nothing that one block reads is written by another: a token's page is
// read from the table where its request held it before, and else from the ring
// entry that it is taken from; taken entries lie in [head, head + free) of the
// ring, given-back ones behind it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_launchers.hpp"

namespace ssm {
namespace {

constexpr int kNT = 512;            // threads of a block
constexpr int kWaves = kNT / 64;
constexpr int kTok = 4;             // consecutive tokens of a thread: one 16-byte store of each 32-bit output

struct Need {
    int have, want;                 // pages held and wanted
    int grow;                       // new tokens
    bool over;                      // wanted pages do not fit the table's row
};

__device__ __forceinline__ int pages_of(int len, uint32_t ps) { return (int)(((uint32_t)len + ps - 1) / ps); }

__device__ __forceinline__ Need need_of(const KvPagesArgs &a, int r) {
    const int lo = max(a.len_old[r], 0), hi = max(a.len_new[r], 0);
    Need n;
    n.have = min(pages_of(lo, a.page_size), a.max_pages);     // a longer row has no entries to read
    n.want = pages_of(hi, a.page_size);
    n.grow = max(hi - lo, 0);
    n.over = n.want > a.max_pages;
    return n;
}

// place i < 2 n of a ring of n entries
__device__ __forceinline__ int wrap(uint32_t i, uint32_t n) { return (int)(i >= n ? i - n : i); }

// inclusive sums over the block's threads; `total` (every thread) is the block's sum
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *part, T &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const T p = part[w];
        before += w < wave ? p : 0;
        total += p;
    }
    __syncthreads();
    return v + before;
}

// first i with end[i] > x (n if none): the request that item x belongs to
__device__ __forceinline__ int owner_of(const int *end, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kNT) kv_pages_kernel(KvPagesArgs a) {
    extern __shared__ int lds[];                       // three running sums of batch entries
    __shared__ int64_t part[kWaves];
    int *tok_end = lds, *take_end = lds + a.batch, *give_end = take_end + a.batch;
    const int total = a.n_pages;
    int head = a.ring[0] % total;
    head += head < 0 ? total : 0;
    const int free = min(max(a.ring[1], 0), total);
    const bool first = blockIdx.x == 0;

    int64_t needed = 0, grown = 0;                     // sums over the requests before this chunk
    int taken = 0, given = 0, denied = 0;
    for (int r0 = 0; r0 < a.batch; r0 += kNT) {
        const int r = r0 + (int)threadIdx.x;
        Need n = {0, 0, 0, false};
        if (r < a.batch) n = need_of(a, r);
        const int need = n.over ? 0 : max(n.want - n.have, 0);
        int64_t s_need, s_grow, s_take, s_give, s_deny;
        const int64_t upto = needed + block_scan<int64_t>(need, part, s_need);
        const bool refused = n.over || (need > 0 && upto > free);
        const int take = refused ? 0 : need;
        const int64_t ends = grown + block_scan<int64_t>(n.grow, part, s_grow);
        // sums below 2^31: taken <= free, given <= batch * max_pages
        const int t_end = taken + (int)block_scan<int64_t>(take, part, s_take);
        const int g_end = given + (int)block_scan<int64_t>(max(n.have - n.want, 0), part, s_give);
        block_scan<int64_t>(refused ? 1 : 0, part, s_deny);
        if (r < a.batch) {
            const int e = (int)min(ends, (int64_t)0x7fffffff);
            tok_end[r] = e;
            take_end[r] = t_end;
            give_end[r] = g_end;
            if (first) {
                a.len_out[r] = max(refused ? a.len_old[r] : a.len_new[r], 0);
                a.starts[r + 1] = e;
            }
        }
        needed += s_need; grown += s_grow;
        taken += (int)s_take; given += (int)s_give; denied += (int)s_deny;
    }
    given = min(given, total - free);                  // no more than the ring has places for
    if (first && threadIdx.x == 0) {
        a.starts[0] = 0;
        a.ring_out[0] = wrap((uint32_t)head + taken, total);
        a.ring_out[1] = free - taken + given;
        a.denied[0] = denied;
    }
    __syncthreads();
    const int tokens = a.batch > 0 ? tok_end[a.batch - 1] : 0;
    const uint32_t ps = (uint32_t)a.page_size;
    const int step = (int)gridDim.x * kNT, me = (int)blockIdx.x * kNT + (int)threadIdx.x;

    // the new tokens
    for (int64_t t0 = (int64_t)me * kTok; t0 < a.n_tokens; t0 += (int64_t)step * kTok) {
        int rq[kTok], po[kTok];
        int64_t sl[kTok];
        int r = t0 < tokens ? owner_of(tok_end, a.batch, (int)t0) : a.batch;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = (int)t0 + i;
            while (r < a.batch && tok_end[r] <= t) ++r;
            rq[i] = -1; po[i] = -1; sl[i] = -1;
            if (r < a.batch) {
                const Need n = need_of(a, r);
                const int before = r > 0 ? take_end[r - 1] : 0;
                rq[i] = r;
                po[i] = max(a.len_old[r], 0) + (t - (r > 0 ? tok_end[r - 1] : 0));
                const int c = (int)((uint32_t)po[i] / ps);
                // a request that wants more pages than it holds and takes none was refused
                if (c < n.have || take_end[r] > before) {
                    const int page = c < n.have ? a.block_table[r * a.table_stride + c]
                                                : a.free_ring[wrap((uint32_t)head + (before + c - n.have), total)];
                    sl[i] = (int64_t)page * ps + ((uint32_t)po[i] - (uint32_t)c * ps);
                }
                if (n.want > n.have && take_end[r] == before) sl[i] = -1;
            }
        }
        if (t0 + kTok <= a.n_tokens) {
            *(int4 *)(a.request + t0) = make_int4(rq[0], rq[1], rq[2], rq[3]);
            *(int4 *)(a.positions + t0) = make_int4(po[0], po[1], po[2], po[3]);
            *(longlong2 *)(a.slots + t0) = make_longlong2(sl[0], sl[1]);
            *(longlong2 *)(a.slots + t0 + 2) = make_longlong2(sl[2], sl[3]);
        } else {
            for (int i = 0; i < kTok && t0 + i < a.n_tokens; ++i) {
                a.request[t0 + i] = rq[i];
                a.positions[t0 + i] = po[i];
                a.slots[t0 + i] = sl[i];
            }
        }
    }
    // pages taken, into the table
    for (int j = me; j < taken; j += step) {
        const int r = owner_of(take_end, a.batch, j);
        const Need n = need_of(a, r);
        const int c = n.have + j - (r > 0 ? take_end[r - 1] : 0);
        a.block_table[r * a.table_stride + c] = a.free_ring[wrap((uint32_t)head + j, total)];
    }
    // pages given back, behind the ring's last entry
    for (int j = me; j < given; j += step) {
        const int r = owner_of(give_end, a.batch, j);
        const int c = need_of(a, r).want + j - (r > 0 ? give_end[r - 1] : 0);
        a.free_ring[wrap((uint32_t)head + (free + j), total)] = a.block_table[r * a.table_stride + c];
    }
}

}  // namespace

hipError_t launch_kv_pages(const KvPagesArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "kv_pages_kernel";
    const int64_t work = (a.n_tokens + kTok - 1) / kTok;
    int64_t blocks = (work + kNT - 1) / kNT;
    blocks = blocks < 8 ? 8 : blocks > 512 ? 512 : blocks;
    hipLaunchKernelGGL(kv_pages_kernel, dim3((unsigned)blocks), dim3(kNT), (size_t)a.batch * 3 * sizeof(int), stream, a);
    return hipGetLastError();
}

}  // namespace ssm
