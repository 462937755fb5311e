// kv_pages.hip -- one scheduling step of a paged key-value cache on the device:
// pages taken from and given back to a ring of free pages, and each new token's
// request, position and slot (ssm_kv_pages_step in include/ssm_attn.h).
//
// Everything follows from three running sums over the requests (pages needed,
// pages given back, new tokens), and the pages that requests take are consecutive
// entries of the ring: request r takes up to place min(sum of the needs up to it, T),
// where T is the largest such sum that the free pages cover.  So every block forms the
// sums for itself (one pass over the lengths, a scan in registers and one wait) and then
// works on its own share of the tokens and moved pages: one launch, no workspace, and no
// order between blocks.  Nothing that one block reads is written by another: a token's
// page is read from the table where its request held it before, and else from the ring
// entry that it is taken from; taken entries lie in [head, head + free) of the
// ring, given-back ones behind it.
//
// Bound: latency (lengths -> sums -> table or ring -> stores), and for long prompts the 16
// bytes stored a token.  Measured, kernel alone: one token for each of 256 requests 5.8 us; prompts
// of up to 2048 tokens for 512 requests, a quarter of them refused, 8.6 MB of outputs, 6.8 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_launchers.hpp"

namespace ssm {
namespace {

constexpr int kNT = 256;            // threads of a block
constexpr int kWaves = kNT / 64;
constexpr int kKeep = 2;            // requests of a thread whose lengths stay in registers
constexpr int kTok = 4;             // consecutive tokens of a thread: one 16-byte store of each 32-bit output

// x / page size, by a shift where that is a power of two
struct Pages {
    uint32_t size;
    int shift;                      // -1: none
    __device__ __forceinline__ explicit Pages(uint32_t n) : size(n), shift((n & (n - 1)) == 0 ? 31 - __clz(n) : -1) {}
    __device__ __forceinline__ int of(uint32_t x) const { return (int)(shift >= 0 ? x >> shift : x / size); }
    __device__ __forceinline__ int to_hold(int len) const { return of((uint32_t)len + size - 1); }
};

struct Need {
    int have, want;                 // pages held and wanted
    int grow;                       // new tokens
    bool over;                      // wanted pages do not fit the table's row
    __device__ __forceinline__ int take() const { return over ? 0 : max(want - have, 0); }
    __device__ __forceinline__ int give() const { return max(have - want, 0); }
};

__device__ __forceinline__ Need need_of(const KvPagesArgs &a, const Pages &pages, int lo, int hi) {
    Need n;
    n.have = min(pages.to_hold(lo), a.max_pages);     // a longer row has no entries to read
    n.want = pages.to_hold(hi);
    n.grow = max(hi - lo, 0);
    n.over = n.want > a.max_pages;
    return n;
}
__device__ __forceinline__ Need need_of(const KvPagesArgs &a, const Pages &pages, int r) {
    return need_of(a, pages, max(a.len_old[r], 0), max(a.len_new[r], 0));
}

// place i < 2 n of a ring of n entries
__device__ __forceinline__ int wrap(uint32_t i, uint32_t n) { return (int)(i >= n ? i - n : i); }

// inclusive sums over a wave: within rows of 16 lanes, then the rows' last lanes onward
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp_i(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true); }
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int64_t dpp_i(int64_t v) {
    const uint32_t lo = (uint32_t)dpp_i<CTRL, ROWS>((int)(uint32_t)v), hi = (uint32_t)dpp_i<CTRL, ROWS>((int)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    v += dpp_i<0x111>(v);
    v += dpp_i<0x112>(v);
    v += dpp_i<0x114>(v);
    v += dpp_i<0x118>(v);
    v += dpp_i<0x142, 0xa>(v);
    v += dpp_i<0x143, 0xc>(v);
    return v;
}
// the largest of a wave's values >= 0, in lane 63
__device__ __forceinline__ int wave_max(int v) {
    v = max(v, dpp_i<0x111>(v));
    v = max(v, dpp_i<0x112>(v));
    v = max(v, dpp_i<0x114>(v));
    v = max(v, dpp_i<0x118>(v));
    v = max(v, dpp_i<0x142, 0xa>(v));
    v = max(v, dpp_i<0x143, 0xc>(v));
    return v;
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
    __shared__ int sum_need[kWaves], sum_give[kWaves], most[kWaves], refusals[kWaves];
    __shared__ int64_t sum_grow[kWaves];
    int *tok_end = lds, *need_end = lds + a.batch, *give_end = need_end + a.batch;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Pages pages((uint32_t)a.page_size);
    const int total = a.n_pages;
    const bool first = blockIdx.x == 0;

    // a thread's requests [r0, r1), their sums, and the sums before them
    const int mine = (a.batch + kNT - 1) / kNT, r0 = tid * mine, r1 = min(r0 + mine, a.batch);
    int lo[kKeep], hi[kKeep];                          // their lengths, where they are few
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int r = min(r0 + i, a.batch - 1);
        lo[i] = max(a.len_old[r], 0);
        hi[i] = max(a.len_new[r], 0);
    }
    int head = a.ring[0];
    const int free = min(max(a.ring[1], 0), total);
    if (head < 0 || head >= total) {
        head %= total;
        head += head < 0 ? total : 0;
    }
    auto each = [&](auto f) {
        if (mine <= kKeep) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (r0 + i < r1) f(r0 + i, lo[i], hi[i], need_of(a, pages, lo[i], hi[i]));
        } else {
            for (int r = r0; r < r1; ++r) {
                const int l = max(a.len_old[r], 0), h = max(a.len_new[r], 0);
                f(r, l, h, need_of(a, pages, l, h));
            }
        }
    };
    int need = 0, give = 0;                            // below 2^31: at most batch * max_pages
    int64_t grow = 0;
    each([&](int, int, int, const Need &n) {
        need += n.take();
        give += n.give();
        grow += n.grow;
    });
    int need_upto = wave_scan(need), give_upto = wave_scan(give);
    int64_t grow_upto = wave_scan(grow);
    if (lane == 63) { sum_need[wave] = need_upto; sum_give[wave] = give_upto; sum_grow[wave] = grow_upto; }
    __syncthreads();
    need_upto -= need; give_upto -= give; grow_upto -= grow;
    int given = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) { need_upto += sum_need[w]; give_upto += sum_give[w]; grow_upto += sum_grow[w]; }
        given += sum_give[w];
    }
    int top = 0, denied = 0;                           // the largest need up to a request that is covered
    each([&](int r, int l, int h, const Need &n) {
        need_upto += n.take();
        give_upto += n.give();
        grow_upto += n.grow;
        const int e = (int)min(grow_upto, (int64_t)0x7fffffff);
        tok_end[r] = e;
        need_end[r] = need_upto;
        give_end[r] = give_upto;
        top = need_upto <= free ? need_upto : top;
        if (first) {
            const bool refused = n.over || (n.take() > 0 && need_upto > free);
            denied += refused;
            a.len_out[r] = refused ? l : h;
            a.starts[r + 1] = e;
        }
    });
    top = wave_max(top);
    denied = wave_scan(denied);
    if (lane == 63) { most[wave] = top; refusals[wave] = denied; }
    __syncthreads();
    int taken = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) taken = max(taken, most[w]);
    given = min(given, total - free);                  // no more than the ring has places for
    if (first && tid == 0) {
        a.starts[0] = 0;
        a.ring_out[0] = wrap((uint32_t)head + taken, total);
        a.ring_out[1] = free - taken + given;
        int d = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) d += refusals[w];
        a.denied[0] = d;
    }
    const int tokens = tok_end[a.batch - 1];
    const int step = (int)gridDim.x * kNT, me = (int)blockIdx.x * kNT + tid;

    // the new tokens
    for (int64_t t0 = (int64_t)me * kTok; t0 < a.n_tokens; t0 += (int64_t)step * kTok) {
        int rq[kTok], po[kTok];
        int64_t sl[kTok];
        int r = t0 < tokens ? owner_of(tok_end, a.batch, (int)t0) : a.batch, end = 0;
        int old = 0, start = 0, have = 0, from = 0;    // of request r: its length and first token; its
        bool granted = false;                          // pages and first taken one; not refused
        const int32_t *table = nullptr;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = (int)t0 + i;
            rq[i] = -1; po[i] = -1; sl[i] = -1;
            if (r < a.batch && t >= end) {             // the next request with new tokens
                while (r < a.batch && tok_end[r] <= t) ++r;
                if (r < a.batch) {
                    const Need n = need_of(a, pages, r);
                    end = tok_end[r];
                    start = r > 0 ? tok_end[r - 1] : 0;
                    from = r > 0 ? min(need_end[r - 1], taken) : 0;
                    old = max(a.len_old[r], 0);
                    have = n.have;
                    // one that wants more pages than it holds and takes none was refused
                    granted = n.want <= n.have || min(need_end[r], taken) > from;
                    table = a.block_table + r * a.table_stride;
                }
            }
            if (r < a.batch) {
                rq[i] = r;
                po[i] = old + (t - start);
                if (granted) {
                    const int c = pages.of((uint32_t)po[i]);
                    const int page = c < have ? table[c] : a.free_ring[wrap((uint32_t)head + (from + c - have), total)];
                    sl[i] = (int64_t)page * pages.size + ((uint32_t)po[i] - (uint32_t)c * pages.size);
                }
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
    // pages taken, into the table (by the last threads first: where there is little to do,
    // these moves and the tokens are at work at the same time)
    for (int j = step - 1 - me; j < taken; j += step) {
        const int r = owner_of(need_end, a.batch, j);
        const Need n = need_of(a, pages, r);
        const int c = n.have + j - (r > 0 ? need_end[r - 1] : 0);
        a.block_table[r * a.table_stride + c] = a.free_ring[wrap((uint32_t)head + j, total)];
    }
    // pages given back, behind the ring's last entry
    for (int j = me < step / 2 ? me + step / 2 : me - step / 2; j < given; j += step) {
        const int r = owner_of(give_end, a.batch, j);
        const int c = need_of(a, pages, r).want + j - (r > 0 ? give_end[r - 1] : 0);
        a.free_ring[wrap((uint32_t)head + (free + j), total)] = a.block_table[r * a.table_stride + c];
    }
}

}  // namespace

hipError_t launch_kv_pages(const KvPagesArgs &a, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "kv_pages_kernel";
    const int64_t work = (a.n_tokens + kTok - 1) / kTok;
    // a thread for 4 tokens; a block a request, for the pages that it may give back or take, of
    // which the host does not know how many there are: 256 requests with 86 of 125 pages each
    // ending 10.4 us on 8 blocks, 6.5 us on 256
    int64_t blocks = (work + kNT - 1) / kNT;
    blocks = blocks < a.batch ? a.batch : blocks;
    blocks = blocks < 8 ? 8 : blocks > 512 ? 512 : blocks;
    hipLaunchKernelGGL(kv_pages_kernel, dim3((unsigned)blocks), dim3(kNT), (size_t)a.batch * 3 * sizeof(int), stream, a);
    return hipGetLastError();
}

}  // namespace ssm
