// topk.hpp -- the largest `want` of n keys by one block, ties to the lowest index, the chosen
// indexes in rising order.
//
// Keys are 32 bits whose order as whole numbers is the wanted one (key_of).  The want-th largest is
// found from the top byte down: counts of the next byte's values among the keys that match so far, in
// shared memory, until a value's keys are wanted whole or all four bytes are known; counts of whole
// numbers do not depend on the order in which they are added.  A second pass counts, index by index,
// the keys above and equal, and so places the chosen ones in their order without a sort.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_device.hpp"

namespace ssm {

// order of floats as whole numbers: -0 as 0, NaN above all
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    if (x != x) return 0xffffffffu;
    return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyLowest = 0x007fffffu;      // of -inf

template <int NT>
struct TopKShared {
    int hist[256];
    int sums[NT / 64];
    int bin, left, whole;
};

// Where to cut: keys above `above` are chosen, and the first `ties` of those equal to it
struct Cut { int64_t above; int ties; };

// 0 < want <= n; every thread of the block calls it
template <int NT, typename Key>
__device__ __forceinline__ Cut find_cut(TopKShared<NT> &sh, int n, int want, Key key) {
    const int tid = threadIdx.x, lane = tid & 63;
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += NT) sh.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += NT) {
            const uint32_t k = key(i);
            if ((k & mask) == prefix) atomicAdd(&sh.hist[k >> shift & 255], 1);
        }
        __syncthreads();
        if (tid < 64) {                           // lane 0 has the highest values
            int c[4], own = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) own += c[i] = sh.hist[255 - 4 * lane - i];
            int before = wave_scan(own) - own;
            if (before < want && want <= before + own) {
                int i = 0;
                while (before + c[i] < want) before += c[i++];
                sh.bin = 255 - 4 * lane - i;
                sh.left = want - before;
                sh.whole = c[i] == want - before;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh.bin << shift;
        mask |= 0xffu << shift;
        want = sh.left;
        if (sh.whole) return {(int64_t)prefix - 1, 0};
    }
    return {(int64_t)prefix, want};
}

// Calls put(place, i) for every chosen index i; places rise with i, from 0 on.
template <int NT, typename Key, typename Put>
__device__ __forceinline__ void put_chosen(TopKShared<NT> &sh, int n, Cut cut, Key key, Put put) {
    constexpr int V = 4, W = NT / 64;             // consecutive indexes of a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int above = 0, equal = 0;                     // before this round's indexes
    for (int base = 0; base < n; base += NT * V) {
        uint32_t k[V];
        int own = 0;                              // keys above in the low half, equal ones in the high half
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + tid * V + v;
            k[v] = i < n ? key(i) : 0u;
            if (i < n) own += ((int64_t)k[v] > cut.above ? 1 : 0) + ((int64_t)k[v] == cut.above ? 1 << 16 : 0);
        }
        int at = wave_scan(own);
        if (lane == 63) sh.sums[wave] = at;
        at -= own;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            at += w < wave ? sh.sums[w] : 0;
            all += sh.sums[w];
        }
        int a = above + (at & 0xffff), e = equal + (at >> 16);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = base + tid * V + v;
            if (i >= n) break;
            if ((int64_t)k[v] > cut.above) {
                put(a + min(e, cut.ties), i);
                ++a;
            } else if ((int64_t)k[v] == cut.above) {
                if (e < cut.ties) put(a + e, i);
                ++e;
            }
        }
        above += all & 0xffff;
        equal += all >> 16;
        __syncthreads();                          // readers of sums
    }
}

}  // namespace ssm
