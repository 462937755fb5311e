// topk.hpp -- the largest `want` of n keys by one block, ties to the lowest index, the chosen
// indexes in rising order.
//
// Keys are 32 bits whose order as whole numbers is the wanted one (key_of).  The want-th largest is
// found from the top 11 bits down (11, 11, 10): counts of the next bits' values among the keys that match so
// far, in shared memory, until a value's keys are wanted whole or all bits are known; counts of whole
// numbers do not depend on the order in which they are added.  (By 8 bits it would be four rounds, and the
// first, sign and most of the exponent, would add most keys of one magnitude to a few counters.)  A second pass counts, index by index, the keys above and equal, and so
// places the chosen ones in their order without a sort.
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
    int hist[2048];
    int sums[NT / 64], equal[NT / 64];
    int bin, left, whole;
};

// Where to cut: keys above `above` are chosen, and the first `ties` of those equal to it
struct Cut { int64_t above; int ties; };

// 0 < want <= n; every thread of the block calls it
template <int NT, typename Key>
__device__ __forceinline__ Cut find_cut(TopKShared<NT> &sh, int n, int want, Key key) {
    constexpr int B = 2048 / NT, W = NT / 64;     // counters of a thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t prefix = 0, mask = 0;
#pragma unroll
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
        const uint32_t digit = round == 2 ? 1023u : 2047u;
#pragma unroll
        for (int i = 0; i < B; ++i) sh.hist[i * NT + tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += NT) {
            const uint32_t k = key(i);
            if ((k & mask) == prefix) atomicAdd(&sh.hist[k >> shift & digit], 1);
        }
        __syncthreads();
        int c[B], own = 0;                        // thread 0 has the highest values
#pragma unroll
        for (int i = 0; i < B; ++i) own += c[i] = sh.hist[2047 - B * tid - i];
        int before = wave_scan(own);
        if (lane == 63) sh.sums[wave] = before;
        before -= own;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) before += w < wave ? sh.sums[w] : 0;
        if (before < want && want <= before + own) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (before < want && want <= before + c[i]) {
                    sh.bin = 2047 - B * tid - i;
                    sh.left = want - before;
                    sh.whole = c[i] == want - before;
                }
                before += c[i];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh.bin << shift;
        mask |= digit << shift;
        want = sh.left;
        if (sh.whole) return {(int64_t)prefix - 1, 0};
    }
    return {(int64_t)prefix, want};
}

// Calls put(place, i) for every chosen index i; places rise with i, from 0 on.  A wave has consecutive
// indexes, 64 at a time, counts them, and goes over them again once it knows what stands before them.
template <int NT, typename Key, typename Put>
__device__ __forceinline__ void put_chosen(TopKShared<NT> &sh, int n, Cut cut, Key key, Put put) {
    constexpr int W = NT / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int part = (n + NT - 1) / NT * 64, i0 = wave * part, i1 = min(i0 + part, n);
    const uint64_t lower = (uint64_t(1) << lane) - 1;
    int above = 0, equal = 0;
#pragma unroll 4
    for (int i = i0 + lane; i - lane < i1; i += 64) {
        const int64_t k = i < i1 ? (int64_t)key(i) : -2;
        above += __popcll(__ballot(k > cut.above));
        equal += __popcll(__ballot(k == cut.above));
    }
    if (lane == 0) { sh.sums[wave] = above; sh.equal[wave] = equal; }
    __syncthreads();
    above = equal = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        above += w < wave ? sh.sums[w] : 0;
        equal += w < wave ? sh.equal[w] : 0;
    }
#pragma unroll 4
    for (int i = i0 + lane; i - lane < i1; i += 64) {
        const int64_t k = i < i1 ? (int64_t)key(i) : -2;
        const uint64_t a = __ballot(k > cut.above), e = __ballot(k == cut.above);
        const int mine = equal + __popcll(e & lower), place = above + __popcll(a & lower) + min(mine, cut.ties);
        if (k > cut.above || (k == cut.above && mine < cut.ties)) put(place, i);
        above += __popcll(a);
        equal += __popcll(e);
    }
}

}  // namespace ssm
