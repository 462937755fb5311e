// attn_device.hpp -- small gfx950 device helpers shared by the kernels over a paged
// key-value cache: cache types, matrix instructions, 8-bit and bf16 conversions, sums
// over the lanes of a wave.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum { KBF16, KF8, KF32 };          // types of a cache

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);   // to nearest even
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// two 8-bit values -> two bf16, exact
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
    return __builtin_bit_cast(uint32_t, r);
}
// bytes of lo (0-3) and hi (4-7) picked by sel
__device__ __forceinline__ uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) {
    return __builtin_amdgcn_perm(hi, lo, sel);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp_i(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true); }
// inclusive sums over a wave: within rows of 16 lanes, then the rows' last lanes onward
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp_i<0x111>(v);
    v += dpp_i<0x112>(v);
    v += dpp_i<0x114>(v);
    v += dpp_i<0x118>(v);
    v += dpp_i<0x142, 0xa>(v);
    v += dpp_i<0x143, 0xc>(v);
    return v;
}
// over the four lanes that hold a head
__device__ __forceinline__ float head_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float head_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <int N> struct Words { uint32_t w[N]; };
template <int N>
__device__ __forceinline__ Words<N> ld_words(const char *p) {
    Words<N> r;
    if constexpr (N == 4) {
        const uint4 u = *(const uint4 *)p;
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *(const uint2 *)p;
        r.w[0] = u.x; r.w[1] = u.y;
    } else {
        r.w[0] = *(const uint32_t *)p;
    }
    return r;
}

// x / page size, by a shift where that is a power of two
struct PageSize {
    uint32_t size;
    int shift;                      // -1: none
    __device__ __forceinline__ explicit PageSize(int n) : size((uint32_t)n), shift((n & (n - 1)) == 0 ? 31 - __clz(n) : -1) {}
    __device__ __forceinline__ int of(int x) const { return (int)(shift >= 0 ? (uint32_t)x >> shift : (uint32_t)x / size); }
    __device__ __forceinline__ int place(int x, int page) const { return x - page * (int)size; }     // page = of(x)
    __device__ __forceinline__ int to_hold(int len) const { return of(len + (int)size - 1); }
};

}  // namespace ssm
