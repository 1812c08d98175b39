// kda_q8.cuh -- 8-bit storage of the recurrent state, shared by the pool's store / load kernels
// and the decode step that works on the pool.
//
// The state of one (sequence, 128-wide value unit) is 128 rows (value columns j) of 128 keys.  A
// row x is stored as 128 codes of one byte and one f32 scale:
//     amax = max_i |x_i|,   scale = amax / M,   code_i = round(x_i * (M / amax)),
// read back as x_i = code_i * scale, with M = 127 and codes rounded to the nearest whole number
// (ties to even) for int8, and M = 448 (the largest finite e4m3 value) and codes rounded to the
// nearest e4m3 value for e4m3.  Both quotients are IEEE divisions in f32 and the products are
// single f32 roundings, so the codes of a row are one exact function of its f32 values, on the
// device or anywhere else.  (A decode step, whose new state nobody else sees, rounds an int8 code
// once, from the exact product.)  An int8 code is off by at most half a step, amax / 254 for every
// element of the row; an e4m3 code by at most 2^-4 of the element (and amax * 2^-10 / 448 below
// the normal range): int8 is the finer one for rows without outliers.
// A row with amax below 2^-100 (where M / amax would leave the normal range) is stored as zeros
// with scale 0; a row that holds a NaN or an infinity gets scale NaN and codes 0, so it reads back
// as NaN throughout.
#pragma once

#include <cuda_fp8.h>

#include "kda_device.cuh"

namespace kda {

template <int FMT>
__device__ __forceinline__ float q8_max() { return FMT == kQ8E4m3 ? 448.0f : 127.0f; }

// Magnitude bits of x: ordered like |x| for finite values, above 0x7f7fffff for inf and NaN, so
// that an integer maximum over a row also finds non-finite elements.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The larger magnitude of two values, with either sign, or a NaN if one of them is (as bits without
// the sign: above every finite value and above inf, so that an integer maximum keeps it).
__device__ __forceinline__ float mag_max(float a, float b) {
    float m;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The largest magnitude of three, without a sign (NaN as above).
__device__ __forceinline__ float mag_max3(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Row scale and multiplier from the row's largest magnitude bits.
template <int FMT>
__device__ __forceinline__ void q8_row(uint32_t amax_bits, float& scale, float& mul) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) {
        scale = __uint_as_float(0x7fc00000u);
        mul = 0.0f;
    } else if (amax_bits < 0x0d800000u) {        // 2^-100
        scale = 0.0f;
        mul = 0.0f;
    } else {
        scale = __fdiv_rn(amax, q8_max<FMT>());
        mul = __fdiv_rn(q8_max<FMT>(), amax);
    }
}

// The scale or the multiplier of q8_row: one division, for lanes that share the two out.
template <int FMT>
__device__ __forceinline__ float q8_row_part(uint32_t amax_bits, bool want_mul) {
    const float amax = __uint_as_float(amax_bits);
    const float q = __fdiv_rn(want_mul ? q8_max<FMT>() : amax, want_mul ? amax : q8_max<FMT>());
    if (amax_bits >= 0x7f800000u) return want_mul ? 0.0f : __uint_as_float(0x7fc00000u);
    return amax_bits < 0x0d800000u ? 0.0f : q;
}

// Four codes as one word, element 0 in the low byte.  mul = 0 gives four zero codes whatever the
// elements are (a NaN or an infinity times 0 would not).
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4(float4 x, float mul) {
    uint32_t w;
    if constexpr (FMT == kQ8E4m3) {
        const float2 m2 = make_float2(mul, mul);
        const float2 lo = __fmul2_rn(make_float2(x.x, x.y), m2), hi = __fmul2_rn(make_float2(x.z, x.w), m2);
        const uint32_t l = __nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3);
        const uint32_t h = __nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3);
        w = __byte_perm(l, h, 0x5410);
    } else {
        // |x * mul| <= 127 (1 + 2^-23): adding 1.5 * 2^23 rounds it to the nearest whole number,
        // ties to even, in the low bits of the sum, whose low byte is the two's complement code.
        // (Not paired: the paired multiply and add were fused into one rounding.)
        const float big = 12582912.0f;
        const uint32_t a = __float_as_uint(__fadd_rn(__fmul_rn(x.x, mul), big));
        const uint32_t b = __float_as_uint(__fadd_rn(__fmul_rn(x.y, mul), big));
        const uint32_t c = __float_as_uint(__fadd_rn(__fmul_rn(x.z, mul), big));
        const uint32_t d = __float_as_uint(__fadd_rn(__fmul_rn(x.w, mul), big));
        w = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    return mul != 0.0f ? w : 0u;
}

// The same for values that are nobody's but the caller's (a decode step's new state): int8 codes are
// rounded once, from the exact product.
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4_once(float4 x, float mul) {
    if constexpr (FMT == kQ8E4m3) return q8_encode4<FMT>(x, mul);
    const float2 m2 = make_float2(mul, mul), big = make_float2(12582912.0f, 12582912.0f);
    const float2 lo = __ffma2_rn(make_float2(x.x, x.y), m2, big), hi = __ffma2_rn(make_float2(x.z, x.w), m2, big);
    const uint32_t w = __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                                   __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
    return mul != 0.0f ? w : 0u;
}

// The values of four codes times their row's scale.
template <int FMT>
__device__ __forceinline__ float4 q8_decode4(uint32_t w, float scale) {
    float4 v;
    if constexpr (FMT == kQ8E4m3) {
        const __half2_raw h0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(h0)), b = __half22float2(__half2(h1));
        v = make_float4(a.x, a.y, b.x, b.y);
    } else {
        // code + 128 under the exponent of 2^23, then minus (2^23 + 128): exact
        const uint32_t u = w ^ 0x80808080u;
        const float2 base = make_float2(-8388736.0f, -8388736.0f);
        const float2 a = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                                                __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), base);
        const float2 b = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)),
                                                __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), base);
        v = make_float4(a.x, a.y, b.x, b.y);
    }
    const float2 s2 = make_float2(scale, scale);
    const float2 lo = __fmul2_rn(make_float2(v.x, v.y), s2), hi = __fmul2_rn(make_float2(v.z, v.w), s2);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// Whether batch row m, with slots im and om, keeps row n from writing slot `out`: it reads that slot,
// or writes it first.  Padding and rows with a slot past the pool do neither.
__device__ __forceinline__ bool pool_rows_clash(int im, int om, int n, int out, int m, int pool_rows) {
    return m != n && (unsigned)im < (unsigned)pool_rows && (unsigned)om < (unsigned)pool_rows &&
           (im == out || (m < n && om == out));
}

// The pool rows that batch row n reads and writes.  A negative slot is padding: the row is skipped.
// A slot past the pool, and an output slot that another row reads or an earlier row writes, raise
// the error word and the row is skipped too, so that no two blocks race on a slot.  Every thread of
// the warp calls it.
__device__ __forceinline__ bool pool_row_warp(const int* slots, const int* slots_out, int n, int N,
                                              int pool_rows, int* err, int& in, int& out) {
    const int lane = threadIdx.x & 31;
    in = slots ? slots[n] : n;
    out = slots_out ? slots_out[n] : in;
    const bool live = in >= 0 && out >= 0;
    bool bad = in >= pool_rows || out >= pool_rows;
    if (slots || slots_out) {
        for (int m = lane; m < N; m += 32) {
            const int im = slots ? slots[m] : m;
            bad |= pool_rows_clash(im, slots_out ? slots_out[m] : im, n, out, m, pool_rows);
        }
    }
    const bool any = __any_sync(0xffffffffu, live && bad);
    if (any && lane == 0 && err) atomicOr(err, kDevErrSlot);
    return live && !any;
}

}  // namespace kda
