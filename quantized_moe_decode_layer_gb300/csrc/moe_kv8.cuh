// Shared device code of the 8-bit key/value cache (moe_kv8*.cu).
//
// A cached value is code * 2^e: an 8-bit code (int8 or e4m3) and one step
// 2^e per block of positions of a head, kept as fp32.  Steps are powers of
// two so that rounding a code again to the same step is exact, and to a
// larger one only drops bits: half steps that at least double add up to less
// than one last step, so a value that was rounded again any number of times
// (a growing block, eviction) is within one step of what was appended.  With
// arbitrary scales each rounding would add its own half step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {

// Status bits of the calls' err word.
constexpr int kKv8ErrRange = 1;       // a position, length or count outside the cache
constexpr int kKv8ErrNonFinite = 2;   // an infinity or NaN was appended

constexpr int kKv8MinExp = -126;      // steps are normal fp32 numbers

// Rows of sequence b that a call works on: 0 for an idle one (pos < 0).
// Sets *bad when the call asks for more than the cache holds.
__device__ __forceinline__ int kv8_rows(const int32_t *pos, const int32_t *counts, int b, int M, int T_cap, int &p0, bool &bad)
{
    p0 = pos[b];
    bad = false;
    if (p0 < 0) return 0;
    int n = counts ? counts[b] : M;
    bad = n < 0 || n > M;
    n = max(0, min(n, M));
    if (p0 > T_cap - n) {             // no overflow: n <= M <= T_cap is checked on the host
        bad = bad || n > 0;
        n = max(0, T_cap - p0);
    }
    return n;
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// Exponent of the smallest step (>= 2^-126) in whose units a rounds to a
// code: a <= 127.5 steps for int8 (127.5 itself becomes 127, half a step
// off as any rounding may be), a <= 448 steps for e4m3.  a finite, >= 0.
template <int FMT>
__device__ __forceinline__ int step_exp(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int x = (int)(u >> 23) - 126;   // a = m 2^x, 1/2 <= m < 1 (normal a)
    const uint32_t f = u & 0x7FFFFFu;
    const int e = FMT == MOE_KV8_INT8 ? x - (f <= 0x7F0000u ? 7 : 6) : x - (f <= 0x600000u ? 9 : 8);
    return max(e, kKv8MinExp);
}

// Four values in units of the step to four codes (bytes 0 .. 3), nearest, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if (FMT == MOE_KV8_INT8) {
        const int ia = max(-127, min(127, __float2int_rn(a))), ib = max(-127, min(127, __float2int_rn(b)));
        const int ic = max(-127, min(127, __float2int_rn(c))), id = max(-127, min(127, __float2int_rn(d)));
        return __byte_perm(__byte_perm((uint32_t)ia, (uint32_t)ib, 0x0040), __byte_perm((uint32_t)ic, (uint32_t)id, 0x0040), 0x5410);
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Four codes to four values in units of the step (exact in fp16).
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4])
{
    if (FMT == MOE_KV8_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
    } else {
        uint32_t lo, hi;
        asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
            : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
}

// 8 codes in units of one step to a larger one: down = 2^(e_old - e_new).
template <int FMT>
__device__ __forceinline__ uint2 recode8(uint2 w, float down)
{
    float a[4], b[4];
    decode4<FMT>(w.x, a);
    decode4<FMT>(w.y, b);
    return make_uint2(encode4<FMT>(a[0] * down, a[1] * down, a[2] * down, a[3] * down),
                      encode4<FMT>(b[0] * down, b[1] * down, b[2] * down, b[3] * down));
}

// Largest magnitude of 8 codes, in units of their step.
template <int FMT>
__device__ __forceinline__ float amax8(uint2 w)
{
    float a[4], b[4];
    decode4<FMT>(w.x, a);
    decode4<FMT>(w.y, b);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
    return m;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Maximum over a CTA of up to 32 warps; `red` holds 33 floats.
__device__ __forceinline__ float cta_max(float v, float *red)
{
    v = warp_max(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        v = warp_max(lane < nw ? red[lane] : -INFINITY);
        if (lane == 0) red[32] = v;
    }
    __syncthreads();
    return red[32];
}

}  // namespace moe
