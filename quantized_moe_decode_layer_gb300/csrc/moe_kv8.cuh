// Shared device code of the 8-bit key/value cache (moe_kv8*.cu).
//
// A cached value is code * 2^e: an 8-bit code (int8 or e4m3) and one step
// 2^e per block of positions of a head, kept as fp32.  Steps are powers of
// two so that rounding a code again to a step it has had, or a smaller one, is
// exact, and to a larger one only drops bits.  int8: half steps that at least double
// add up to less than the last, so a value that was rounded again any number of
// times (a growing block, eviction) is within one step, the largest it has had, of
// what was appended.  e4m3: the first rounding is off by 2^-4 of the value at most, and a
// larger step costs only what falls below 2^-6 steps, where codes are 2^-9 apart: halves
// of that add up to less than 2^-9 steps.  With arbitrary scales each
// rounding would add its own half step (or 2^-4).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "moe_kv8.h"

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

// Four values in units of the step (at most 127.5 or 448 of them) to four
// codes (bytes 0 .. 3), nearest, ties to even.  int8: adding 1.5 2^23 leaves
// the rounded value in the low mantissa bits.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if (FMT == MOE_KV8_INT8) {
        auto r = [](float x) { return __float_as_uint(__fadd_rn(fminf(fmaxf(x, -127.f), 127.f), 12582912.f)); };
        return __byte_perm(__byte_perm(r(a), r(b), 0x0040), __byte_perm(r(c), r(d), 0x0040), 0x5410);
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Codes to fp16 pairs, exactly.  pairs(w): (byte 0, byte 2) and (byte 1, byte
// 3) for int8 -- fp16 0x6400 | u is 1024 + u, so flipping a code's top bit
// gives 1024 + 128 + code, and one subtraction is exact --, (0, 1) and (2, 3)
// for e4m3.
template <int FMT>
__device__ __forceinline__ void pairs(uint32_t w, uint32_t &x, uint32_t &y)
{
    if (FMT == MOE_KV8_INT8) {
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        uint32_t a, b;                                // (w & mask) ^ flip
        asm("lop3.b32 %0, %1, 0x00FF00FF, %2, 0x6A;" : "=r"(a) : "r"(w), "r"(0x64806480u));
        asm("lop3.b32 %0, %1, 0x00FF00FF, %2, 0x6A;" : "=r"(b) : "r"(w >> 8), "r"(0x64806480u));
        const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&a), off), hb = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        x = *reinterpret_cast<const uint32_t *>(&ha);
        y = *reinterpret_cast<const uint32_t *>(&hb);
    } else {
        asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
            : "=r"(x), "=r"(y) : "r"(w));
    }
}

// Two fp32 numbers to bf16, low and high half, nearest; past the largest finite
// number that number (a code of a block of the largest steps may stand for 2^128).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

// Four codes to four values in units of the step.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4])
{
    uint32_t x, y;
    pairs<FMT>(w, x, y);
    const float2 a = __half22float2(as_half2(x)), b = __half22float2(as_half2(y));
    v[0] = a.x;
    v[1] = FMT == MOE_KV8_INT8 ? b.x : a.y;
    v[2] = FMT == MOE_KV8_INT8 ? a.y : b.x;
    v[3] = b.y;
}

// 4 codes in units of one step to units of another: times ratio, a power of
// two of at most 2^17 (that many times, no code of such a block can be
// larger: the new step holds the block's largest).
template <int FMT>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio)
{
    if (FMT == MOE_KV8_INT8) {
        // in fp16: code * ratio + 1536 is rounded once, to the integer in its
        // low byte; below 2^-14 every code rounds to 0 as it does at 2^-14,
        // and above 2^7 there are only zeros
        const __half2 r = __float2half2_rn(fminf(fmaxf(ratio, 6.103515625e-05f), 128.f)), magic = __float2half2_rn(1536.f);
        uint32_t x, y;
        pairs<FMT>(w, x, y);
        const __half2 a = __hfma2(as_half2(x), r, magic), b = __hfma2(as_half2(y), r, magic);
        return __byte_perm(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b), 0x6240);
    }
    float v[4];
    decode4<FMT>(w, v);
    return encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
}
template <int FMT>
__device__ __forceinline__ uint2 recode8(uint2 w, float ratio)
{
    return make_uint2(recode4<FMT>(w.x, ratio), recode4<FMT>(w.y, ratio));
}

// Largest magnitude of 8 codes, in units of their step.
template <int FMT>
__device__ __forceinline__ float amax8(uint2 w)
{
    uint32_t a, b, c, d;
    pairs<FMT>(w.x, a, b);
    pairs<FMT>(w.y, c, d);
    const __half2 m = __hmax2(__hmax2(__habs2(as_half2(a)), __habs2(as_half2(b))), __hmax2(__habs2(as_half2(c)), __habs2(as_half2(d))));
    return fmaxf(__low2float(m), __high2float(m));
}

// Every kernel of the cache is launched as a dependent of the one before it on
// the stream: its CTAs may be placed while that one ends.  A call's first
// kernel waits before anything else, and only then lets the next be placed
// (after_previous); so when a call's later kernel runs, whatever came before
// the call is complete, and it may read the call's inputs ahead of its own
// wait (wait_for_previous) for what the call's earlier kernels write.  No CTA
// leaves without the wait: a kernel's end means the end of all before it.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void place_next() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void after_previous()
{
    wait_for_previous();
    place_next();
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace moe
