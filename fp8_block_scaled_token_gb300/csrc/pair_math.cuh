// pair_math.cuh -- numbers held as the sum of two fp32 numbers, for decisions
// that fp32 alone is too coarse for (a step of a cumulative sum over a large
// vocabulary, scores next to the last that is chosen).  Nothing here uses 64-bit
// floating point, whose rate on this GPU is a hundredth of fp32's.
//
// 2^z: z = n + j/32 + y with |y| <= 2^-6, and 2^z = 2^n T[j] (1 + p(y)), with T[j]
// = 2^(j/32) in two numbers, a lane's registers (two shuffles are cheaper than
// the bank conflicts of a gather from shared memory), p the power series to y^4;
// the error is below 2^-28, 2^-31 in the mean.
#pragma once

#include <cstdint>

namespace fp8bs {

// 2^(j/32): the nearest fp32 number and the rest relative to it.
static __device__ const float2 kPow32[32] = {
    {0x1.000000p+0f, 0x0.0p+0f},          {0x1.059b0ep+0f, -0x1.947414p-25f},
    {0x1.0b5586p+0f, 0x1.8d96d4p-25f},    {0x1.11301ep+0f, -0x1.dda2fcp-25f},
    {0x1.172b84p+0f, -0x1.9c0c22p-27f},   {0x1.1d4874p+0f, -0x1.a2fbb2p-25f},
    {0x1.2387a6p+0f, 0x1.964904p-25f},    {0x1.29e9e0p+0f, -0x1.2b0dbcp-25f},
    {0x1.306fe0p+0f, 0x1.125002p-25f},    {0x1.371a74p+0f, -0x1.cde8cep-26f},
    {0x1.3dea64p+0f, 0x1.370be4p-25f},    {0x1.44e086p+0f, 0x1.336de2p-30f},
    {0x1.4bfdaep+0f, -0x1.0a3550p-25f},   {0x1.5342b6p+0f, -0x1.c541b4p-26f},
    {0x1.5ab07ep+0f, -0x1.00d8acp-27f},   {0x1.6247ecp+0f, -0x1.6cb284p-25f},
    {0x1.6a09e6p+0f, 0x1.26055cp-26f},    {0x1.71f75ep+0f, 0x1.8b2bb8p-26f},
    {0x1.7a1148p+0f, -0x1.05cb44p-25f},   {0x1.82589ap+0f, -0x1.1c2142p-26f},
    {0x1.8ace54p+0f, 0x1.67a1cap-28f},    {0x1.93737cp+0f, -0x1.348e56p-25f},
    {0x1.9c4918p+0f, 0x1.a3b5e4p-28f},    {0x1.a5503cp+0f, -0x1.0b7ec8p-25f},
    {0x1.ae89fap+0f, -0x1.f9c304p-27f},   {0x1.b7f770p+0f, -0x1.e4c886p-26f},
    {0x1.c199bep+0f, -0x1.6961b4p-28f},   {0x1.cb720ep+0f, -0x1.b5151ep-28f},
    {0x1.d5818ep+0f, -0x1.a5217cp-28f},   {0x1.dfc974p+0f, -0x1.ab7132p-26f},
    {0x1.ea4afap+0f, 0x1.61428ep-28f},    {0x1.f50766p+0f, -0x1.2ad5f8p-27f}};

constexpr float kShift = 393216.0f;       // 1.5 * 2^18: adding it rounds to multiples of 1/32
constexpr int kShiftBits = 0x48C00000;    // its bits

// n of pow_split.
__device__ __forceinline__ int pow_exponent(float zh) { return (__float_as_int(zh + kShift) - kShiftBits) >> 5; }

// 2^(zh + zl) = 2^n th (1 + rest); `entry` is the lane's of kPow32; a whole warp calls it.
__device__ __forceinline__ int pow_split(float zh, float zl, float2 entry, float &th, float &rest)
{
    const float u = zh + kShift;
    const int bits = __float_as_int(u);
    const float y = (zh - (u - kShift)) + zl;
    th = __shfl_sync(0xffffffffu, entry.x, bits & 31);
    const float tl = __shfl_sync(0xffffffffu, entry.y, bits & 31);
    constexpr float k1 = 0x1.62e430p-1f, k2 = 0x1.ebfbe0p-3f, k3 = 0x1.c6b08ep-5f, k4 = 0x1.3b2ab6p-7f; // ln(2)^k / k!
    rest = fmaf(fmaf(fmaf(fmaf(y, k4, k3), y, k2), y, k1), y, tl);
    return (bits - kShiftBits) >> 5;
}

struct Pair {
    float hi, lo; // hi = fl32(hi + lo)
};

// a + b for any a and b; an infinite or NaN sum has no low part.
__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = a + b, t = s - a;
    const float e = (a - (s - t)) + (b - t);
    return {s, fabsf(s) < __int_as_float(0x7f800000) ? e : 0.0f};
}

// a + b where |a| >= |b|, or a = 0.
__device__ __forceinline__ Pair fast_two_sum(float a, float b)
{
    const float s = a + b;
    return {s, fabsf(s) < __int_as_float(0x7f800000) ? b - (s - a) : 0.0f};
}

__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const Pair s = two_sum(a.hi, b.hi);
    return fast_two_sum(s.hi, s.lo + (a.lo + b.lo));
}

// a / b, b a normal number.
__device__ __forceinline__ Pair divide(Pair a, Pair b)
{
    const float q = __fdiv_rn(a.hi, b.hi);
    const float r = fmaf(-q, b.hi, a.hi) + fmaf(-q, b.lo, a.lo);
    return fast_two_sum(q, __fdiv_rn(r, b.hi));
}

} // namespace fp8bs
