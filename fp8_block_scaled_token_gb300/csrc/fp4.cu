// fp4.cu -- microscaled 4-bit (E2M1) quantisation and reading it back.
//
// E2M1 has the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two block formats:
//   NV (16 consecutive K share one E4M3 scale, every row one fp32 scale):
//     r    = fl32(amax_row / 2688)  (2688 = 6 * 448; 1 where that is below 2^-126)
//     b    = e4m3_rn(fl32(fl32(amax_16 / 6) / r))
//     d    = fl32(dec(b) * r)
//     code = e2m1_rn_satfinite(fl32(v / d)), 0 where b is 0
//   MX (32 consecutive K share one power of two, the OCP microscaling rule):
//     e    = floor(log2(amax_32)) - 2, clamped to [-127, 127] (0 for a zero block)
//     code = e2m1_rn_satfinite(v / 2^e)   (exact scaling)
// A code's value is fl32(code * d), or code * 2^e.
// A NaN or an infinity makes its row's r NaN or infinite (NV), or its block's
// scale byte 255, NaN (MX): every product with it is NaN, whatever the codes,
// which have no NaN of their own.
//
// Two codes to a byte, the lower K in the lower four bits; K is padded with
// zero codes and zero scales to whole 256-wide blocks.  Scale bytes in the
// 512-byte atoms of ptx.cuh, four blocks of K to an atom.
//
// Each input and output byte moves once, but for NV rows longer than registers
// hold (18,432 bf16 or 12,288 fp32 values), whose rest is read for the maximum
// and again for the codes.  5,120 x 17,408 bf16: quantising takes
// 48 us (227 MB, 0.7 of the measured copy bandwidth; MX 36 us), bound by the
// instructions of the conversion and of the check that keeps codes exact
// without a division a value; reading back to fp32 61 us (406 MB, at the
// memory's rate).  The activations'
// cast is a few microseconds of latency at decode sizes.
#include <cuda_bf16.h>

#include "fp8bs_testing.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kFp4Chunk = 16; // values a thread converts at a time: one NV block, half an MX block
// A row's chunks are held in registers between its maximum and the conversion,
// three (fp32: two) a thread, by as many whole warps as that takes: no warp
// waits for one that has a chunk more.  5,120 x 17,408, there and back: 110 us;
// 256 threads of four and a rest read twice 115, four a thread and fewer warps
// 107 but with spills.  Rows past 384 threads' read the rest twice (4,096 x
// 34,816: 182 us, 189 with up to 512 threads, of which an SM holds fewer).
constexpr int kMaxRowThreads = 384;
template <bool kBf16> constexpr int kRowHold = kBf16 ? 3 : 2;

// Eight fp32 values -> eight E2M1 codes, the first in the lowest four bits.
// The hardware conversion rounds to nearest even and saturates to +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float *v)
{
    uint32_t r;
    // cvt ...e2m1x2.f32 d, hi_src, lo_src: the first source lands in the upper four bits.
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// One value's code.
__device__ __forceinline__ uint32_t e2m1_code(float v)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "mov.b32 %0, {b, b, b, b};\n\t}"
        : "=r"(r)
        : "f"(v), "f"(0.0f));
    return r & 0xFu;
}

// Eight codes -> their values.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float *v)
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{\n\t.reg .f16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.f32.f16 %0, lo;\n\t"
            "cvt.f32.f16 %1, hi;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(h[i]));
    }
}

// Value of a UE4M3 scale byte (sign bit clear).
__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    float f;
    asm("{\n\t.reg .b32 h;\n\t.reg .f16 lo, hi;\n\t"
        "cvt.rn.f16x2.e4m3x2 h, %1;\n\t"
        "mov.b32 {lo, hi}, h;\n\t"
        "cvt.f32.f16 %0, lo;\n\t}"
        : "=f"(f)
        : "h"(static_cast<uint16_t>(byte)));
    return f;
}

__device__ __forceinline__ float nv_row_scale(float amax)
{
    const float r = __fdiv_rn(amax, 2688.0f);
    return r < 1.17549435e-38f ? 1.0f : r;
}

// Relative half-width of the interval in which an approximate quotient and
// the correctly rounded one both lie: v * rcp.approx(d) is within a few fp32
// ulps (2^-23 each) of v / d, and so are the products below.
constexpr float kQuotientSlack = 1.0f / 524288.0f; // 2^-19

// Where rcp.approx of x and the products with it stay normal numbers.
__device__ __forceinline__ bool plain_range(float x) { return x >= 1.17549435e-38f && x <= 8.5e37f; }

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// E4M3 code of fl32(fl32(amax / 6) / r); inv6 = 1 / (6 r) approximately, or
// NaN where nv_inv6 wants the divisions.
__device__ __forceinline__ uint32_t nv_scale_code(float amax, float r, float inv6)
{
    const float s = amax * inv6;
    const uint32_t both = e4m3x4(s * (1.0f - kQuotientSlack), s * (1.0f + kQuotientSlack), 0.0f, 0.0f);
    if ((both & 0xFFu) == (both >> 8) && s == s)
        return both & 0xFFu;
    return e4m3x4(__fdiv_rn(__fdiv_rn(amax, 6.0f), r), 0.0f, 0.0f, 0.0f) & 0xFFu;
}

// 1 / (6 r) approximately for rows where nv_scale_code may use it, else NaN.
// fl32(amax / 6) is off by more than kQuotientSlack where it is not a normal
// number.  With r >= 2^-112 such a block's quotient is below 2^-14, far under
// the least code's boundary of 2^-10, and its code 0 either way; the rows of
// smaller r (largest value below 5.2e-31) are divided.
__device__ __forceinline__ float nv_inv6(float r)
{
    return r >= 1.92592994e-34f && plain_range(r) ? rcp_approx(r) * (1.0f / 6.0f) : __int_as_float(0x7fffffff);
}

// Raw bits of sixteen consecutive source values.
template <bool kBf16> struct Raw16 {
    uint4 w[kBf16 ? 2 : 4];
};

template <bool kBf16> __device__ __forceinline__ Raw16<kBf16> load16(const void *row, int k0)
{
    Raw16<kBf16> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) +
                                                     static_cast<long long>(k0) * (kBf16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (kBf16 ? 2 : 4); ++i)
        r.w[i] = p[i];
    return r;
}

// Values 8 h ... 8 h + 7 of the sixteen.
template <bool kBf16> __device__ __forceinline__ void values8(const Raw16<kBf16> &r, int h, float (&v)[8])
{
    if (kBf16) {
        const uint32_t w[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = bf16_lo(w[q]);
            v[2 * q + 1] = bf16_hi(w[q]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = r.w[(kBf16 ? 0 : 2 * h) + i];
            v[4 * i] = __uint_as_float(w.x);
            v[4 * i + 1] = __uint_as_float(w.y);
            v[4 * i + 2] = __uint_as_float(w.z);
            v[4 * i + 3] = __uint_as_float(w.w);
        }
    }
}

// Word i of the raw bits, i a run-time number (registers have no address: a
// tree of selections).
template <int kWords> __device__ __forceinline__ uint32_t pick(const uint32_t (&w)[kWords], int i)
{
    uint32_t t[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        t[k] = w[k];
#pragma unroll
    for (int n = kWords / 2; n >= 1; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k)
            t[k] = (i & n) ? t[k + n] : t[k];
    return t[0];
}

// Value i of the sixteen.
template <bool kBf16> __device__ __forceinline__ float value_at(const Raw16<kBf16> &r, int i)
{
    uint32_t w[kBf16 ? 8 : 16];
#pragma unroll
    for (int q = 0; q < (kBf16 ? 2 : 4); ++q) {
        w[4 * q] = r.w[q].x;
        w[4 * q + 1] = r.w[q].y;
        w[4 * q + 2] = r.w[q].z;
        w[4 * q + 3] = r.w[q].w;
    }
    if (kBf16) {
        const uint32_t two = pick(w, i >> 1);
        return (i & 1) ? bf16_hi(two) : bf16_lo(two);
    }
    return __uint_as_float(pick(w, i));
}

// Codes of sixteen values over the scale d (0: zero codes): e2m1 of the
// correctly rounded quotient.  As in quantize4 (quant_math.cuh): both ends of
// an interval that holds it are converted, and since the conversion is
// monotonic equal codes are the quotient's.  The IEEE division is left for the
// values with a rounding boundary inside theirs, one at a time: with bf16
// values 0.2 % lie exactly on one (value and row maximum have eight bits and
// the block's scale four, so equality is common), which is in half of a warp's
// steps (all sixteen divided there: 5,120 x 17,408 to 4 bits and back 138 us,
// not 115).
template <bool kBf16> __device__ __forceinline__ uint2 nv_codes16(const Raw16<kBf16> &raw, float d)
{
    const float rd = rcp_approx(d);
    const float r_lo = rd * (1.0f - kQuotientSlack), r_hi = rd * (1.0f + kQuotientSlack);
    uint32_t codes[2], differ[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[8], q[8];
        values8<kBf16>(raw, h, v);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            mul2(q[i], q[i + 1], v[i], v[i + 1], r_lo);
        codes[h] = e2m1x8(q);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            mul2(q[i], q[i + 1], v[i], v[i + 1], r_hi);
        differ[h] = codes[h] ^ e2m1x8(q);
    }
    if (!plain_range(d)) {
        codes[0] = codes[1] = 0u;
        differ[0] = differ[1] = d == 0.0f ? 0u : 0xFFFFFFFFu;
    }
#pragma unroll 1
    while ((differ[0] | differ[1]) != 0u) {
        const bool second = differ[0] == 0u;
        const int shift = (__ffs(static_cast<int>(second ? differ[1] : differ[0])) - 1) & ~3;
        const float q = __fdiv_rn(value_at<kBf16>(raw, (second ? 8 : 0) + (shift >> 2)), d);
        const uint32_t keep = ~(0xFu << shift);
        const uint32_t code = e2m1_code(q) << shift;
        if (second) {
            codes[1] = (codes[1] & keep) | code;
            differ[1] &= keep;
        } else {
            codes[0] = (codes[0] & keep) | code;
            differ[0] &= keep;
        }
    }
    return make_uint2(codes[0], codes[1]);
}

// The larger magnitude of each half (with the signs' exclusive or), NaN where
// either is NaN.
__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The larger of two magnitudes, NaN if either is: the bits of non-negative
// numbers order like the values, and NaN above infinity.
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// Their largest magnitude, NaN if one is NaN.
template <bool kBf16> __device__ __forceinline__ float abs_max16(const Raw16<kBf16> &r)
{
    if (kBf16) {
        uint32_t m = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(r.w[0].x, r.w[0].y), abs_max_bf16x2(r.w[0].z, r.w[0].w)),
                                    abs_max_bf16x2(abs_max_bf16x2(r.w[1].x, r.w[1].y), abs_max_bf16x2(r.w[1].z, r.w[1].w)));
        return __uint_as_float(max((m << 16) & 0x7FFF0000u, m & 0x7FFF0000u));
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (kBf16 ? 2 : 4); ++i)
        m = max(max(m, max(r.w[i].x & 0x7FFFFFFFu, r.w[i].y & 0x7FFFFFFFu)),
                max(r.w[i].z & 0x7FFFFFFFu, r.w[i].w & 0x7FFFFFFFu));
    return __uint_as_float(m);
}

// Sixteen values -> two words of codes, and in `word` the scale bytes of the
// lane's atom, each at its place; whole warps call it (the word is put
// together from the lanes of one atom).  amax: their abs_max16; inv6: as
// nv_scale_code.
template <bool kBf16, bool kNv>
__device__ __forceinline__ uint2 quant16(const Raw16<kBf16> &raw, float amax, float r, float inv6, int c, bool live,
                                         uint32_t &word)
{
    uint2 codes;
    if (kNv) {
        const uint32_t byte = nv_scale_code(amax, r, inv6);
        codes = nv_codes16<kBf16>(raw, byte != 0u ? e4m3_value(byte) * r : 0.0f);
        word = byte << (8 * (c & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
    } else {
        amax = max_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const uint32_t b = __float_as_uint(amax);
        const int E = static_cast<int>(b >> 23);
        int e = E == 0 ? (b == 0u ? 0 : -127) : E - 127 - 2;
        e = e < -127 ? -127 : e;
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23); // 2^-e, e <= 125
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            values8<kBf16>(raw, h, v[h]);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i >> 3][i & 7] *= inv;
        codes = make_uint2(e2m1x8(v[0]), e2m1x8(v[1]));
        const uint32_t byte = E == 255 ? 255u : static_cast<uint32_t>(e + 127); // (NaN or infinite: 255 is NaN)
        word = live ? byte << (8 * ((c >> 1) & 3)) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    return codes;
}

// One CTA per row, sixteen values per thread and step; the first kHold steps'
// values stay in registers between the row's maximum (NV) and the conversion,
// a longer row's rest is read twice.
// kTiled: weights, codes of row r of the 128-row tile at [(tile * kg + kb) *
// 128 + r][128 bytes], rows past `rows` written as zeros; otherwise
// activations, codes [row][kg * 128].  Atoms [128-row tile][kg * atoms a
// unit][512] either way; the activations' rows past M are not written (they
// only ever meet token columns that are not stored).
// (No __restrict__: an activation cast starts while the kernel that writes x may
// still run, and x must not pass for constant over this kernel's whole life.)
// (56 registers: three CTAs of 384 threads an SM, 117 us with two)
template <bool kBf16, bool kNv, bool kTiled>
__global__ void __maxnreg__((kBf16 ? 56 : 64))
    fp4_quant_rows_kernel(const void *x, int rows, int K, long long ldx, int kg, uint8_t *xq, uint8_t *sf,
                          float *row_scale, int overlap, unsigned long long *runs)
{
    constexpr int kHold = kRowHold<kBf16>;
    const int threads = static_cast<int>(blockDim.x);
    __shared__ float warp_amax[kMaxRowThreads / 32];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(runs + (kTiled ? FP8BS_RUNS_FP4_QUANT_WEIGHT : FP8BS_RUNS_FP4_QUANT_ACT), 1ull);
    if (!kTiled) {
        // Launched early behind whatever kernel is before it (its launch
        // latency is then hidden); it touches nothing before the wait.  The
        // product that follows may be let in before the wait only if the
        // caller vouches for the weights, which it prefetches.
        if (overlap)
            grid_launch_dependents();
        grid_dependency_wait();
        if (!overlap)
            grid_launch_dependents();
    }
    const int row = blockIdx.x;
    const bool real = row < rows;
    const uint8_t *src = static_cast<const uint8_t *>(x) + static_cast<long long>(row) * ldx * (kBf16 ? 2 : 4);
    const int chunks = kg * 16; // of the padded row, a multiple of 16
    const int whole = real ? K / kFp4Chunk : 0; // chunks that hold values
    Raw16<kBf16> held[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int c = static_cast<int>(threadIdx.x) + i * threads;
#pragma unroll
        for (int q = 0; q < (kBf16 ? 2 : 4); ++q)
            held[i].w[q] = make_uint4(0u, 0u, 0u, 0u);
        if (c < whole)
            held[i] = load16<kBf16>(src, c * kFp4Chunk);
    }
    float r = 1.0f, inv6 = 0.0f;
    float held_amax[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        held_amax[i] = abs_max16<kBf16>(held[i]);
    if (kNv && real) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            amax = max_or_nan(amax, held_amax[i]);
#pragma unroll 1
        for (int c = static_cast<int>(threadIdx.x) + kHold * threads; c < whole; c += threads)
            amax = max_or_nan(amax, abs_max16<kBf16>(load16<kBf16>(src, c * kFp4Chunk)));
        amax = warp_max(amax);
        if ((threadIdx.x & 31) == 0)
            warp_amax[threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = warp_max(static_cast<int>(threadIdx.x & 31) < threads / 32 ? warp_amax[threadIdx.x & 31] : 0.0f);
        r = nv_row_scale(amax);
        inv6 = nv_inv6(r);
    }
    if (threadIdx.x == 0 && real && row_scale != nullptr)
        row_scale[row] = r;
    const int tile = row >> 7, rt = row & 127;
    constexpr int kPerAtom = kNv ? 4 : 8; // chunks
    uint8_t *const xq_row = xq + (kTiled ? (static_cast<long long>(tile) * kg * 128 + rt) * 128 : static_cast<long long>(row) * kg * 128);
    uint8_t *const sf_row = sf + static_cast<long long>(tile) * (chunks / kPerAtom) * 512 + 16 * (rt & 31) + 4 * (rt >> 5);
    // whole warps take part in the shuffles of quant16, also past the last chunk
    auto convert = [&](int c, const Raw16<kBf16> &raw, float amax) {
        uint32_t word;
        const uint2 codes = quant16<kBf16, kNv>(raw, amax, r, inv6, c, c < whole, word);
        if (c < chunks) {
            // (64-bit offsets: a row of 2^26 values and more has codes past 4 GB, one of 2^29 its scales)
            *reinterpret_cast<uint2 *>(xq_row + static_cast<unsigned long long>(static_cast<unsigned>(c) >> 4) * (kTiled ? 16384u : 128u) +
                                       (c & 15) * 8) = codes;
            if (c % kPerAtom == 0)
                *reinterpret_cast<uint32_t *>(sf_row + static_cast<unsigned long long>(static_cast<unsigned>(c) / kPerAtom) * 512u) = word;
        }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (i * threads + (static_cast<int>(threadIdx.x) & ~31) < chunks)
            convert(static_cast<int>(threadIdx.x) + i * threads, held[i], held_amax[i]);
#pragma unroll 1
    for (int c = static_cast<int>(threadIdx.x) + kHold * threads; (c & ~31) < chunks; c += threads) {
        Raw16<kBf16> raw = {};
        if (c < whole)
            raw = load16<kBf16>(src, c * kFp4Chunk);
        convert(c, raw, abs_max16<kBf16>(raw));
    }
}

// Packed weights -> values.  A warp takes four stores of one row, each lane
// 16 bytes a store (four fp32 or eight bf16 values), so that every store writes
// 512 consecutive bytes; the codes a lane needs for one are two or four bytes.
// (Sixteen values a thread, stored 64 bytes apart: 92 us for 5,120 x 17,408 to
// fp32 against the 406 MB moved.)
constexpr int kDequantSteps = 4;

template <bool kBf16, bool kNv>
__global__ void __launch_bounds__(256)
    fp4_dequant_kernel(const uint8_t *__restrict__ wq, const uint8_t *__restrict__ sf,
                       const float *__restrict__ row_scale, int N, int K, int kg, int segs, void *__restrict__ w,
                       unsigned long long *runs)
{
    constexpr int kPer = kBf16 ? 8 : 4; // values a lane and store
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(runs + FP8BS_RUNS_FP4_DEQUANT, 1ull);
    const int lane = threadIdx.x & 31;
    const long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); // (row, segment)
    if (i >= static_cast<long long>(N) * segs)
        return;
    const int n = static_cast<int>(i / segs);
    const int k0 = static_cast<int>(i % segs) * (kDequantSteps * 32 * kPer) + lane * kPer;
    const int tile = n >> 7, rt = n & 127;
    const uint8_t *const codes = wq + static_cast<long long>(tile) * kg * 16384 + rt * 128;
    const uint8_t *const scales = sf + static_cast<long long>(tile) * kg * (kNv ? 2048 : 1024) + 16 * (rt & 31) + 4 * (rt >> 5);
    const float row = row_scale != nullptr ? row_scale[n] : 1.0f;
    uint32_t cw[kDequantSteps];
    uint32_t byte[kDequantSteps];
#pragma unroll
    for (int t = 0; t < kDequantSteps; ++t) {
        const int k = k0 + t * 32 * kPer;
        cw[t] = byte[t] = 0u;
        if (k < K) {
            const uint8_t *c = codes + static_cast<long long>(k >> 8) * 16384 + ((k & 255) >> 1);
            cw[t] = kBf16 ? *reinterpret_cast<const uint32_t *>(c) : *reinterpret_cast<const uint16_t *>(c);
            const int blk = k >> (kNv ? 4 : 5);
            byte[t] = scales[static_cast<long long>(blk >> 2) * 512 + (blk & 3)];
        }
    }
#pragma unroll
    for (int t = 0; t < kDequantSteps; ++t) {
        const int k = k0 + t * 32 * kPer;
        if (k >= K)
            continue;
        const float s = kNv ? e4m3_value(byte[t])
                            : __uint_as_float(byte[t] == 0u ? 0x400000u : byte[t] == 255u ? 0x7FFFFFFFu : byte[t] << 23);
        const float d = s * row;
        float v[8];
        e2m1x8_values(cw[t], v);
        const long long o = static_cast<long long>(n) * K + k;
        if (kBf16) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j] * d, v[2 * j + 1] * d);
                h[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(w) + o), make_uint4(h[0], h[1], h[2], h[3]));
        } else {
            __stcs(reinterpret_cast<float4 *>(static_cast<float *>(w) + o),
                   make_float4(v[0] * d, v[1] * d, v[2] * d, v[3] * d));
        }
    }
}

// Threads that hold a row, in whole warps.
static int row_threads(int chunks, int hold)
{
    const int t = ((chunks + hold - 1) / hold + 31) & ~31;
    return t < kMaxRowThreads ? t : kMaxRowThreads;
}

fp8bs_status launch_fp4_quant_weights(const void *w, int wtype, int N, int K, int fmt, uint8_t *wq, uint8_t *sf,
                                      float *rows, cudaStream_t stream, const DeviceInfo &dev)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((N + 127) / 128) * 128u, 1, 1);
    cfg.stream = stream;
    const int kg = (K + 255) / 256;
    const bool bf = wtype == FP8BS_BF16, nv = fmt == FP8BS_FP4_NV;
    cfg.blockDim = dim3(static_cast<unsigned>(row_threads(kg * 16, bf ? kRowHold<true> : kRowHold<false>)), 1, 1);
    auto kernel = bf ? (nv ? fp4_quant_rows_kernel<true, true, true> : fp4_quant_rows_kernel<true, false, true>)
                     : (nv ? fp4_quant_rows_kernel<false, true, true> : fp4_quant_rows_kernel<false, false, true>);
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, w, N, K, static_cast<long long>(K), kg, wq, sf,
                                            rows, 0, dev.runs));
}

fp8bs_status launch_fp4_quant_act(const void *x, int M, int K, int ldx, int fmt, uint8_t *xq, uint8_t *sf,
                                  float *rows, bool pdl, cudaStream_t stream, const DeviceInfo &dev)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M), 1, 1);
    cfg.blockDim = dim3(kMaxRowThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = fmt == FP8BS_FP4_NV ? fp4_quant_rows_kernel<true, true, false>
                                      : fp4_quant_rows_kernel<true, false, false>;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, x, M, K, static_cast<long long>(ldx), (K + 255) / 256, xq, sf,
                                            rows, pdl ? 1 : 0, dev.runs));
}

fp8bs_status launch_fp4_dequant_weights(const uint8_t *wq, const uint8_t *sf, const float *rows, int N, int K,
                                        int fmt, void *w, int wtype, cudaStream_t stream, const DeviceInfo &dev)
{
    const int seg = kDequantSteps * 32 * (wtype == FP8BS_BF16 ? 8 : 4);
    const int segs = (K + seg - 1) / seg;
    const long long warps = static_cast<long long>(N) * segs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    const bool nv = fmt == FP8BS_FP4_NV;
    auto kernel = wtype == FP8BS_BF16 ? (nv ? fp4_dequant_kernel<true, true> : fp4_dequant_kernel<true, false>)
                                      : (nv ? fp4_dequant_kernel<false, true> : fp4_dequant_kernel<false, false>);
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, wq, sf, rows, N, K, (K + 255) / 256, segs, w, dev.runs));
}

} // namespace fp8bs
