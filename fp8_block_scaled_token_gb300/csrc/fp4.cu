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
//
// Two codes to a byte, the lower K in the lower four bits; K is padded with
// zero codes and zero scales to whole 256-wide blocks.  Scale bytes in the
// 512-byte atoms of ptx.cuh, four blocks of K to an atom.
//
// All three kernels move each input and output byte once (the row kernels
// read a row a second time, from L1/L2) and are bound by memory, or at a few
// tokens by latency.
#include <cuda_bf16.h>

#include "fp8bs_testing.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kFp4Chunk = 16; // values a thread converts at a time: one NV block, half an MX block

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

// Codes of eight values over the scale d > 0: e2m1 of the correctly rounded
// quotient.  As in quantize4 (quant_math.cuh): q = v * rcp(d) is within 2^-19
// |q| of the rounded quotient, the conversion is monotonic, so where both ends
// of that interval have the same code it is the quotient's; only where a
// rounding boundary falls inside is the IEEE division done.
__device__ __forceinline__ uint32_t nv_codes8(const float *v, float d)
{
    float q[8];
    if (d >= 1.17549435e-38f && d <= 8.5e37f) { // where the approximate reciprocal is a normal number
        float r, lo[8], hi[8];
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = v[i] * r;
            const float e = fabsf(q[i]) * (1.0f / 524288.0f);
            lo[i] = q[i] - e;
            hi[i] = q[i] + e;
        }
        const uint32_t cl = e2m1x8(lo), ch = e2m1x8(hi);
        if (cl == ch)
            return cl;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __fdiv_rn(v[i], d);
    return e2m1x8(q);
}

// Sixteen values of row element k0.. (bf16 or fp32 source, 16-byte aligned).
template <bool kBf16> __device__ __forceinline__ void load16(const void *row, int k0, float (&v)[16])
{
    if (kBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + k0);
        const uint4 a = p[0], b = p[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + k0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = p[i];
            v[4 * i] = f.x;
            v[4 * i + 1] = f.y;
            v[4 * i + 2] = f.z;
            v[4 * i + 3] = f.w;
        }
    }
}

__device__ __forceinline__ float abs_max16(const float (&v)[16])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// One CTA per row: the row's largest magnitude (NV), then sixteen values per
// thread and step.  kTiled: weights, codes of row r of the 128-row tile at
// [(tile * kg + kb) * 128 + r][128 bytes], rows past `rows` written as zeros;
// otherwise activations, codes [row][kg * 128].  Atoms [128-row tile][kg *
// atoms a unit][512] either way; the activations' rows past M are not written
// (they only ever meet token columns that are not stored).
template <bool kBf16, bool kNv, bool kTiled, int kThreads>
__global__ void __launch_bounds__(kThreads)
    fp4_quant_rows_kernel(const void *__restrict__ x, int rows, int K, long long ldx, int kg, uint8_t *__restrict__ xq,
                          uint8_t *__restrict__ sf, float *__restrict__ row_scale, unsigned long long *runs)
{
    __shared__ float warp_amax[kThreads / 32];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(runs + (kTiled ? FP8BS_RUNS_FP4_QUANT_WEIGHT : FP8BS_RUNS_FP4_QUANT_ACT), 1ull);
    if (!kTiled) {
        grid_launch_dependents();
        grid_dependency_wait();
    }
    const int row = blockIdx.x;
    const bool real = row < rows;
    const uint8_t *src = static_cast<const uint8_t *>(x) + static_cast<long long>(row) * ldx * (kBf16 ? 2 : 4);
    const int chunks = kg * 16; // of the padded row, a multiple of 16
    float r = 1.0f;
    if (kNv && real) {
        float amax = 0.0f;
        for (int c = threadIdx.x; c * kFp4Chunk < K; c += kThreads) {
            float v[16];
            load16<kBf16>(src, c * kFp4Chunk, v);
            amax = fmaxf(amax, abs_max16(v));
        }
        amax = warp_max(amax);
        if ((threadIdx.x & 31) == 0)
            warp_amax[threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = warp_amax[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i)
            amax = fmaxf(amax, warp_amax[i]);
        r = nv_row_scale(amax);
    }
    if (threadIdx.x == 0 && real && row_scale != nullptr)
        row_scale[row] = r;
    const int tile = row >> 7, rt = row & 127;
    // whole warps take part in the shuffles below, also past the last chunk
    for (int c0 = 0; c0 < chunks; c0 += kThreads) {
        const int c = c0 + static_cast<int>(threadIdx.x);
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = 0.0f;
        if (real && c * kFp4Chunk < K)
            load16<kBf16>(src, c * kFp4Chunk, v);
        float amax = abs_max16(v);
        uint32_t byte;
        uint2 codes = make_uint2(0u, 0u);
        if (kNv) {
            const float s = __fdiv_rn(__fdiv_rn(amax, 6.0f), r);
            byte = e4m3x4(s, 0.0f, 0.0f, 0.0f) & 0xFFu;
            if (byte != 0u) {
                const float d = e4m3_value(byte) * r;
                codes.x = nv_codes8(v, d);
                codes.y = nv_codes8(v + 8, d);
            }
            byte <<= 8 * (c & 3);
            byte |= __shfl_xor_sync(0xffffffffu, byte, 1);
            byte |= __shfl_xor_sync(0xffffffffu, byte, 2);
        } else {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const uint32_t b = __float_as_uint(amax);
            const int E = static_cast<int>(b >> 23);
            int e = E == 0 ? (b == 0u ? 0 : -127) : E - 127 - 2;
            e = e < -127 ? -127 : e;
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23); // 2^-e, e <= 125
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] *= inv;
            codes.x = e2m1x8(v);
            codes.y = e2m1x8(v + 8);
            byte = real && c * kFp4Chunk < K ? static_cast<uint32_t>(e + 127) << (8 * ((c >> 1) & 3)) : 0u;
            byte |= __shfl_xor_sync(0xffffffffu, byte, 2);
            byte |= __shfl_xor_sync(0xffffffffu, byte, 4);
        }
        if (c < chunks) {
            const int kb = c >> 4;
            const long long at = kTiled ? ((static_cast<long long>(tile) * kg + kb) * 128 + rt) * 128 + (c & 15) * 8
                                        : (static_cast<long long>(row) * kg + kb) * 128 + (c & 15) * 8;
            *reinterpret_cast<uint2 *>(xq + at) = codes;
            const int per_atom = kNv ? 4 : 8; // chunks
            if (c % per_atom == 0) {
                const long long atom = static_cast<long long>(tile) * (chunks / per_atom) + c / per_atom;
                *reinterpret_cast<uint32_t *>(sf + atom * 512 + 16 * (rt & 31) + 4 * (rt >> 5)) = byte;
            }
        }
    }
}

// Packed weights -> values, sixteen per thread.
template <bool kBf16, bool kNv>
__global__ void __launch_bounds__(256)
    fp4_dequant_kernel(const uint8_t *__restrict__ wq, const uint8_t *__restrict__ sf,
                       const float *__restrict__ row_scale, int N, int K, int kg, void *__restrict__ w,
                       unsigned long long *runs)
{
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(runs + FP8BS_RUNS_FP4_DEQUANT, 1ull);
    const int per_row = K / kFp4Chunk;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(N) * per_row)
        return;
    const int n = static_cast<int>(i / per_row), c = static_cast<int>(i % per_row);
    const int tile = n >> 7, rt = n & 127;
    const uint2 codes = *reinterpret_cast<const uint2 *>(
        wq + ((static_cast<long long>(tile) * kg + (c >> 4)) * 128 + rt) * 128 + (c & 15) * 8);
    const int blk = kNv ? c : c >> 1;
    const long long atom = static_cast<long long>(tile) * (kg * (kNv ? 4 : 2)) + (blk >> 2);
    const uint32_t byte = sf[atom * 512 + 16 * (rt & 31) + 4 * (rt >> 5) + (blk & 3)];
    const float s = kNv ? e4m3_value(byte) : __uint_as_float(byte == 0u ? 0x400000u : byte << 23);
    const float d = row_scale != nullptr ? s * row_scale[n] : s;
    float v[16];
    e2m1x8_values(codes.x, v);
    e2m1x8_values(codes.y, v + 8);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        v[j] *= d;
    const long long o = static_cast<long long>(n) * K + c * kFp4Chunk;
    if (kBf16) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            h[j] = *reinterpret_cast<const uint32_t *>(&b);
        }
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(w) + o);
        out[0] = make_uint4(h[0], h[1], h[2], h[3]);
        out[1] = make_uint4(h[4], h[5], h[6], h[7]);
    } else {
        float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(w) + o);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            out[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
}

fp8bs_status launch_fp4_quant_weights(const void *w, int wtype, int N, int K, int fmt, uint8_t *wq, uint8_t *sf,
                                      float *rows, cudaStream_t stream, const DeviceInfo &dev)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((N + 127) / 128) * 128u, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    const bool nv = fmt == FP8BS_FP4_NV;
    auto kernel = wtype == FP8BS_BF16
                      ? (nv ? fp4_quant_rows_kernel<true, true, true, 256> : fp4_quant_rows_kernel<true, false, true, 256>)
                      : (nv ? fp4_quant_rows_kernel<false, true, true, 256> : fp4_quant_rows_kernel<false, false, true, 256>);
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, w, N, K, static_cast<long long>(K), (K + 255) / 256, wq, sf,
                                            rows, dev.runs));
}

fp8bs_status launch_fp4_quant_act(const void *x, int M, int K, int ldx, int fmt, uint8_t *xq, uint8_t *sf,
                                  float *rows, bool pdl, cudaStream_t stream, const DeviceInfo &dev)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(M), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    auto kernel = fmt == FP8BS_FP4_NV ? fp4_quant_rows_kernel<true, true, false, 256>
                                      : fp4_quant_rows_kernel<true, false, false, 256>;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, x, M, K, static_cast<long long>(ldx), (K + 255) / 256, xq, sf,
                                            rows, dev.runs));
}

fp8bs_status launch_fp4_dequant_weights(const uint8_t *wq, const uint8_t *sf, const float *rows, int N, int K,
                                        int fmt, void *w, int wtype, cudaStream_t stream, const DeviceInfo &dev)
{
    const long long chunks = static_cast<long long>(N) * (K / kFp4Chunk);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((chunks + 255) / 256), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    const bool nv = fmt == FP8BS_FP4_NV;
    auto kernel = wtype == FP8BS_BF16 ? (nv ? fp4_dequant_kernel<true, true> : fp4_dequant_kernel<true, false>)
                                      : (nv ? fp4_dequant_kernel<false, true> : fp4_dequant_kernel<false, false>);
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, wq, sf, rows, N, K, (K + 255) / 256, w, dev.runs));
}

} // namespace fp8bs
