// norm.cu -- root-mean-square norm of a row with the residual's addition
// before it and the 8-bit cast with its scales behind it, as one kernel: what
// stands in front of a quantised linear layer.
//
//   h = bf16_rn(fl32(x + r))  (or x), stored as the new residual
//   u = fl32(h * g),  rs = 1 / sqrt(mean(h^2) + eps)
//   y = bf16_rn(fl32(u * rs))                              (where wanted)
//   E4M3 with fp32 scales: per 128 values s = fl32(amax|u| / 448) (1 for
//     zeros), code = e4m3_rn(fl32(u / s)), stored scale fl32(s * rs)
//   MX: per 32 values of v = fl32(u * rs) a power of two and codes, as mx.cu
//
// The norm's factor rs is the same for a whole row, so under fp32 scales a
// group's codes do not depend on it: they are converted and stored while the
// row's sum of squares is still being put together, and rs goes into the scales.
// The cast takes fp32 values, not y's bf16: one rounding fewer.
//
// One CTA per row, eight consecutive values a thread and step, so that a group
// of 128 is 16 lanes and a 16-byte access per lane is coalesced.  The row stays
// in registers as bf16 between the sum and what needs it: each input byte is
// read once and each output byte written once.
#include <cmath>

#include "fp8bs_testing.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxChunks = 4; // of eight values a thread
constexpr int kNormMaxK = kNormMaxThreads * kNormMaxChunks * 8;

struct NormParams {
    int M, K;
    const uint16_t *x;
    long long ldx;
    const uint16_t *res; // or nullptr
    long long ldr;
    uint16_t *res_out;
    long long ldo;
    const void *gamma;
    float eps;
    uint16_t *y; // or nullptr
    uint8_t *xq;
    float *xs;   // fp32 scales
    uint8_t *sf; // MX: scale atoms
    bool kmajor; // fp32 scales [K/128][M]
    unsigned long long *runs;
};

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void values8(const uint4 &w, float (&v)[8])
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
    }
}

// Eight weights of the norm from element k on.
template <bool kBf16> __device__ __forceinline__ void gamma8(const void *gamma, int k, float (&g)[8])
{
    if (kBf16) {
        values8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(gamma) + k), g);
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(gamma) + k);
        const float4 a = p[0], b = p[1];
        g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
        g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
    }
}

__device__ __forceinline__ float abs_max8(const float (&v)[8])
{
    return fmaxf(abs_max4(v[0], v[1], v[2], v[3]), abs_max4(v[4], v[5], v[6], v[7]));
}

// kChunks: steps of blockDim.x * 8 values that cover the row.
// No __restrict__: x and the residual may still be being written when a kernel
// launched programmatically starts, and res_out may be the residual itself.
template <bool kMx, bool kBf16, int kChunks>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_quant_kernel(const NormParams p)
{
    __shared__ float part[2][32];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + (kMx ? FP8BS_RUNS_NORM_MX : FP8BS_RUNS_NORM_FP8), 1ull);
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kg = p.K / 128;
    if (kMx && static_cast<int>(blockIdx.x) >= p.M) { // one atom's words of the rows past M
        grid_dependency_wait();
        const int g = blockIdx.x - p.M, tt = p.M / 128;
        uint32_t *const words = reinterpret_cast<uint32_t *>(p.sf + (static_cast<long long>(tt) * kg + g) * 512);
        for (int r = threadIdx.x; r < 128; r += blockDim.x)
            if (r >= p.M % 128)
                words[4 * (r & 31) + (r >> 5)] = 0u;
        return;
    }
    const int m = blockIdx.x;
    const int step = static_cast<int>(blockDim.x) * 8;
    const int k0 = static_cast<int>(threadIdx.x) * 8;
    grid_dependency_wait();
    uint4 raw[kChunks];
    {
        const uint16_t *const xr = p.x + m * p.ldx;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            raw[c] = make_uint4(0u, 0u, 0u, 0u);
            if (k < p.K)
                raw[c] = *reinterpret_cast<const uint4 *>(xr + k);
        }
    }
    if (p.res != nullptr) {
        uint4 add[kChunks];
        const uint16_t *const rr = p.res + m * p.ldr;
        uint16_t *const ro = p.res_out + m * p.ldo;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            add[c] = make_uint4(0u, 0u, 0u, 0u);
            if (k < p.K)
                add[c] = *reinterpret_cast<const uint4 *>(rr + k);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            float a[8], b[8];
            values8(raw[c], a);
            values8(add[c], b);
            raw[c] = make_uint4(bf16x2_rn(a[0] + b[0], a[1] + b[1]), bf16x2_rn(a[2] + b[2], a[3] + b[3]),
                                bf16x2_rn(a[4] + b[4], a[5] + b[5]), bf16x2_rn(a[6] + b[6], a[7] + b[7]));
            if (k < p.K)
                *reinterpret_cast<uint4 *>(ro + k) = raw[c];
        }
    }
    // Squares past fp32's range (values above 2^64 / sqrt(K)) are summed again
    // with the row times 2^-80; a row with an infinity or NaN keeps its sum.
    float pre = 1.0f, rs;
    float sg[kChunks]; // fp32 scales of this thread's groups, before rs
#pragma unroll 1
    for (int turn = 0;; ++turn) {
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            float h[8];
            values8(raw[c], h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] *= pre;
                ss = fmaf(h[i], h[i], ss);
            }
            if (!kMx) {
                float g[8] = {};
                if (k < p.K)
                    gamma8<kBf16>(p.gamma, k, g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[i] *= g[i];
                float am = abs_max8(h);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                float s = __fdiv_rn(am, kE4M3Max);
                sg[c] = s;
                s = s == 0.0f ? 1.0f : s; // zeros, or amax below 448 * 2^-150
                if (k < p.K)
                    *reinterpret_cast<uint2 *>(p.xq + static_cast<long long>(m) * p.K + k) =
                        make_uint2(quantize4(h[0], h[1], h[2], h[3], s), quantize4(h[4], h[5], h[6], h[7], s));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0)
            part[turn][warp] = ss;
        __syncthreads();
        ss = lane < static_cast<int>(blockDim.x >> 5) ? part[turn][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.K)) + p.eps * pre * pre);
        if (turn == 1 || ss != INFINITY)
            break;
        pre = 8.27180613e-25f; // 2^-80
    }
    if (!kMx) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            if (k < p.K && (lane & 15) == 0)
                p.xs[p.kmajor ? static_cast<long long>(k >> 7) * p.M + m : static_cast<long long>(m) * kg + (k >> 7)] =
                    sg[c] == 0.0f ? 1.0f : sg[c] * rs;
        }
        if (p.y == nullptr)
            return;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = c * step + k0;
        float v[8], g[8] = {};
        values8(raw[c], v);
        if (k < p.K)
            gamma8<kBf16>(p.gamma, k, g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] * pre * g[i] * rs;
        if (p.y != nullptr && k < p.K)
            *reinterpret_cast<uint4 *>(p.y + static_cast<long long>(m) * p.K + k) =
                make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
        if (kMx) {
            float am = abs_max8(v);
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int e = mx_shared_exponent(am);
            const float inv = mx_inv_scale(e);
            uint32_t byte = static_cast<uint32_t>(e + 127) << (8 * ((lane >> 2) & 3));
            byte |= __shfl_xor_sync(0xffffffffu, byte, 4);
            byte |= __shfl_xor_sync(0xffffffffu, byte, 8);
            if (k < p.K) {
                *reinterpret_cast<uint2 *>(p.xq + static_cast<long long>(m) * p.K + k) =
                    make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                               e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
                if ((lane & 15) == 0) {
                    const int r = m & 127;
                    reinterpret_cast<uint32_t *>(p.sf + (static_cast<long long>(m >> 7) * kg + (k >> 7)) * 512)
                        [4 * (r & 31) + (r >> 5)] = byte;
                }
            }
        }
    }
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <bool kMx, bool kBf16> auto norm_kernel(int chunks)
{
    return chunks == 1   ? rmsnorm_quant_kernel<kMx, kBf16, 1>
           : chunks == 2 ? rmsnorm_quant_kernel<kMx, kBf16, 2>
                         : rmsnorm_quant_kernel<kMx, kBf16, 4>;
}

fp8bs_status launch_norm(const NormParams &p, bool mx, bool gamma_bf16, bool pdl, cudaStream_t stream)
{
    const int words = p.K / 8;
    int chunks = 1;
    while (words > chunks * kNormMaxThreads)
        chunks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(static_cast<unsigned>(((words + chunks - 1) / chunks + 31) / 32 * 32), 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(p.M + (mx && p.M % 128 != 0 ? p.K / 128 : 0)), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    auto kernel = mx ? (gamma_bf16 ? norm_kernel<true, true>(chunks) : norm_kernel<true, false>(chunks))
                     : (gamma_bf16 ? norm_kernel<false, true>(chunks) : norm_kernel<false, false>(chunks));
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

fp8bs_status rmsnorm_quant(const void *x, int ldx, const void *residual, int ldr, void *residual_out, int ldo,
                           const void *gamma, fp8bs_dtype gamma_type, float eps, int M, int K, void *y, uint8_t *xq,
                           void *scales, bool mx, unsigned flags, void *stream)
{
    if (!x || !gamma || !xq || !scales || M < 1 || K < 1 || ldx < K || (residual == nullptr) != (residual_out == nullptr) ||
        (residual != nullptr && (ldr < K || ldo < K)) || (gamma_type != FP8BS_F32 && gamma_type != FP8BS_BF16) ||
        !(eps >= 7.88860905e-31f) || !std::isfinite(eps) || (flags & ~FP8BS_FLAG_OVERLAP_PREV) != 0)
        return FP8BS_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > kNormMaxK || (mx && M > kMaxTokens))
        return FP8BS_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(gamma, 16) || !aligned(y, 16) || !aligned(xq, 16) ||
        !aligned(scales, mx ? 16 : 4) ||
        (residual != nullptr && (!aligned(residual, 16) || ldr % 8 != 0 || !aligned(residual_out, 16) || ldo % 8 != 0)))
        return FP8BS_ERR_MISALIGNED;
    DeviceInfo dev;
    fp8bs_status st = current_device(&dev);
    if (st != FP8BS_OK)
        return st;
    NormParams p = {};
    p.M = M;
    p.K = K;
    p.x = static_cast<const uint16_t *>(x);
    p.ldx = ldx;
    p.res = static_cast<const uint16_t *>(residual);
    p.ldr = ldr;
    p.res_out = static_cast<uint16_t *>(residual_out);
    p.ldo = ldo;
    p.gamma = gamma;
    p.eps = eps;
    p.y = static_cast<uint16_t *>(y);
    p.xq = xq;
    p.xs = mx ? nullptr : static_cast<float *>(scales);
    p.sf = mx ? static_cast<uint8_t *>(scales) : nullptr;
    p.kmajor = M > 16;
    p.runs = dev.runs;
    return launch_norm(p, mx, gamma_type == FP8BS_BF16, (flags & FP8BS_FLAG_OVERLAP_PREV) != 0,
                       static_cast<cudaStream_t>(stream));
}

} // namespace

} // namespace fp8bs

using namespace fp8bs;

extern "C" {

fp8bs_status fp8_rmsnorm_quant_act(const void *x, int ldx, const void *residual, int ldr, void *residual_out, int ldro,
                                   const void *gamma, fp8bs_dtype gamma_type, float eps, int M, int K, void *y,
                                   uint8_t *xq, float *xs, unsigned flags, void *stream)
{
    return rmsnorm_quant(x, ldx, residual, ldr, residual_out, ldro, gamma, gamma_type, eps, M, K, y, xq, xs, false,
                         flags, stream);
}

fp8bs_status fp8_mx_rmsnorm_quant_act(const void *x, int ldx, const void *residual, int ldr, void *residual_out,
                                      int ldro, const void *gamma, fp8bs_dtype gamma_type, float eps, int M, int K,
                                      void *y, uint8_t *xq, uint8_t *xs_atoms, unsigned flags, void *stream)
{
    return rmsnorm_quant(x, ldx, residual, ldr, residual_out, ldro, gamma, gamma_type, eps, M, K, y, xq, xs_atoms, true,
                         flags, stream);
}

} // extern "C"
