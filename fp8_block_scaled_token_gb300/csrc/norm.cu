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
// Eight consecutive values a thread and step, so that a group of 128 is 16 lanes
// and a 16-byte access per lane is coalesced.  The row stays in registers between
// the sum and what needs it: each input byte is read once and each output byte
// written once.  16,384 rows of 5,120 with residual and y: 115 us, 6.6 TB/s (0.99 of
// the measured copy bandwidth); 512 rows 5.1 us; up to 150 rows 2.1 to 2.7 us, which
// is latency.  The first form took 255 us: packed fp32, a bf16 addition, a corrected
// quotient (codes8) in place of converting both ends of an interval, and far_row apart
// from the usual rows leave 30 instructions a value, 58 % of the issue slots.
#include "fp8bs_testing.h"
#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormManyThreads = 320; // where several CTAs share an SM
constexpr int kNormMidThreads = 640;
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

// Raw bits of eight weights of the norm, and their values.
template <bool kBf16> struct Gamma8 {
    uint4 w[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *gamma, int k)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(gamma) + k * (kBf16 ? 2 : 4));
        w[0] = p[0];
        if (!kBf16)
            w[kBf16 ? 0 : 1] = p[1];
    }
    __device__ __forceinline__ void values(float (&g)[8]) const
    {
        if (kBf16) {
            values8(w[0], g);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 a = w[kBf16 ? 0 : i];
                g[4 * i] = __uint_as_float(a.x);
                g[4 * i + 1] = __uint_as_float(a.y);
                g[4 * i + 2] = __uint_as_float(a.z);
                g[4 * i + 3] = __uint_as_float(a.w);
            }
        }
    }
};

// d0 = a0 * b0, d1 = a1 * b1 as one packed instruction.
__device__ __forceinline__ void mul2v(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 ra, rb;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\t"
        "mov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// bf16_rn(fl32(a + b)) of two values: rounded to bf16 at once, which is the
// same.  fl32 rounds only where one is below 2^-16 of the other, and such a sum
// is not near the middle between two bf16 numbers.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float abs_max8(const float (&v)[8])
{
    return fmaxf(abs_max4(v[0], v[1], v[2], v[3]), abs_max4(v[4], v[5], v[6], v[7]));
}

// Between these a quotient by s can be corrected as below without leaving the
// normal numbers: the remainder of a quotient of 2^-10 is 2^-34 s or more.
constexpr float kPlainLo = 8.077935669e-28f; // 2^-90
constexpr float kPlainHi = 1.237940039e+27f; // 2^90

// Codes of eight values over s: e4m3 of the correctly rounded quotients.  With y
// = fl32(1 / s), q = fl32(v y) and the exact remainder v - q s (one fma), fl32(q +
// (v - q s) y) is the correctly rounded quotient (Markstein 1990), three packed
// instructions a pair; quantize4 takes the scales at the ends of the range, NaN and infinity.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s)
{
    if (!(s >= kPlainLo && s <= kPlainHi))
        return make_uint2(quantize4(v[0], v[1], v[2], v[3], s), quantize4(v[4], v[5], v[6], v[7], s));
    const float y = -__frcp_rn(s); // negative, so that a zero keeps its sign: -0 -> +0, +0, +0 -> -(+0)
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float r0 = v[i], r1 = v[i + 1];
        mul2v(q[i], q[i + 1], v[i], v[i + 1], y, y);
        fma2(r0, r1, q[i], q[i + 1], s, s);
        fma2(q[i], q[i + 1], r0, r1, y, y);
    }
    return make_uint2(e4m3x4(-q[0], -q[1], -q[2], -q[3]), e4m3x4(-q[4], -q[5], -q[6], -q[7]));
}

// fl32(a / 448), in the same way.
__device__ __forceinline__ float over_448(float a)
{
    if (!(a >= kPlainLo && a <= kPlainHi))
        return __fdiv_rn(a, kE4M3Max);
    constexpr float y = 1.0f / 448.0f;
    const float q = a * y;
    return fmaf(fmaf(-q, kE4M3Max, a), y, q);
}

// Eight values of a row at k in the MX format; whole warps, K past the row's end stores nothing.
__device__ __forceinline__ void store_mx8(const NormParams &p, int m, int k, int K, float (&v)[8])
{
    const int lane = threadIdx.x & 31;
    float am = abs_max8(v);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const int e = mx_shared_exponent(am);
    const float inv = mx_inv_scale(e);
    uint32_t byte = static_cast<uint32_t>(e + 127) << (8 * ((lane >> 2) & 3));
    byte |= __shfl_xor_sync(0xffffffffu, byte, 4);
    byte |= __shfl_xor_sync(0xffffffffu, byte, 8);
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        mul2(v[i], v[i + 1], v[i], v[i + 1], inv);
    if (k < K) {
        *reinterpret_cast<uint2 *>(p.xq + static_cast<long long>(m) * p.K + k) =
            make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
        if ((lane & 15) == 0) {
            const int r = m & 127;
            reinterpret_cast<uint32_t *>(p.sf + (static_cast<long long>(m >> 7) * (p.K / 128) + (k >> 7)) * 512)
                [4 * (r & 31) + (r >> 5)] = byte;
        }
    }
}

// A row whose sum of squares leaves fp32's range (a value above 2^64 / sqrt(K)): the sum
// is taken of the row times 2^-80, in fp32, and everything else of the row as it is, so that
// small values beside large ones keep their bits.  A product with gamma past the range is
// taken times 2^-80 too, under fp32 scales with the rest of its group.  A row with an
// infinity keeps an infinite sum.  Every thread of the CTA calls it, with mine = false
// where its row is none of those; `h`: what this thread stored or read before.
template <bool kMx, bool kBf16>
__device__ __forceinline__ void far_row(const NormParams &p, const uint16_t *h, int m, bool mine, float *sum)
{
    constexpr float t = 0x1p-80f, t1 = 0x1p-56f, t2 = 0x1p-24f; // t = t1 t2: 1 / rms itself may be subnormal
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x >> 5);
    const int K = mine ? p.K : 0, step = static_cast<int>(blockDim.x) * 8, k0 = static_cast<int>(threadIdx.x) * 8;
    float ss = 0.0f;
#pragma unroll 1
    for (int k = k0; k < K; k += step) {
        float v[8];
        values8(*reinterpret_cast<const uint4 *>(h + k), v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(v[i] * t, v[i] * t, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0)
        sum[warp] = ss;
    __syncthreads();
    if (!mine)
        return;
    ss = lane < warps ? sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(K)) + p.eps * t * t); // of the row times t
    const float r1 = rs * t1;                                                           // r1 * t2: of the row
#pragma unroll 1
    for (int base = 0; base < K; base += step) {
        const int k = base + k0;
        Gamma8<kBf16> gamma = {};
        float v[8] = {}, g[8], u[8], far[8], y[8];
        if (k < K) {
            gamma.load(p.gamma, k);
            values8(*reinterpret_cast<const uint4 *>(h + k), v);
        }
        gamma.values(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = v[i] * g[i];
            far[i] = v[i] * t * g[i];
            y[i] = fabsf(u[i]) < INFINITY ? u[i] * r1 * t2 : far[i] * rs;
        }
        if (p.y != nullptr && k < K)
            *reinterpret_cast<uint4 *>(p.y + static_cast<long long>(m) * p.K + k) =
                make_uint4(bf16x2_rn(y[0], y[1]), bf16x2_rn(y[2], y[3]), bf16x2_rn(y[4], y[5]), bf16x2_rn(y[6], y[7]));
        if (kMx) {
            store_mx8(p, m, k, K, y);
        } else {
            float am = abs_max8(u), am_far = abs_max8(far);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                am_far = fmaxf(am_far, __shfl_xor_sync(0xffffffffu, am_far, o));
            }
            const bool over = am == INFINITY;
            const float s = over_448(over ? am_far : am);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                u[i] = over ? far[i] : u[i];
            const uint2 codes = codes8(u, s == 0.0f ? 1.0f : s);
            if (k < K) {
                *reinterpret_cast<uint2 *>(p.xq + static_cast<long long>(m) * p.K + k) = codes;
                if ((lane & 15) == 0)
                    p.xs[p.kmajor ? static_cast<long long>(k >> 7) * p.M + m : static_cast<long long>(m) * (p.K / 128) + (k >> 7)] =
                        s == 0.0f ? 1.0f : over ? s * rs : s * r1 * t2;
            }
        }
    }
}

// A CTA: blockDim.y rows of blockDim.x threads; kMost threads at most, kMin CTAs to an SM.
template <bool kMx, bool kBf16, int kChunks, int kMost, int kMin>
__global__ void __launch_bounds__(kMost, kMin) rmsnorm_quant_kernel(const NormParams p)
{
    __shared__ float part[2][32];
    if (blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0)
        atomicAdd(p.runs + (kMx ? FP8BS_RUNS_NORM_MX : FP8BS_RUNS_NORM_FP8), 1ull);
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = static_cast<int>(blockDim.x >> 5); // of a row
    const int kg = p.K / 128;
    const int rows = static_cast<int>(blockDim.y);
    const int ctas = (p.M + rows - 1) / rows;
    if (kMx && static_cast<int>(blockIdx.x) >= ctas) { // one atom's words of the rows past M
        grid_dependency_wait();
        const int g = blockIdx.x - ctas, tt = p.M / 128;
        uint32_t *const words = reinterpret_cast<uint32_t *>(p.sf + (static_cast<long long>(tt) * kg + g) * 512);
        for (int r = threadIdx.y * blockDim.x + threadIdx.x; r < 128; r += blockDim.x * blockDim.y)
            if (r >= p.M % 128)
                words[4 * (r & 31) + (r >> 5)] = 0u;
        return;
    }
    const int m = static_cast<int>(blockIdx.x) * rows + threadIdx.y;
    const int K = m < p.M ? p.K : 0; // a row past the last: no loads, no stores
    const int step = static_cast<int>(blockDim.x) * 8;
    const int k0 = static_cast<int>(threadIdx.x) * 8;
    float *const sum = part[0] + threadIdx.y * warps;
    Gamma8<kBf16> gamma[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        gamma[c] = {};
        if (c * step + k0 < K)
            gamma[c].load(p.gamma, c * step + k0);
    }
    grid_dependency_wait();
    uint4 h[kChunks];
    {
        const uint16_t *const xr = p.x + m * p.ldx;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            h[c] = make_uint4(0u, 0u, 0u, 0u);
            if (k < K)
                h[c] = *reinterpret_cast<const uint4 *>(xr + k);
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
            if (k < K)
                add[c] = *reinterpret_cast<const uint4 *>(rr + k);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            h[c] = make_uint4(add_bf16x2(h[c].x, add[c].x), add_bf16x2(h[c].y, add[c].y),
                              add_bf16x2(h[c].z, add[c].z), add_bf16x2(h[c].w, add[c].w));
            if (k < K)
                *reinterpret_cast<uint4 *>(ro + k) = h[c];
        }
    }
    float u[kChunks][8];
    float sg[kChunks]; // fp32 scales of this thread's groups, before rs
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = c * step + k0;
        float g[8];
        values8(h[c], u[c]);
        gamma[c].values(g);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            fma2(s0, s1, u[c][i], u[c][i + 1], u[c][i], u[c][i + 1]);
            mul2v(u[c][i], u[c][i + 1], u[c][i], u[c][i + 1], g[i], g[i + 1]);
        }
        if (!kMx) {
            float am = abs_max8(u[c]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const float s = over_448(am);
            sg[c] = s;
            const uint2 codes = codes8(u[c], s == 0.0f ? 1.0f : s); // 0: zeros, or amax below 448 * 2^-150
            if (k < K)
                *reinterpret_cast<uint2 *>(p.xq + static_cast<long long>(m) * p.K + k) = codes;
        }
    }
    float ss = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0)
        sum[warp] = ss;
    __syncthreads();
    ss = lane < warps ? sum[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.K)) + p.eps);
    if (!kMx) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            if (k < K && (lane & 15) == 0)
                p.xs[p.kmajor ? static_cast<long long>(k >> 7) * p.M + m : static_cast<long long>(m) * kg + (k >> 7)] =
                    sg[c] == 0.0f ? 1.0f : sg[c] * rs;
        }
    }
    if (kMx || p.y != nullptr) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = c * step + k0;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                mul2(v[i], v[i + 1], u[c][i], u[c][i + 1], rs);
            if (p.y != nullptr && k < K)
                *reinterpret_cast<uint4 *>(p.y + static_cast<long long>(m) * p.K + k) =
                    make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
            if (kMx)
                store_mx8(p, m, k, K, v);
        }
    }
    // Last, so that the usual row keeps nothing for it: each thread writes its own places once more.
    const bool far = ss == INFINITY;
    if (rows == 1 ? far : __syncthreads_or(far))
        far_row<kMx, kBf16>(p, p.res != nullptr ? p.res_out + m * p.ldo : p.x + m * p.ldx, m, far, sum + 32);
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Registers for the values in flight against CTAs to an SM: four CTAs of 320 threads hold two steps (three: 120
// us for 16,384 rows of 5,120, not 115; five spill 240 bytes a thread, 162), two hold four (three: 53 us for 4,096
// of 8,192, not 47.7).  Spills where the registers are few: 20 bytes of stores in two steps at 48 registers under
// fp32 scales, 68 to 88 in four steps of 1,024 threads.
template <bool kMx, bool kBf16> auto norm_kernel(int chunks, int threads)
{
    if (threads <= kNormManyThreads)
        return chunks == 1   ? rmsnorm_quant_kernel<kMx, kBf16, 1, kNormManyThreads, 4>
               : chunks == 2 ? rmsnorm_quant_kernel<kMx, kBf16, 2, kNormManyThreads, 4>
                             : rmsnorm_quant_kernel<kMx, kBf16, 4, kNormManyThreads, 2>;
    if (chunks == 4 && threads <= kNormMidThreads)
        return rmsnorm_quant_kernel<kMx, kBf16, 4, kNormMidThreads, 1>;
    return chunks == 1   ? rmsnorm_quant_kernel<kMx, kBf16, 1, kNormMaxThreads, 1>
           : chunks == 2 ? rmsnorm_quant_kernel<kMx, kBf16, 2, kNormMaxThreads, 1>
                         : rmsnorm_quant_kernel<kMx, kBf16, 4, kNormMaxThreads, 1>;
}

fp8bs_status launch_norm(const NormParams &p, bool mx, bool gamma_bf16, bool pdl, cudaStream_t stream, int sms)
{
    const int words = p.K / 8;
    // Up to a row an SM: the whole row's loads in flight at once, in one large CTA (152 rows of 5,120 2.5 us,
    // 2.9 in small ones).  More: small CTAs, four to an SM (200 rows 3.5 us against 3.8, 16,384 rows 115 against
    // 224), with several rows each where a row needs few threads (16,384 rows of 256: 9.5 us, 17.4 with one).
    const int most = p.M <= sms ? kNormMaxThreads : kNormManyThreads;
    int chunks = 1;
    while (words > chunks * most && chunks < kNormMaxChunks)
        chunks *= 2;
    const int threads = ((words + chunks - 1) / chunks + 31) / 32 * 32;
    const int rows = most == kNormMaxThreads ? 1 : most / threads > 1 ? most / threads : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(static_cast<unsigned>(threads), static_cast<unsigned>(rows), 1);
    cfg.gridDim = dim3(static_cast<unsigned>((p.M + rows - 1) / rows + (mx && p.M % 128 != 0 ? p.K / 128 : 0)), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    auto kernel = mx ? (gamma_bf16 ? norm_kernel<true, true>(chunks, threads) : norm_kernel<true, false>(chunks, threads))
                     : (gamma_bf16 ? norm_kernel<false, true>(chunks, threads) : norm_kernel<false, false>(chunks, threads));
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

fp8bs_status rmsnorm_quant(const void *x, int ldx, const void *residual, int ldr, void *residual_out, int ldo,
                           const void *gamma, fp8bs_dtype gamma_type, float eps, int M, int K, void *y, uint8_t *xq,
                           void *scales, bool mx, unsigned flags, void *stream)
{
    if (!x || !gamma || !xq || !scales || M < 1 || K < 1 || ldx < K || (residual == nullptr) != (residual_out == nullptr) ||
        (residual != nullptr && (ldr < K || ldo < K)) || (gamma_type != FP8BS_F32 && gamma_type != FP8BS_BF16) ||
        !(eps >= 7.88860905e-31f && eps <= 1.26765060e+30f) || (flags & ~FP8BS_FLAG_OVERLAP_PREV) != 0)
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
                       static_cast<cudaStream_t>(stream), dev.sms);
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
