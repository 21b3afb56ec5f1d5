// moe_route.cuh -- what the kernels that open an expert layer share: their
// parameters, the order of logits, the cast of the activations and the launch.
#pragma once

#include "fp8bs_testing.h"
#include "moe.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kRouteThreads = 256;
constexpr int kTG = kMoeTokenGroup;
static_assert(kRouteThreads / 32 == kTG, "one warp chooses for each token of a group");

struct RouteParams {
    int M, H, E, top_k, npad;
    const uint16_t *x;
    int ldx;
    const void *wr;
    int renorm;
    int32_t *ids;
    float *topw;
    float *logits;
    float *wtok;
    unsigned *group_done; // arrival counters; moe_plan_kernel: [0], and its bit mask after the counters
    unsigned *masks;      // [groups][kMoeMaxExperts / 32] chosen experts
    uint8_t *xq;
    float *xs;
    unsigned long long *runs;
};

// Order-preserving key of a logit: larger value, larger key; NaN is 0, below
// every number.
__device__ __forceinline__ uint32_t route_key(float v)
{
    const uint32_t b = __float_as_uint(v);
    if (v != v)
        return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp: one (token, 128 of H) group of the cast; scales [H/128][M].
__device__ __forceinline__ void cast_group(const RouteParams &p, long long group)
{
    const int lane = threadIdx.x & 31;
    const int kg = p.H / 128;
    if (group >= static_cast<long long>(p.M) * kg)
        return;
    const int m = static_cast<int>(group % p.M), g = static_cast<int>(group / p.M);
    const uint2 raw = *reinterpret_cast<const uint2 *>(p.x + static_cast<long long>(m) * p.ldx + g * 128 + lane * 4);
    uint32_t codes;
    const float s = quant_group_warp(raw, codes);
    *reinterpret_cast<uint32_t *>(p.xq + static_cast<long long>(m) * p.H + g * 128 + lane * 4) = codes;
    if (lane == 0)
        p.xs[g * p.M + m] = s;
}

RouteParams route_params(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev);

} // namespace fp8bs
