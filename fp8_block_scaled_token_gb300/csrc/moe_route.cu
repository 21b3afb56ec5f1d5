// moe_route.cu -- the first kernel of an expert layer: router logits, the
// choice of the experts and their weights, the list of experts that any token
// chose, and the E4M3 cast of the activations (which does not depend on the
// choice and runs beside it).
//
//   l[m, e] = sum_h x[m, h] * wr[e, h]                    (fp32)
//   ids[m]  = the top_k experts of largest l, descending, ties to the lowest
//             expert; NaN logits order below every number
//   w[m, j] = exp(l_j - l_max) / sum exp(l - l_max), the sum over the chosen
//             experts (renormalised) or over all of them
//
// Grid: one CTA per (expert, group of 8 tokens), then one CTA per four (token,
// 128 of H) groups of the cast.  The last CTA of a token group chooses for its
// eight tokens, and the last group's CTA lists the active experts; arrivals
// are counted, nobody waits.
#include <cuda_bf16.h>

#include "fp8bs_testing.h"
#include "moe.h"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

constexpr int kRouteThreads = 128;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kTG = kMoeTokenGroup;

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
    unsigned *group_done; // [8], then the groups' counter, then the bit mask
    int *active;
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

// The active experts of the bit mask, ascending, and the mask back to zero
// (one warp, after every bit is set).
__device__ __forceinline__ void list_active(unsigned *mask, int E, int *active)
{
    const int lane = threadIdx.x & 31;
    const int words = (E + 31) / 32;
    const unsigned m = lane < words ? atomicExch(mask + lane, 0u) : 0u;
    int before = 0, total = 0;
    for (int i = 0; i < words; ++i) {
        const int c = __popc(__shfl_sync(0xffffffffu, m, i));
        before += i < lane ? c : 0;
        total += c;
    }
    for (unsigned rest = m; rest != 0u; rest &= rest - 1u)
        active[1 + before++] = lane * 32 + __ffs(rest) - 1;
    if (lane == 0)
        active[0] = total;
}

// One warp: the choice for one token.
__device__ __forceinline__ void choose(const RouteParams &p, int m)
{
    constexpr int kPer = kMoeMaxExperts / 32;
    const int lane = threadIdx.x & 31;
    float l[kPer];
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < p.E ? __ldcg(p.logits + static_cast<long long>(m) * p.E + e) : 0.0f;
        key[i] = e < p.E ? route_key(l[i]) : 0u;
    }
    float lmax = 0.0f, sum = 0.0f, mine_l = 0.0f;
    int mine_e = -1;
    unsigned taken = 0; // bit i: this lane's expert i * 32 + lane is chosen
    for (int j = 0; j < p.top_k; ++j) {
        // this lane's best remaining expert, then the warp's
        uint32_t k = 0;
        int e = 0x7fffffff;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int ei = i * 32 + lane;
            if (ei < p.E && !(taken >> i & 1u) && (e == 0x7fffffff || key[i] > k)) {
                k = key[i];
                e = ei;
                v = l[i];
            }
        }
        const uint32_t kmax = __reduce_max_sync(0xffffffffu, k);
        const uint32_t emin = __reduce_min_sync(0xffffffffu, k == kmax ? static_cast<uint32_t>(e) : 0xffffffffu);
        const int owner = static_cast<int>(emin & 31u);
        v = __shfl_sync(0xffffffffu, v, owner);
        if (lane == owner)
            taken |= 1u << (emin >> 5);
        if (j == 0)
            lmax = v;
        if (lane == j) {
            mine_e = static_cast<int>(emin);
            mine_l = v;
        }
    }
    // p = exp(l - lmax); where the largest is infinite the difference is NaN,
    // as the formula gives
    float pj = lane < p.top_k ? expf(mine_l - lmax) : 0.0f;
    if (p.renorm) {
        sum = pj;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i * 32 + lane < p.E)
                sum += expf(l[i] - lmax);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    pj = __fdiv_rn(pj, sum);
    if (lane < p.top_k) {
        p.ids[static_cast<long long>(m) * p.top_k + lane] = mine_e;
        p.topw[static_cast<long long>(m) * p.top_k + lane] = pj;
        if (p.wtok != nullptr) {
            p.wtok[static_cast<long long>(mine_e) * p.npad + m] = pj;
            atomicOr(p.group_done + kMoeMaxTokens / kTG + 1 + (mine_e >> 5), 1u << (mine_e & 31));
        }
    }
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

template <bool kBf16>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p)
{
    __shared__ float part[kRouteWarps][kTG];
    __shared__ unsigned arrived;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_MOE_ROUTE, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (p.M + kTG - 1) / kTG;
    const int routing = p.E * groups;
    if (static_cast<int>(blockIdx.x) >= routing) {
        cast_group(p, static_cast<long long>(blockIdx.x - routing) * kRouteWarps + warp);
        return;
    }
    const int e = blockIdx.x % p.E, tg = blockIdx.x / p.E;
    const int t0 = tg * kTG;
    const int nt = p.M - t0 < kTG ? p.M - t0 : kTG;
    // the 128-value blocks of H, dealt to the warps in turn, four values a lane
    float acc[kTG];
#pragma unroll
    for (int t = 0; t < kTG; ++t)
        acc[t] = 0.0f;
    for (int h = warp * 128 + lane * 4; h < p.H; h += kRouteThreads * 4) {
        float w[4];
        if (kBf16) {
            const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.wr) +
                                                             static_cast<long long>(e) * p.H + h);
            w[0] = bf16_lo(r.x);
            w[1] = bf16_hi(r.x);
            w[2] = bf16_lo(r.y);
            w[3] = bf16_hi(r.y);
        } else {
            const float4 r = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.wr) +
                                                               static_cast<long long>(e) * p.H + h);
            w[0] = r.x;
            w[1] = r.y;
            w[2] = r.z;
            w[3] = r.w;
        }
#pragma unroll
        for (int t = 0; t < kTG; ++t) {
            if (t < nt) {
                const uint2 r = *reinterpret_cast<const uint2 *>(p.x + static_cast<long long>(t0 + t) * p.ldx + h);
                acc[t] = fmaf(bf16_lo(r.x), w[0], acc[t]);
                acc[t] = fmaf(bf16_hi(r.x), w[1], acc[t]);
                acc[t] = fmaf(bf16_lo(r.y), w[2], acc[t]);
                acc[t] = fmaf(bf16_hi(r.y), w[3], acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kTG; ++t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        if (lane == 0)
            part[warp][t] = acc[t];
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < nt) {
        float s = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kRouteWarps; ++i)
            s += part[i][threadIdx.x];
        __stcg(p.logits + static_cast<long long>(t0 + threadIdx.x) * p.E + e, s);
        if (p.wtok != nullptr)
            __stcg(p.wtok + static_cast<long long>(e) * p.npad + t0 + threadIdx.x, 0.0f);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        arrived = atomic_add_acq_rel_gpu(p.group_done + tg, 1u);
    __syncthreads();
    if (arrived != static_cast<unsigned>(p.E - 1))
        return;
    __threadfence(); // the other CTAs' logits and zeroed weights, for every thread of this one
    for (int t = warp; t < nt; t += kRouteWarps)
        choose(p, t0 + t);
    __syncthreads();
    if (threadIdx.x == 0) {
        p.group_done[tg] = 0u;
        __threadfence();
        arrived = p.wtok != nullptr ? atomic_add_acq_rel_gpu(p.group_done + kMoeMaxTokens / kTG, 1u) : 0xffffffffu;
    }
    __syncthreads();
    if (arrived != static_cast<unsigned>(groups - 1) || p.wtok == nullptr)
        return;
    __threadfence();
    if (warp == 0)
        list_active(p.group_done + kMoeMaxTokens / kTG + 1, p.E, p.active);
    if (threadIdx.x == 0)
        p.group_done[kMoeMaxTokens / kTG] = 0u;
}

// The same bookkeeping for a choice that the caller made: one CTA per expert
// adds up the tokens' weights for it, the last one lists the active experts;
// then the cast's CTAs.  Experts outside [0, E) are skipped; a token that names
// an expert twice gives it the sum of the two weights, in slot order.
__global__ void __launch_bounds__(kRouteThreads) moe_plan_kernel(const RouteParams p)
{
    __shared__ unsigned arrived;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_MOE_PLAN, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) >= p.E) {
        cast_group(p, static_cast<long long>(blockIdx.x - p.E) * kRouteWarps + warp);
        return;
    }
    const int e = blockIdx.x;
    bool any = false;
    if (static_cast<int>(threadIdx.x) < p.M) {
        const int m = threadIdx.x;
        float w = 0.0f;
        for (int j = 0; j < p.top_k; ++j)
            if (p.ids[static_cast<long long>(m) * p.top_k + j] == e) {
                w += p.topw[static_cast<long long>(m) * p.top_k + j];
                any = true;
            }
        p.wtok[static_cast<long long>(e) * p.npad + m] = w;
    }
    const bool used = __syncthreads_or(any);
    if (threadIdx.x == 0) {
        unsigned *mask = p.group_done + kMoeMaxTokens / kTG + 1;
        if (used)
            atomicOr(mask + (e >> 5), 1u << (e & 31));
        __threadfence();
        arrived = atomic_add_acq_rel_gpu(p.group_done, 1u);
    }
    __syncthreads();
    if (arrived != static_cast<unsigned>(p.E - 1))
        return;
    __threadfence();
    if (warp == 0)
        list_active(p.group_done + kMoeMaxTokens / kTG + 1, p.E, p.active);
    if (threadIdx.x == 0)
        p.group_done[0] = 0u;
}

fp8bs_status launch_moe_route(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    RouteParams p = {};
    p.M = L.M;
    p.H = L.H;
    p.E = L.E;
    p.top_k = L.top_k;
    p.npad = moe_token_pad(L.M);
    p.x = static_cast<const uint16_t *>(L.x);
    p.ldx = L.ldx;
    p.wr = L.wr;
    p.renorm = L.renorm;
    p.ids = L.ids;
    p.topw = L.topw;
    p.logits = reinterpret_cast<float *>(L.workspace + w.logits_off);
    const bool layer = L.w13 != nullptr; // the choice alone needs neither the cast nor the plan
    p.wtok = layer ? reinterpret_cast<float *>(L.workspace + w.wtok_off) : nullptr;
    p.group_done = reinterpret_cast<unsigned *>(L.workspace + w.route_off);
    p.active = reinterpret_cast<int *>(L.workspace + w.active_off);
    p.xq = L.workspace + w.xq_off;
    p.xs = reinterpret_cast<float *>(L.workspace + w.xs_off);
    p.runs = dev.runs;
    const long long cast = layer ? (static_cast<long long>(L.M) * (L.H / 128) + kRouteWarps - 1) / kRouteWarps : 0;
    const int groups = (L.M + kTG - 1) / kTG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cast + (L.wr != nullptr ? L.E * groups : L.E)), 1, 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (L.flags & FP8BS_FLAG_OVERLAP_PREV) ? 1 : 0;
    auto kernel = L.wr == nullptr ? moe_plan_kernel
                  : L.wr_type == FP8BS_BF16 ? moe_route_kernel<true>
                                            : moe_route_kernel<false>;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

} // namespace fp8bs
