// moe_route.cu -- the first kernel of an expert layer: router logits, the
// choice of the experts and their weights, the sets of experts that the tokens
// chose, and the E4M3 cast of the activations (which does not depend on the
// choice and runs beside it).
//
//   l[m, e] = sum_h x[m, h] * wr[e, h]                    (fp32)
//   ids[m]  = the top_k experts of largest l, descending, ties to the lowest
//             expert; NaN logits order below every number
//   w[m, j] = exp(l_j - l_max) / sum exp(l - l_max), the sum over the chosen
//             experts (renormalised) or over all of them
//
// Grid: one CTA per (one or four experts, group of 8 tokens), then the CTAs of
// the cast, a warp per (token, 128 of H).  The last CTA of a token group chooses for its
// eight tokens and leaves a bit mask of the experts they chose; arrivals are
// counted, nobody waits.  A few microseconds of latency, not bandwidth:
// loads are issued for all eight tokens at once, and the choice keeps its
// loops rolled (unrolled code run once costs more in instruction fetches than
// it saves).
#include <cuda_bf16.h>

#include "moe_route.cuh"

namespace fp8bs {

constexpr int kRouteWide = 1024; // at most, for long rows

// One warp: the choice for token m.  Its E logits are in `l` (shared memory);
// kInRegs (E <= 128): each lane keeps the keys of its experts lane, lane + 32,
// ... in registers as well, which makes a round of the choice two warp
// reductions and a few selections (8 of 128 experts: 3.1 -> 1.6 us of the
// layer's critical path).  `mask`: the group's bit mask of experts (shared).
template <bool kInRegs>
__device__ __forceinline__ void choose(const RouteParams &p, int m, const float *l, unsigned *mask)
{
    constexpr int kRegs = kInRegs ? 4 : 1;
    const int lane = threadIdx.x & 31;
    float mine_l = 0.0f, lmax = 0.0f;
    int mine_e = 0;
    // Each lane keeps the best of its experts that are not taken yet (ties to
    // the lowest); only the lane whose expert is taken looks again.
    unsigned taken = 0; // bit i: expert 32 i + lane
    uint32_t key[kRegs];
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
        key[i] = kInRegs && 32 * i + lane < p.E ? route_key(l[32 * i + lane]) : 0u;
    uint32_t k = 0;
    int e = 0x7fffffff;
    auto look = [&]() {
        k = 0;
        e = 0x7fffffff;
        if (kInRegs) {
#pragma unroll
            for (int i = 0; i < kRegs; ++i)
                if (32 * i + lane < p.E && !(taken >> i & 1u) && (e == 0x7fffffff || key[i] > k)) {
                    k = key[i];
                    e = 32 * i + lane;
                }
        } else {
#pragma unroll 1
            for (int i = 0; 32 * i + lane < p.E; ++i) {
                const uint32_t ki = route_key(l[32 * i + lane]);
                if (!(taken >> i & 1u) && (e == 0x7fffffff || ki > k)) {
                    k = ki;
                    e = 32 * i + lane;
                }
            }
        }
    };
    look();
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t kmax = __reduce_max_sync(0xffffffffu, k);
        const int best = static_cast<int>(__reduce_min_sync(0xffffffffu, k == kmax ? static_cast<uint32_t>(e) : 0x7fffffffu));
        if (lane == j)
            mine_e = best;
        if (lane == (best & 31)) {
            taken |= 1u << (best >> 5);
            look();
        }
    }
    mine_l = l[mine_e];
    lmax = __shfl_sync(0xffffffffu, mine_l, 0);
    // exp(l - lmax) / sum; an infinite largest logit gives NaN, as the formula does
    float pj = lane < p.top_k ? expf(mine_l - lmax) : 0.0f;
    float sum = pj;
    if (!p.renorm) {
        sum = 0.0f;
#pragma unroll 1
        for (int i = lane; i < p.E; i += 32)
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
            atomicOr(mask + (mine_e >> 5), 1u << (mine_e & 31));
        }
    }
}

// kEx experts a CTA: one where the CTAs then fill the GPU at most twice (each
// reads its tokens' rows of x from L2: 42 MB at 64 tokens, 64 experts and H =
// 5,120), four otherwise.
// kMost threads at most: kRouteThreads, or kRouteWide for one expert a CTA and
// H above 4,096, where a thread for every eight values of H puts the whole
// row's loads in flight at once (M = 8, 64 experts, H = 5,120: the layer 91.8
// -> 90.9 us; at H = 2,048 the smaller register budget costs 0.2 us).
template <bool kBf16, int kEx, int kMost>
__global__ void __launch_bounds__(kMost) moe_route_kernel(const RouteParams p)
{
    __shared__ float part[kMost / 32][kEx * kTG];
    __shared__ unsigned arrived;
    __shared__ unsigned smask[kMoeMaxExperts / 32];
    __shared__ float logit[kTG][kMoeMaxExperts];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_MOE_ROUTE, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
    const int groups = (p.M + kTG - 1) / kTG;
    const int per_group = (p.E + kEx - 1) / kEx; // CTAs
    const int routing = per_group * groups;
    if (static_cast<int>(blockIdx.x) >= routing) {
        cast_group(p, static_cast<long long>(blockIdx.x - routing) * warps + warp);
        return;
    }
    const int e0 = blockIdx.x % per_group * kEx, tg = blockIdx.x / per_group;
    const int t0 = tg * kTG;
    const int nt = p.M - t0 < kTG ? p.M - t0 : kTG;
    // eight values of H a thread and step, all tokens' loads in flight at once
    // (tokens past the last and experts past E re-read the last; those sums
    // are not used)
    float acc[kEx][kTG];
#pragma unroll
    for (int q = 0; q < kEx; ++q)
#pragma unroll
        for (int t = 0; t < kTG; ++t)
            acc[q][t] = 0.0f;
    const uint16_t *const x0 = p.x + static_cast<long long>(t0) * p.ldx;
#pragma unroll(kEx == 1 && kMost == kRouteThreads ? 2 : 1)
    for (int h = threadIdx.x * 8; h < p.H; h += threads * 8) {
        uint4 xr[kTG];
#pragma unroll
        for (int t = 0; t < kTG; ++t)
            xr[t] = *reinterpret_cast<const uint4 *>(x0 + static_cast<long long>(t < nt ? t : nt - 1) * p.ldx + h);
        uint4 wr[kEx][kBf16 ? 1 : 2];
#pragma unroll
        for (int q = 0; q < kEx; ++q) {
            const long long e = e0 + q < p.E ? e0 + q : p.E - 1;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wr) +
                                                               (e * p.H + h) * (kBf16 ? 2 : 4));
            wr[q][0] = src[0];
            if (!kBf16)
                wr[q][kBf16 ? 0 : 1] = src[1];
        }
#pragma unroll
        for (int q = 0; q < kEx; ++q) {
            float w[8];
            if (kBf16) {
                const uint32_t rw[4] = {wr[q][0].x, wr[q][0].y, wr[q][0].z, wr[q][0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[2 * i] = bf16_lo(rw[i]);
                    w[2 * i + 1] = bf16_hi(rw[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 r = wr[q][kBf16 ? 0 : i];
                    w[4 * i] = __uint_as_float(r.x);
                    w[4 * i + 1] = __uint_as_float(r.y);
                    w[4 * i + 2] = __uint_as_float(r.z);
                    w[4 * i + 3] = __uint_as_float(r.w);
                }
            }
#pragma unroll
            for (int t = 0; t < kTG; ++t) {
                const uint32_t xw[4] = {xr[t].x, xr[t].y, xr[t].z, xr[t].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[q][t] = fmaf(bf16_lo(xw[i]), w[2 * i], acc[q][t]);
                    acc[q][t] = fmaf(bf16_hi(xw[i]), w[2 * i + 1], acc[q][t]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int q = 0; q < kEx; ++q)
#pragma unroll
            for (int t = 0; t < kTG; ++t)
                acc[q][t] += __shfl_xor_sync(0xffffffffu, acc[q][t], o);
    }
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < kEx; ++q)
#pragma unroll
            for (int t = 0; t < kTG; ++t)
                part[warp][q * kTG + t] = acc[q][t];
    }
    __syncthreads();
    if (threadIdx.x < kEx * kTG) {
        const int t = threadIdx.x % kTG, e = e0 + threadIdx.x / kTG;
        if (t < nt && e < p.E) {
            float s = part[0][threadIdx.x];
            for (int i = 1; i < warps; ++i)
                s += part[i][threadIdx.x];
            __stcg(p.logits + static_cast<long long>(t0 + t) * p.E + e, s);
            if (p.wtok != nullptr)
                __stcg(p.wtok + static_cast<long long>(e) * p.npad + t0 + t, 0.0f);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        arrived = atomic_add_acq_rel_gpu(p.group_done + tg, 1u);
    if (threadIdx.x < kMoeMaxExperts / 32)
        smask[threadIdx.x] = 0u;
    __syncthreads();
    if (arrived != static_cast<unsigned>(per_group - 1))
        return;
    __threadfence(); // the other CTAs' logits and zeroed weights, for every thread of this one
    if (warp < nt) {
        float *const l = logit[warp];
        for (int i = lane; i < p.E; i += 32)
            l[i] = __ldcg(p.logits + static_cast<long long>(t0 + warp) * p.E + i);
        __syncwarp();
        if (p.E <= 128)
            choose<true>(p, t0 + warp, l, smask);
        else
            choose<false>(p, t0 + warp, l, smask);
    }
    if (threadIdx.x == 0)
        p.group_done[tg] = 0u;
    __syncthreads();
    if (p.wtok != nullptr && threadIdx.x < kMoeMaxExperts / 32)
        p.masks[tg * (kMoeMaxExperts / 32) + threadIdx.x] = smask[threadIdx.x];
}

// The same bookkeeping for a choice that the caller made: one CTA per expert
// adds up the tokens' weights for it, the last one leaves the mask of all;
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
        cast_group(p, static_cast<long long>(blockIdx.x - p.E) * (kRouteThreads / 32) + warp);
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
        unsigned *mask = p.group_done + kMoeMaxTokens / kTG;
        if (used)
            atomicOr(mask + (e >> 5), 1u << (e & 31));
        __threadfence();
        arrived = atomic_add_acq_rel_gpu(p.group_done, 1u);
    }
    __syncthreads();
    if (arrived != static_cast<unsigned>(p.E - 1))
        return;
    __threadfence();
    if (threadIdx.x < kMoeMaxExperts / 32)
        p.masks[threadIdx.x] = atomicExch(p.group_done + kMoeMaxTokens / kTG + threadIdx.x, 0u);
    if (threadIdx.x == 0)
        p.group_done[0] = 0u;
}

RouteParams route_params(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
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
    p.masks = reinterpret_cast<unsigned *>(L.workspace + w.masks_off);
    p.xq = L.workspace + w.xq_off;
    p.xs = reinterpret_cast<float *>(L.workspace + w.xs_off);
    p.runs = dev.runs;
    return p;
}

fp8bs_status launch_moe_route(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    if (L.scores.scored)
        return launch_moe_scored(L, w, dev);
    const RouteParams p = route_params(L, w, dev);
    const bool layer = L.w13 != nullptr;
    const int groups = (L.M + kTG - 1) / kTG;
    const bool four = L.E * groups > 2 * dev.sms; // experts a CTA
    const bool wide = L.wr != nullptr && !four && L.H > 4096;
    const int threads = !wide ? kRouteThreads : L.H >= 8 * kRouteWide ? kRouteWide : (L.H / 8 + 31) / 32 * 32;
    const int warps = threads / 32;
    const long long cast = layer ? (static_cast<long long>(L.M) * (L.H / 128) + warps - 1) / warps : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cast + (L.wr == nullptr ? L.E : (four ? (L.E + 3) / 4 : L.E) * groups)), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (L.flags & FP8BS_FLAG_OVERLAP_PREV) ? 1 : 0;
    const bool bf = L.wr_type == FP8BS_BF16;
    auto kernel = L.wr == nullptr ? moe_plan_kernel
                  : four ? (bf ? moe_route_kernel<true, 4, kRouteThreads> : moe_route_kernel<false, 4, kRouteThreads>)
                  : wide ? (bf ? moe_route_kernel<true, 1, kRouteWide> : moe_route_kernel<false, 1, kRouteWide>)
                         : (bf ? moe_route_kernel<true, 1, kRouteThreads> : moe_route_kernel<false, 1, kRouteThreads>);
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

} // namespace fp8bs
