// moe_scored.cu -- the first kernel of an expert layer whose experts are chosen by
// scores, bias and groups: router product, choice, weights, the sets of experts,
// and the E4M3 cast of the activations beside it (as moe_route.cu).
//
//   l[m, e] = sum_h x[m, h] * wr[e, h]
//   s = sigmoid(l) or softmax(l) over all experts,  c = s + bias
//   groups of E / groups consecutive experts, the top_groups of largest sum of
//   their one or two largest c; ids[m] = the top_k experts of largest c in those
//   w = s of the chosen, over their sum where renormalised, times scale
//
// A logit's products of 256 of H are added up in fp32 (ten roundings on a way: four
// multiply-adds, a sum of two, five levels over the lanes), and so are a warp's turns
// and a CTA's sum in the end: off by at most (10 + H / 256) 2^-24 of the sum of |x wr|, by
// 1.2e-7 in the mean square for normal x and logits of deviation 1.5 (H = 2,048 to
// 20,480).  From the CTAs' sums on logits and scores are pairs of fp32 numbers
// (pair_math.cuh), where fp32 alone would lose more: its own step at a logit of 3 is
// 2^-22, and a score next to 1 has lost the difference of two logits.
//
// Product: a warp holds 256 of H of eight tokens in registers and runs through up
// to eight experts' rows; the eight sums are put together over the lanes by halving
// (nine shuffles for eight sums).  x is read once for those experts, H is split over
// the warps of a CTA and up to four CTAs, whose partial sums the chooser adds in
// order.  The last CTA of a token group chooses for its eight tokens, a warp each;
// arrivals are counted, nobody waits.  A few microseconds of latency, not
// bandwidth, and much of it the fetching of instructions that run once: loops stay
// rolled (the choice unrolled into registers, 74 KB of code, took 21.5 us in all for 8
// tokens of 256 experts and H = 5,120, where its instructions alone would take 1.5;
// this form 10.9, and 14.6 for 64 tokens of 160 experts).
#include <cmath>

#include "moe_route.cuh"
#include "pair_math.cuh"

namespace fp8bs {

struct ScoredParams {
    RouteParams r;
    MoeScores sc;
    int hw, splits, loops; // warps that share H in a CTA, CTAs that do, 256-wide units of a warp
    int ex, sets;          // experts of a warp (2, 4 or 8), CTAs over the experts
};

// Whether the order of the scores plus bias is that of the logits, so that no
// score is needed for the choice (and none loses digits next to 1 or to 0).
__device__ __forceinline__ bool by_logit(const MoeScores &sc)
{
    return sc.bias == nullptr && (sc.top_groups == sc.groups || sc.group_best == 1);
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a + b, the error in `lo` besides what is there.
__device__ __forceinline__ float sum_into(float a, float b, float &lo)
{
    const float s = a + b, t = s - a;
    lo += (a - (s - t)) + (b - t);
    return s;
}

// exp(x + xl) for x <= 0 and |xl| <= 2^-23 |x|, that of -80 below it, as hi + lo
// (pow_split's steps with the product held by an fma); a whole warp calls it, `entry`
// the lane's of kPow32.
__device__ __forceinline__ Pair exp_of(float x, float xl, float2 entry)
{
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0c0p-26f; // log2(e)
    constexpr float k1 = 0x1.62e430p-1f, k2 = 0x1.ebfd1cp-3f, k3 = 0x1.c6b168p-5f; // nearest cubic to 2^y - 1 over y, |y| <= 2^-6
    xl = x >= -80.0f ? xl : 0.0f; // a large number's low part is large, and y has to stay within 2^-6
    x = max_nan(x, -80.0f);
    const float u = fmaf(x, kHi, kShift);
    const uint32_t bits = __float_as_uint(u);
    const float y = fmaf(xl, kHi, fmaf(x, kLo, fmaf(x, kHi, kShift - u)));
    const float th = __shfl_sync(0xffffffffu, entry.x, bits & 31u), tl = __shfl_sync(0xffffffffu, entry.y, bits & 31u);
    const float rest = fmaf(fmaf(fmaf(y, k3, k2), y, k1), y, tl);
    const float hi = __uint_as_float(__float_as_uint(th) + ((bits - static_cast<uint32_t>(kShiftBits)) >> 5 << 23));
    return fast_two_sum(hi, hi * rest); // (rest is up to 2^-6: what divides by this takes low parts for small)
}

// 1 / (1 + a) for 0 <= a <= 2^10.
__device__ __forceinline__ Pair inverse_of_1_plus(Pair a)
{
    const float d = 1.0f + a.hi;
    const float dl = (a.hi >= 1.0f ? 1.0f - (d - a.hi) : a.hi - (d - 1.0f)) + a.lo;
    const float q = rcp_approx(d);
    return {q, q * (fmaf(-q, d, 1.0f) - q * dl)};
}

__device__ __forceinline__ Pair times(Pair a, Pair b)
{
    const float p = a.hi * b.hi;
    return {p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi)};
}

// Bytes from global to shared memory, and the wait for this thread's.
__device__ __forceinline__ void copy_async_4(float *to, const float *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_16(float *to, const float *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A score as one number whose order is the scores': the high part's key, 27 bits of
// the low part's (so 43 bits or more of the value) and 31 - i, which puts lower experts
// of a lane first.  Never 0; NaN is below every number.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t bits_key(float v) // route_key of a number
{
    const uint32_t b = __float_as_uint(v);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ void store_key(Pair s, int i, uint32_t *hi, uint32_t *lo)
{
    const float t = s.hi + s.lo;
    const float rest = s.lo - (t - s.hi);
    *hi = t != t ? 0u : bits_key(t);
    *lo = (bits_key(fabsf(t) < INFINITY ? rest : 0.0f) & ~31u) | static_cast<uint32_t>(31 - i);
}
__device__ __forceinline__ float key_value(uint32_t k) // of route_key
{
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ Key larger(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ Key lesser(Key a, Key b) { return a > b ? b : a; }

// One warp: the choice for token m.  `a`: kMoeMaxSplits planes of E numbers of this
// warp in shared memory, first the partial sums of the logits, then the scores' high
// and low parts (or their keys) and the logits; expert 32 i + lane is the lane's own.
// `mask`: the token group's bit mask of experts (shared).  Four experts of a lane at
// a time: one alone is a chain of 120 dependent instructions.
__device__ __forceinline__ void choose_scored(const ScoredParams &q, int m, float *a, unsigned *mask)
{
    const RouteParams &p = q.r;
    const MoeScores &sc = q.sc;
    const int lane = threadIdx.x & 31, E = p.E;
    const float2 entry = kPow32[lane];
    float *const hi = a, *const lo = a + E, *const l = a + 2 * E;
    uint32_t *const key_hi = reinterpret_cast<uint32_t *>(hi), *const key_lo = reinterpret_cast<uint32_t *>(lo);
    const bool plain = by_logit(sc);
#pragma unroll 1
    for (int s = 0; s < q.splits; ++s) {
        const float *const from = p.logits + (static_cast<long long>(s) * p.M + m) * E;
        if (E % 4 == 0) {
#pragma unroll 1
            for (int e = 4 * lane; e < E; e += 128)
                copy_async_16(a + s * E + e, from + e);
        } else {
#pragma unroll 1
            for (int e = lane; e < E; e += 32)
                copy_async_4(a + s * E + e, from + e);
        }
    }
    copy_async_wait();
    __syncwarp();
    float lmax = -INFINITY, lmax_lo = 0.0f; // the largest logit, NaN aside
#pragma unroll 1
    for (int e0 = lane; e0 < E; e0 += 128) {
        Pair s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i] = {e0 + 32 * i < E ? a[e0 + 32 * i] : 0.0f, 0.0f};
#pragma unroll 1
        for (int k = 1; k < q.splits; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[i].hi = sum_into(s[i].hi, e0 + 32 * i < E ? a[k * E + e0 + 32 * i] : 0.0f, s[i].lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + 32 * i;
            if (e < E) {
                const bool finite = fabsf(s[i].hi) < INFINITY;
                const float t = finite ? s[i].hi + s[i].lo : s[i].hi;
                const float rest = finite ? s[i].lo - (t - s[i].hi) : 0.0f;
                l[e] = t;
                lmax_lo = t > lmax || (t == lmax && rest > lmax_lo) ? rest : lmax_lo;
                lmax = fmaxf(lmax, t);
                if (plain) {
                    store_key({t, rest}, e >> 5, key_hi + e, key_lo + e);
                } else {
                    hi[e] = t;
                    lo[e] = rest;
                }
            }
        }
    }
    const float lane_max = lmax;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    // Softmax: exp(l - lmax) and its sum; then (sigmoid: at once) the scores.  Sigmoid goes
    // through exp(-|l|), which cannot overflow.
    Pair inv = {1.0f, 0.0f};
    if (!plain && !sc.sigmoid) {
        // l - lmax with both low parts: logits of 2^24 and more differ by units there
        lmax_lo = lane_max == lmax ? lmax_lo : -INFINITY;
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1)
            lmax_lo = fmaxf(lmax_lo, __shfl_xor_sync(0xffffffffu, lmax_lo, o));
        Pair all = {0.0f, 0.0f};
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 64) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = e0 + 32 * i + lane;
                const bool there = e < E;
                float dl = there ? lo[e] - lmax_lo : 0.0f;
                const float d = sum_into(there ? hi[e] : lmax, -lmax, dl);
                Pair x = two_sum(d, fabsf(d) < INFINITY ? dl : 0.0f);
                if (x.hi > 0.0f) // by a rounding of the low parts' difference
                    x = {0.0f, 0.0f};
                const Pair s = exp_of(x.hi, x.lo, entry);
                if (there) {
                    all.hi = sum_into(all.hi, s.hi, all.lo);
                    all.lo += s.lo;
                    hi[e] = s.hi;
                    lo[e] = s.lo;
                }
            }
        }
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, all.hi, o), w = __shfl_xor_sync(0xffffffffu, all.lo, o);
            all.lo += w;
            all.hi = sum_into(all.hi, h, all.lo);
        }
        inv = inverse_of_1_plus({all.hi - 1.0f, all.lo}); // (the sum is 1 or more, so nothing is lost)
    }
    if (!plain) {
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 128) {
            Pair s[4];
            float b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + 32 * i + lane;
                s[i] = e < E ? Pair{hi[e], lo[e]} : Pair{0.0f, 0.0f};
                b[i] = sc.bias != nullptr && e < E ? __ldg(sc.bias + e) : 0.0f;
            }
            if (sc.sigmoid) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool neg = s[i].hi < 0.0f;
                    const Pair x = exp_of(neg ? s[i].hi : -s[i].hi, neg ? s[i].lo : -s[i].lo, entry);
                    const Pair r = inverse_of_1_plus(x), t = times(x, r);
                    s[i] = {neg ? t.hi : r.hi, neg ? t.lo : r.lo};
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[i] = times(s[i], inv);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + 32 * i + lane;
                s[i].hi = sum_into(s[i].hi, b[i], s[i].lo);
                if (e < E)
                    store_key({s[i].hi, fabsf(s[i].hi) < INFINITY ? s[i].lo : 0.0f}, e >> 5, key_hi + e, key_lo + e);
            }
        }
    }
    __syncwarp();
    auto key_of = [&](int e) { return static_cast<Key>(key_hi[e]) << 32 | key_lo[e]; };
    unsigned taken = 0; // bit i: expert 32 i + lane cannot be chosen (any more)
    if (sc.top_groups < sc.groups) {
        const int per = E / sc.groups;
        int w = 1; // lanes of a group
        while (2 * w * sc.groups <= 32)
            w *= 2;
        const int g = lane / w;
        Key b1 = 0, b2 = 0; // the group's two largest
        if (g < sc.groups) {
#pragma unroll 4
            for (int e = lane % w; e < per; e += w) {
                const Key t = key_of(g * per + e);
                b2 = larger(b2, lesser(b1, t));
                b1 = larger(b1, t);
            }
        }
#pragma unroll 1
        for (int o = w / 2; o > 0; o /= 2) {
            const Key o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = larger(larger(b2, o2), lesser(b1, o1));
            b1 = larger(b1, o1);
        }
        Pair score = {key_value(static_cast<uint32_t>(b1 >> 32)), key_value(static_cast<uint32_t>(b1) & ~31u)};
        if (sc.group_best == 2)
            score = add(score, {key_value(static_cast<uint32_t>(b2 >> 32)), key_value(static_cast<uint32_t>(b2) & ~31u)});
        uint32_t mine_hi, mine_lo;
        store_key(score, 31, &mine_hi, &mine_lo);
        const Key mine = static_cast<Key>(mine_hi) << 32 | mine_lo;
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < sc.groups; ++i) {
            const Key t = __shfl_sync(0xffffffffu, mine, i * w);
            rank += t > mine || (t == mine && i < g) ? 1 : 0;
        }
        const unsigned open = __ballot_sync(0xffffffffu, g < sc.groups && rank < sc.top_groups);
        const unsigned over = (1u << 20) / per + 1; // e / per = e * over >> 20 for e < 512, per <= 512
#pragma unroll 4
        for (int i = 0; 32 * i + lane < E; ++i)
            taken |= (open >> ((((32 * i + lane) * over) >> 20) * w & 31) & 1u) == 0u ? 1u << i : 0u;
    }
    // A lane's three best that are not taken, 0 for none; it looks again only
    // after all of them are.
    Key b1 = 0, b2 = 0, b3 = 0;
    bool look = true;
    int mine_e = 0;
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
        if (look) {
#pragma unroll 4
            for (int i = 0; 32 * i + lane < E; ++i) {
                Key t = (taken >> i & 1u) == 0u ? key_of(32 * i + lane) : 0;
                Key u = lesser(b1, t);
                b1 = larger(b1, t);
                b3 = larger(b3, lesser(b2, u));
                b2 = larger(b2, u);
            }
            look = false;
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(b1 >> 32));
        unsigned at = __ballot_sync(0xffffffffu, b1 != 0 && static_cast<uint32_t>(b1 >> 32) == top);
        if ((at & (at - 1)) != 0u) { // equal high parts: the rest; equal there too: the lowest lane
            const bool in = (at >> lane & 1u) != 0u;
            const uint32_t rest = __reduce_max_sync(0xffffffffu, in ? static_cast<uint32_t>(b1) : 0u);
            at = __ballot_sync(0xffffffffu, in && static_cast<uint32_t>(b1) == rest);
        }
        const int from = __ffs(static_cast<int>(at)) - 1;
        const int i = 31 - static_cast<int>(__shfl_sync(0xffffffffu, static_cast<uint32_t>(b1), from) & 31u);
        mine_e = lane == j ? 32 * i + from : mine_e;
        if (lane == from) {
            taken |= 1u << i;
            b1 = b2;
            b2 = b3;
            b3 = 0;
            look = b1 == 0;
        }
    }
    const bool chosen = lane < p.top_k;
    const float lm = l[mine_e];
    float top = chosen ? lm : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // sigmoid, renormalised: over exp of the largest logit where all are negative, so that not all of them vanish
    const bool neg = !(lm >= 0.0f);
    const float shift = !sc.sigmoid ? (p.renorm ? top : lmax) : p.renorm ? fminf(top, 0.0f) : 0.0f;
    float w = expf(sc.sigmoid && !neg ? -lm : lm - shift);
    if (sc.sigmoid)
        w = __fdiv_rn(neg ? w : 1.0f, 1.0f + (neg ? expf(lm) : w));
    if (p.renorm || !sc.sigmoid) {
        float sum = chosen ? w : 0.0f;
        if (!p.renorm) {
            sum = 0.0f;
#pragma unroll 4
            for (int e = lane; e < E; e += 32)
                sum += expf(l[e] - lmax);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w = __fdiv_rn(w, sum);
    }
    w *= sc.scale;
    if (inv.hi != inv.hi)
        w = inv.hi; // no score of the token is a number: a NaN or infinite logit is in the softmax's sum
    if (chosen) {
        p.ids[static_cast<long long>(m) * p.top_k + lane] = mine_e;
        p.topw[static_cast<long long>(m) * p.top_k + lane] = w;
        if (p.wtok != nullptr) {
            p.wtok[static_cast<long long>(mine_e) * p.npad + m] = w;
            atomicOr(mask + (mine_e >> 5), 1u << (mine_e & 31));
        }
    }
}

// The sums over the warp of eight values a lane: on return the first is that of
// value 4 b4 + 2 b3 + b2 of the lane's number's bits.
__device__ __forceinline__ float sums_of_8(float (&v)[8])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16, n = 4; n >= 1; o /= 2, n /= 2) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n];
            v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// Raw bits of eight router weights of a lane.
template <bool kBf16> struct Weights8 {
    uint4 w[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const RouteParams &p, int e, int h, bool there)
    {
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i)
            w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (there) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.wr) +
                                                               (static_cast<long long>(e) * p.H + h) * (kBf16 ? 2 : 4));
            w[0] = src[0];
            if (!kBf16)
                w[kBf16 ? 0 : 1] = src[1];
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
            const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kBf16) {
                    v[2 * k] = bf16_lo(a[k]);
                    v[2 * k + 1] = bf16_hi(a[k]);
                } else {
                    v[4 * i + k] = __uint_as_float(a[k]);
                }
            }
        }
    }
};

constexpr int kMostEx = 8; // experts of a warp

template <bool kBf16>
__global__ void __launch_bounds__(kRouteThreads, 2) moe_scored_kernel(const __grid_constant__ ScoredParams q)
{
    __shared__ float part[kTG][kMostEx][kTG]; // [warp][expert][token]
    __shared__ unsigned arrived;
    __shared__ unsigned smask[kMoeMaxExperts / 32];
    extern __shared__ __align__(16) float scratch[]; // kMoeMaxSplits planes of E numbers a warp; 16-byte copies go there
    const RouteParams &p = q.r;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_MOE_SCORED, 1ull);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    grid_dependency_wait();
    const int groups = (p.M + kTG - 1) / kTG;
    const int per_group = q.sets * q.splits; // CTAs
    const int routing = per_group * groups;
    if (static_cast<int>(blockIdx.x) >= routing) {
        cast_group(p, static_cast<long long>(blockIdx.x - routing) * (kRouteThreads / 32) + warp);
        return;
    }
    const int tg = blockIdx.x / per_group, in = blockIdx.x - tg * per_group;
    const int set = in / q.splits, split = in - set * q.splits;
    const int share = warp / q.hw; // of the CTA's experts
    const int t0 = tg * kTG;
    const int nt = p.M - t0 < kTG ? p.M - t0 : kTG;
    const int e0 = (set * (kRouteThreads / 32 / q.hw) + share) * q.ex; // this warp's experts
    const uint16_t *const x0 = p.x + static_cast<long long>(t0) * p.ldx;
#pragma unroll 1
    for (int n = 0; n < q.loops; ++n) {
        const int h = ((n * q.splits + split) * q.hw + warp - share * q.hw) * 256 + lane * 8;
        const bool in_row = h < p.H;
        uint4 xr[kTG];
#pragma unroll
        for (int t = 0; t < kTG; ++t) {
            xr[t] = make_uint4(0u, 0u, 0u, 0u);
            if (in_row && t < nt)
                xr[t] = *reinterpret_cast<const uint4 *>(x0 + static_cast<long long>(t) * p.ldx + h);
        }
        Weights8<kBf16> next[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            next[i].load(p, e0 + i, h, in_row && e0 + i < p.E);
        float x[kTG][8];
#pragma unroll
        for (int t = 0; t < kTG; ++t) {
            const uint32_t a[4] = {xr[t].x, xr[t].y, xr[t].z, xr[t].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[t][2 * i] = bf16_lo(a[i]);
                x[t][2 * i + 1] = bf16_hi(a[i]);
            }
        }
#pragma unroll 1
        for (int k = 0; k < q.ex; k += 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float w[8], v[kTG];
                next[i].values(w);
                const int e = e0 + k + 2 + i;
                next[i].load(p, e, h, in_row && k + 2 < q.ex && e < p.E);
#pragma unroll
                for (int t = 0; t < kTG; ++t) {
                    float a = 0.0f, b = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        fma2(a, b, x[t][j], x[t][j + 1], w[j], w[j + 1]);
                    v[t] = a + b;
                }
                const float sum = sums_of_8(v);
                float *const to = &part[warp][k + i][lane >> 2];
                if ((lane & 3) == 0)
                    *to = n == 0 ? sum : *to + sum;
            }
        }
    }
    __syncthreads();
    // the warps that share H, in order; a thread per (share of the experts, expert, token)
    const int shares = kRouteThreads / 32 / q.hw;
#pragma unroll 1
    for (int i = threadIdx.x; i < shares * q.ex * kTG; i += kRouteThreads) {
        const int t = i % kTG, s = i / (kTG * q.ex), k = i / kTG - s * q.ex;
        const int e = (set * shares + s) * q.ex + k;
        if (t < nt && e < p.E) {
            Pair a = {part[s * q.hw][k][t], 0.0f};
            for (int j = 1; j < q.hw; ++j) {
                const Pair b = two_sum(a.hi, part[s * q.hw + j][k][t]);
                a = {b.hi, a.lo + b.lo};
            }
            __stcg(p.logits + (static_cast<long long>(split) * p.M + t0 + t) * p.E + e, a.hi + a.lo);
            if (p.wtok != nullptr && split == 0)
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
    __threadfence(); // the other CTAs' sums and zeroed weights, for every thread of this one
    if (warp < nt)
        choose_scored(q, t0 + warp, scratch + warp * kMoeMaxSplits * p.E, smask);
    if (threadIdx.x == 0)
        p.group_done[tg] = 0u;
    __syncthreads();
    if (p.wtok != nullptr && threadIdx.x < kMoeMaxExperts / 32)
        p.masks[tg * (kMoeMaxExperts / 32) + threadIdx.x] = smask[threadIdx.x];
}

fp8bs_status launch_moe_scored(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    ScoredParams q = {};
    q.r = route_params(L, w, dev);
    q.sc = L.scores;
    constexpr int kWarps = kRouteThreads / 32;
    const int units = (L.H + 255) / 256;
    const int groups = (L.M + kTG - 1) / kTG;
    // Warps that share H, CTAs that do, experts of a warp: the least of a wave's fixed time (about 2 us: launch, first
    // loads, arrival) and a unit's (0.8 us and 0.2 for each expert), in fifths of a microsecond, two CTAs an SM.  Of ten
    // shapes from 1 x 64 to 64 x 512 it takes the best of the 30 to 48 choices, or one that is up to 4 % slower; the
    // worst takes 2 to 16 times as long.
    long long best = 0;
    for (int hw = kWarps; hw >= 1; hw /= 2)
        for (int splits = 1; splits <= kMoeMaxSplits; ++splits)
            for (int ex = kMostEx; ex >= 2; ex /= 2) {
                const int loops = (units + hw * splits - 1) / (hw * splits);
                if ((splits > 1 && units <= hw * (splits - 1)) || (hw > 1 && units <= hw / 2))
                    continue; // a CTA or half of the warps would have nothing to do
                const long long sets = (L.E + ex * (kWarps / hw) - 1) / (ex * (kWarps / hw));
                const long long waves = (sets * splits * groups + 2 * dev.sms - 1) / (2 * dev.sms);
                const long long cost = waves * (10 + static_cast<long long>(loops) * (4 + ex));
                if (best == 0 || cost < best) {
                    best = cost;
                    q.hw = hw;
                    q.splits = splits;
                    q.ex = ex;
                    q.loops = loops;
                    q.sets = static_cast<int>(sets);
                }
            }
    const long long cast = L.w13 != nullptr ? (static_cast<long long>(L.M) * (L.H / 128) + kWarps - 1) / kWarps : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cast + static_cast<long long>(q.sets) * q.splits * groups), 1, 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(kTG) * L.E * kMoeMaxSplits * 4;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (L.flags & FP8BS_FLAG_OVERLAP_PREV) ? 1 : 0;
    const bool bf = L.wr_type == FP8BS_BF16;
    auto kernel = bf ? moe_scored_kernel<true> : moe_scored_kernel<false>;
    static unsigned long long done[2];
    const fp8bs_status st = ensure_smem_attr(reinterpret_cast<const void *>(kernel), kTG * kMoeMaxExperts * kMoeMaxSplits * 4, dev.device,
                                             done + (bf ? 1 : 0));
    return st != FP8BS_OK ? st : launch_status(cudaLaunchKernelEx(&cfg, kernel, q));
}

} // namespace fp8bs
