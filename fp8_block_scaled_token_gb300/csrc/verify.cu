// verify.cu -- verification of drafted tokens against the target model's
// logits, from given random numbers, and the choice of the next token.
//
//   p_j = softmax(x_j / T) of a sequence's rows j = 0 .. len (T = 0: all of it on
//   the largest logit, the lowest index among equals)
//   draft j is accepted where u_j q_j(t_j) < p_j(t_j); at the first that is not,
//   the next token is drawn from max(p_j - q_j, 0), or after the last from p_len:
//   the first index whose cumulative weight passes r times the total.
//
// The choice is a whole number that a cumulative sum over up to a million
// entries decides, so the weights are held to 2^-28 of themselves, 2^-31 in the
// mean (two fp32 numbers), and summed as 64-bit integers in units of 2^-48 (a
// chunk, relative to a power of two near its largest) and 2^-41 (a row): integer
// sums have no order, which makes the result bitwise reproducible.
//
// w(x) = 2^((x - ref) c), c = log2(e) / T as two fp32 numbers.  |ref| is no
// smaller than |x| for every x that counts, so that t = fl(x - ref) and e = x -
// (t + ref) are exact (fast two-sum); z = t c + e c in two fp32 numbers, and
// 2^z as in pair_math.cuh.
//
// verify_stats_kernel: a CTA per (row, 8,192 logits), rows in the order of
// their positions.  Maximum, then the sum of the weights, from registers: one
// read.  The last CTA of a row puts the chunks together and decides the draft.
// A row that is not accepted leaves its position in the sequence's word, and
// CTAs of later positions that start after that have nothing to do.
// verify_choose_kernel: a CTA per (sequence, chunk).  The chunk that holds the
// target weight looks for the token; with the draft's probabilities all chunks
// sum max(p - q, 0) first and the last one looks.  Nothing waits.
#include <cmath>

#include "fp8bs_testing.h"
#include "internal.h"
#include "pair_math.cuh"
#include "ptx.cuh"

namespace fp8bs {

constexpr int kVerifyThreads = 256;
constexpr int kChunk = 8192;      // logits of a CTA
constexpr int kVerifyMaxDraft = 31;
constexpr int kVerifyMaxRows = 4096;
constexpr int kVerifyMaxVocab = 1 << 20;
constexpr float kChunkUnits = 281474976710656.0f;  // 2^48
constexpr float kRowUnits = 2199023255552.0f;      // 2^41: a row's total stays below 2^62

struct ChunkStat {
    float top;       // largest logit; NaN where the chunk holds a NaN or +infinity
    int exponent;    // the sum's unit is 2^(exponent - 48)
    long long sum;   // after the row is put together: in the row's units; T = 0: the index of `top`
};

struct RowStat {
    int verdict;     // 1 accepted, 0 not (or no draft at this position), 2 no distribution
    int exponent;    // weights are relative to 2^exponent
    float top;       // largest logit
    int best;        // T = 0: its index
    long long total; // of the weights, in row units
    float prob;      // of the drafted token
    int pad;
};

struct VerifyParams {
    int B, L, V, chunks;
    const uint8_t *logits;
    long long ldl; // logits
    const int32_t *draft, *draft_len;
    const float *q;
    long long ldq;
    const float *accept_u, *sample_u, *temperature;
    int32_t *tokens, *accepted;
    float *probs;
    unsigned *row_done, *stopped, *seq_done; // zero between calls
    ChunkStat *chunk;
    RowStat *row;
    long long *residual; // [B][chunks]
    unsigned long long *runs;
};

// Temperature and reference of one row (or chunk), and a lane's table entry.
struct Scale {
    float ch, cl; // log2(e) / T
    float T;
};

__device__ __forceinline__ Scale make_scale(float T)
{
    Scale s;
    s.T = T;
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0c0p-26f; // log2(e)
    s.ch = __fdiv_rn(kHi, T);
    s.cl = __fdiv_rn(fmaf(-s.ch, T, kHi) + kLo, T);
    return s;
}

// Temperatures that are taken: 0, or those that keep every step in range.
__device__ __forceinline__ bool good_temperature(float T) { return T == 0.0f || (T >= 9.5367432e-07f && T <= 1048576.0f); }

// The reference for logits up to `top`: no smaller in magnitude than any logit
// above the cutoff.
__device__ __forceinline__ float reference(float top, float T) { return top >= 0.0f ? top + 128.0f * T : top - 128.0f * T; }
__device__ __forceinline__ float cutoff(float top, float T) { return top - 64.0f * T; } // weights below 2^-92 count as 0

// z = (x - ref) c for x above the cutoff.
__device__ __forceinline__ void exponent_of(float x, float ref, const Scale &s, float &zh, float &zl)
{
    const float t = x - ref;
    const float e = x - (t + ref);
    zh = t * s.ch;
    zl = fmaf(e, s.ch, fmaf(t, s.cl, fmaf(t, s.ch, -zh)));
}

// The weight of x relative to 2^exponent as hi + lo (0 below the cutoff); a
// whole warp calls it.
__device__ __forceinline__ void weight(float x, float top, float ref, float cut, int exponent, const Scale &s,
                                       float2 entry, float &hi, float &lo)
{
    const bool live = x >= cut;
    float zh, zl, th, rest;
    exponent_of(live ? x : top, ref, s, zh, zl);
    const int n = pow_split(zh, zl, entry, th, rest);
    hi = live ? __uint_as_float(__float_as_uint(th) + (static_cast<uint32_t>(n - exponent) << 23)) : 0.0f;
    lo = hi * rest;
}

__device__ __forceinline__ long long fixed(float hi, float lo, float units)
{
    return __float2ll_rn(hi * units) + __float2ll_rn(lo * units);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One row's logits, in 16-byte words counted from the aligned address at or
// before its first.
template <bool kBf16> struct Row {
    static constexpr int kPer = kBf16 ? 8 : 4;                     // logits of a word
    static constexpr int kWords = kChunk / kPer / kVerifyThreads;  // words of a thread
    const uint8_t *words;
    int lead; // logits that the first word has before the row
    int V;

    __device__ __forceinline__ Row(const VerifyParams &p, long long row)
    {
        constexpr int kSize = kBf16 ? 2 : 4;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p.logits) + static_cast<uintptr_t>(row * p.ldl * kSize);
        words = reinterpret_cast<const uint8_t *>(a & ~static_cast<uintptr_t>(15));
        lead = static_cast<int>(a & 15) / kSize;
        V = p.V;
    }
    __device__ __forceinline__ int index(int word) const { return word * kPer - lead; } // of its first logit
    // A word; -infinity for what is not in the row (whose memory is not read).
    __device__ __forceinline__ uint4 load(int word) const
    {
        const int i = index(word);
        if (i >= 0 && i + kPer <= V)
            return *reinterpret_cast<const uint4 *>(words + static_cast<long long>(word) * 16);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = kBf16 ? 0xFF80FF80u : 0xFF800000u;
        if (i + kPer > 0 && i < V) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (i + e < 0 || i + e >= V)
                    continue;
                if (kBf16) {
                    const uint32_t h = *reinterpret_cast<const uint16_t *>(words + static_cast<long long>(word) * 16 + e * 2);
                    w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xFFFFu) | (h << 16) : (w[e >> 1] & 0xFFFF0000u) | h;
                } else {
                    w[e & 3] = *reinterpret_cast<const uint32_t *>(words + static_cast<long long>(word) * 16 + e * 4);
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float value(const uint4 &w, int e)
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        if (!kBf16)
            return __uint_as_float(a[e & 3]);
        return __uint_as_float((e & 1) ? a[(e >> 1) & 3] & 0xFFFF0000u : a[(e >> 1) & 3] << 16);
    }
    __device__ __forceinline__ float at(int i) const // one logit
    {
        const long long k = static_cast<long long>(i) + lead;
        if (kBf16)
            return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(words + k * 2)) << 16);
        return *reinterpret_cast<const float *>(words + k * 4);
    }
};

__device__ __forceinline__ float temperature(const VerifyParams &p, int b)
{
    return p.temperature == nullptr ? 1.0f : p.temperature[b];
}

__device__ __forceinline__ int drafted(const VerifyParams &p, int b) // tokens of sequence b
{
    if (p.draft_len == nullptr)
        return p.L;
    const int n = p.draft_len[b];
    return n < 0 ? 0 : n > p.L ? p.L : n;
}

// Whether an earlier position of the sequence has stopped it.  The word holds
// 64 - position of the earliest so far, 0 for none.
__device__ __forceinline__ bool behind_a_stop(const VerifyParams &p, int b, int j)
{
    const unsigned s = load_acquire_gpu(p.stopped + b);
    return s != 0u && 64 - static_cast<int>(s) < j;
}

// The row's chunks put together, and the verdict on its draft; one warp.
template <bool kBf16>
__device__ __forceinline__ void finish_row(const VerifyParams &p, int b, int j, int len, const Row<kBf16> &x)
{
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(b) * (p.L + 1) + j;
    ChunkStat *const st = p.chunk + row * p.chunks;
    const float T = temperature(p, b);
    const float2 entry = kPow32[lane];
    float top = -INFINITY;
    for (int c = lane; c < p.chunks; c += 32)
        top = max_nan(top, __ldcg(&st[c].top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    RowStat r = {};
    r.top = top;
    if (!(top > -INFINITY && top < INFINITY) || !good_temperature(T)) {
        r.verdict = 2;
    } else {
        const int t = j < len ? p.draft[static_cast<long long>(b) * p.L + j] : -1;
        const bool inside = t >= 0 && t < p.V;
        double wt = 0.0, total = 1.0; // the drafted token's weight and that of all
        if (T == 0.0f) {
            int best = 0x7fffffff;
            for (int c = lane; c < p.chunks; c += 32)
                if (__ldcg(&st[c].top) == top)
                    best = min(best, static_cast<int>(__ldcg(&st[c].sum)));
            best = __reduce_min_sync(0xffffffffu, best);
            r.best = best;
            wt = t == best ? 1.0 : 0.0;
        } else {
            const Scale s = make_scale(T);
            const float ref = reference(top, T), cut = cutoff(top, T);
            float zh, zl, th, rest;
            exponent_of(top, ref, s, zh, zl);
            r.exponent = pow_split(zh, zl, entry, th, rest);
            long long sum = 0;
            for (int c0 = 0; c0 < p.chunks; c0 += 32) {
                const int c = c0 + lane;
                const float ctop = c < p.chunks ? __ldcg(&st[c].top) : -INFINITY;
                const bool live = ctop >= cut;
                // the chunk's reference seen from the row's, by a two-sum without conditions
                const float cref = live ? reference(ctop, T) : ref;
                const float d = cref - ref, bb = d - cref;
                const float e = (cref - (d - bb)) + (-ref - bb);
                zh = d * s.ch;
                zl = fmaf(e, s.ch, fmaf(d, s.cl, fmaf(d, s.ch, -zh)));
                const int n = pow_split(zh, zl, entry, th, rest);
                long long g = 0;
                if (live) {
                    const int k = __ldcg(&st[c].exponent) + n - r.exponent + 41 - 48;
                    const double f = (static_cast<double>(th) + static_cast<double>(th * rest)) *
                                     static_cast<double>(__ldcg(&st[c].sum));
                    g = k < -200 ? 0 : __double2ll_rn(f * __hiloint2double((1023 + k) << 20, 0));
                }
                if (c < p.chunks) {
                    __stcg(&st[c].sum, g);
                    sum += g;
                }
            }
            r.total = warp_sum(sum);
            total = static_cast<double>(r.total);
            if (inside) {
                float hi, lo;
                weight(x.at(t), top, ref, cut, r.exponent, s, entry, hi, lo);
                wt = (static_cast<double>(hi) + static_cast<double>(lo)) * static_cast<double>(kRowUnits);
            }
        }
        if (j < len) {
            const long long d = static_cast<long long>(b) * p.L + j;
            const double q = p.q == nullptr ? 1.0 : inside ? static_cast<double>(p.q[d * p.ldq + t]) : 0.0;
            r.prob = static_cast<float>(wt / total);
            r.verdict = inside && static_cast<double>(p.accept_u[d]) * q * total < wt ? 1 : 0;
        }
    }
    if (lane == 0) {
        p.row[row] = r;
        if (r.verdict != 1)
            atomicMax(p.stopped + b, static_cast<unsigned>(64 - j));
    }
}

template <bool kBf16> __global__ void __launch_bounds__(kVerifyThreads) verify_stats_kernel(const VerifyParams p)
{
    using R = Row<kBf16>;
    __shared__ float wtop[kVerifyThreads / 32];
    __shared__ long long wsum[kVerifyThreads / 32];
    __shared__ int skip, finish;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_VERIFY_STATS, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x % p.chunks);
    const int rank = static_cast<int>(blockIdx.x / p.chunks);
    const int j = rank / p.B, b = rank % p.B;
    const int len = drafted(p, b);
    if (j > len)
        return;
    if (threadIdx.x == 0)
        skip = behind_a_stop(p, b, j) ? 1 : 0;
    __syncthreads();
    const long long row = static_cast<long long>(b) * (p.L + 1) + j;
    const R x(p, row);
    if (skip == 0) {
        const int w0 = c * (kChunk / R::kPer) + static_cast<int>(threadIdx.x);
        uint4 raw[R::kWords];
#pragma unroll
        for (int s = 0; s < R::kWords; ++s)
            raw[s] = x.load(w0 + s * kVerifyThreads);
        const float T = temperature(p, b);
        const float2 entry = kPow32[lane];
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < R::kWords; ++s)
#pragma unroll
            for (int e = 0; e < R::kPer; ++e)
                top = max_nan(top, R::value(raw[s], e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0)
            wtop[warp] = top;
        __syncthreads();
        top = wtop[0];
#pragma unroll
        for (int i = 1; i < kVerifyThreads / 32; ++i)
            top = max_nan(top, wtop[i]);
        ChunkStat out = {top, 0, 0};
        long long sum = 0;
        if (top > -INFINITY && top < INFINITY && good_temperature(T)) {
            if (T == 0.0f) {
                sum = 0x7fffffff;
#pragma unroll
                for (int s = R::kWords - 1; s >= 0; --s)
#pragma unroll
                    for (int e = R::kPer - 1; e >= 0; --e)
                        if (R::value(raw[s], e) == top)
                            sum = x.index(w0 + s * kVerifyThreads) + e;
                sum = __reduce_min_sync(0xffffffffu, static_cast<int>(sum));
            } else {
                const Scale sc = make_scale(T);
                const float ref = reference(top, T), cut = cutoff(top, T);
                float zh, zl, th, rest;
                exponent_of(top, ref, sc, zh, zl);
                out.exponent = pow_split(zh, zl, entry, th, rest);
                // Weights below 2, at most 32 of them: `high` holds their multiples of 2^-16 exactly,
                // `low` what is left.
                float high = 0.0f, low = 0.0f;
#pragma unroll
                for (int s = 0; s < R::kWords; ++s)
#pragma unroll
                    for (int e = 0; e < R::kPer; ++e) {
                        float hi, lo;
                        weight(R::value(raw[s], e), top, ref, cut, out.exponent, sc, entry, hi, lo);
                        const float q = (hi + 192.0f) - 192.0f;
                        high += q;
                        low += hi - q;
                        low += lo;
                    }
                sum = warp_sum(fixed(high, low, kChunkUnits));
            }
        }
        if (lane == 0)
            wsum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            out.sum = wsum[0];
            for (int i = 1; i < kVerifyThreads / 32; ++i)
                out.sum = T == 0.0f ? min(out.sum, wsum[i]) : out.sum + wsum[i];
            ChunkStat *const to = p.chunk + row * p.chunks + c;
            __stcg(&to->top, out.top);
            __stcg(&to->exponent, out.exponent);
            __stcg(&to->sum, out.sum);
        }
    }
    if (threadIdx.x == 0) {
        const unsigned before = atomic_add_acq_rel_gpu(p.row_done + row, 1u);
        finish = 0;
        if (before == static_cast<unsigned>(p.chunks - 1)) {
            p.row_done[row] = 0u;
            finish = behind_a_stop(p, b, j) ? 0 : 1; // where a chunk was left out, this sees why
        }
    }
    __syncthreads();
    if (finish != 0 && warp == 0) {
        __threadfence();
        finish_row<kBf16>(p, b, j, len, x);
    }
}

// What a drawn token's weight is.
enum VerifyMode { kFromTarget, kWithoutDraft, kResidual };

template <bool kBf16> struct Picker {
    const VerifyParams &p;
    Row<kBf16> x;
    Scale s;
    float top, ref, cut;
    int exponent;
    float2 entry;
    VerifyMode mode;
    int except;     // kWithoutDraft
    const float *q; // kResidual
    float Wh, Wl;   // the row's total, relative to 2^exponent

    // Weight in row units of logit i with value v (whole warps call it).
    __device__ __forceinline__ long long units(float v, int i)
    {
        float hi, lo;
        weight(v, top, ref, cut, exponent, s, entry, hi, lo);
        if (mode == kResidual) {
            const float qi = i >= 0 && i < p.V ? q[i] : 0.0f;
            const float ph = qi * Wh;
            const float pl = fmaf(qi, Wl, fmaf(qi, Wh, -ph));
            const float d = hi - ph, bb = d - hi;
            const float e = (hi - (d - bb)) + (-ph - bb);
            lo = (lo - pl) + e;
            hi = d;
            if (!(hi + lo > 0.0f))
                hi = lo = 0.0f;
        } else if (mode == kWithoutDraft && i == except) {
            hi = lo = 0.0f;
        }
        return fixed(hi, lo, kRowUnits);
    }
};

// The first logit of chunk c whose cumulative weight passes `target`; the last
// one with a weight where rounding leaves none, -1 where none has any.  All
// threads call it and get the answer.
template <bool kBf16>
__device__ __forceinline__ int look(Picker<kBf16> &k, int c, long long target, long long *wsum, int *found)
{
    using R = Row<kBf16>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w0 = c * (kChunk / R::kPer) + static_cast<int>(threadIdx.x) * R::kWords;
    if (threadIdx.x < 2)
        found[threadIdx.x] = threadIdx.x == 0 ? 0x7fffffff : -1;
    long long mine = 0;
    int last = -1;
#pragma unroll 1
    for (int s = 0; s < R::kWords; ++s) {
        const uint4 w = k.x.load(w0 + s);
#pragma unroll
        for (int e = 0; e < R::kPer; ++e) {
            const int i = k.x.index(w0 + s) + e;
            const long long g = k.units(R::value(w, e), i);
            mine += g;
            if (g > 0)
                last = i;
        }
    }
    long long upto = mine; // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o)
            upto += v;
    }
    __syncthreads(); // wsum and found are free, and found is set
    if (lane == 31)
        wsum[warp] = upto;
    if (last >= 0)
        atomicMax(found + 1, last);
    __syncthreads();
    for (int i = 0; i < warp; ++i)
        upto += wsum[i];
    const bool here = upto - mine <= target && target < upto;
    if (__any_sync(0xffffffffu, here)) {
        long long at = upto - mine;
        bool done = !here;
#pragma unroll 1
        for (int s = 0; s < R::kWords; ++s) {
            const uint4 w = k.x.load(w0 + s);
#pragma unroll
            for (int e = 0; e < R::kPer; ++e) {
                const int i = k.x.index(w0 + s) + e;
                at += k.units(R::value(w, e), i);
                if (!done && at > target) {
                    found[0] = i;
                    done = true;
                }
            }
        }
    }
    __syncthreads();
    const int at = found[0] != 0x7fffffff ? found[0] : found[1];
    __syncthreads();
    return at;
}

// Chunk of the target weight sample_u * (sum of `sum(c)`) and what lies before it;
// one warp.  Returns -1 where the sum is not positive.
template <class Sum>
__device__ __forceinline__ int target_chunk(int chunks, float u, Sum sum, long long &target)
{
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int c = lane; c < chunks; c += 32)
        total += sum(c);
    total = warp_sum(total);
    if (total <= 0)
        return -1;
    target = __double2ll_rz(static_cast<double>(u) * static_cast<double>(total));
    target = target < 0 ? 0 : target >= total ? total - 1 : target;
    long long before = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
        const long long g = c0 + lane < chunks ? sum(c0 + lane) : 0;
        long long upto = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += v;
        }
        upto += before;
        const unsigned past = __ballot_sync(0xffffffffu, upto > target);
        if (past != 0u) {
            const int l = __ffs(static_cast<int>(past)) - 1;
            target -= __shfl_sync(0xffffffffu, upto - g, l);
            return c0 + l;
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
}

template <bool kBf16> __global__ void __launch_bounds__(kVerifyThreads) verify_choose_kernel(const VerifyParams p)
{
    using R = Row<kBf16>;
    __shared__ long long wsum[kVerifyThreads / 32];
    __shared__ long long starget;
    __shared__ int found[2], schunk, sn, last_one, swhole;
    __shared__ RowStat sr;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_VERIFY_CHOOSE, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x % p.chunks), b = static_cast<int>(blockIdx.x / p.chunks);
    const int len = drafted(p, b);
    const long long row0 = static_cast<long long>(b) * (p.L + 1);
    if (warp == 0) {
        // the first position that was not accepted (position len never is); rows behind it may be old
        const int v = lane <= len ? __ldcg(&p.row[row0 + lane].verdict) : 0;
        const int n = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, v != 1))) - 1;
        if (c == 0) {
            if (lane < n) {
                p.tokens[row0 + lane] = p.draft[static_cast<long long>(b) * p.L + lane];
                p.probs[row0 + lane] = __ldcg(&p.row[row0 + lane].prob);
            } else if (lane > n && lane <= p.L) {
                p.tokens[row0 + lane] = -1;
                p.probs[row0 + lane] = 0.0f;
            }
            if (lane == 0) {
                p.accepted[b] = n;
                p.stopped[b] = 0u;
            }
        }
        if (lane == 0) {
            sn = n;
            sr = p.row[row0 + n];
        }
    }
    __syncthreads();
    const int n = sn;
    const float T = temperature(p, b);
    if (sr.verdict == 2 || T == 0.0f) {
        if (c == 0 && threadIdx.x == 0) {
            p.tokens[row0 + n] = sr.verdict == 2 ? -1 : sr.best;
            p.probs[row0 + n] = sr.verdict == 2 ? NAN : 1.0f;
        }
        return;
    }
    const ChunkStat *const st = p.chunk + (row0 + n) * p.chunks;
    const float u = p.sample_u[b];
    Picker<kBf16> k = {p, R(p, row0 + n), make_scale(T), sr.top, reference(sr.top, T), cutoff(sr.top, T), sr.exponent,
                       kPow32[lane], kFromTarget, -1, nullptr, 0.0f, 0.0f};
    if (n < len) {
        const int t = p.draft[static_cast<long long>(b) * p.L + n];
        if (p.q != nullptr) {
            k.mode = kResidual;
            k.q = p.q + (static_cast<long long>(b) * p.L + n) * p.ldq;
            const double W = static_cast<double>(sr.total) * (1.0 / static_cast<double>(kRowUnits));
            k.Wh = static_cast<float>(W);
            k.Wl = static_cast<float>(W - static_cast<double>(k.Wh));
        } else if (t >= 0 && t < p.V) {
            k.mode = kWithoutDraft;
            k.except = t;
        }
    }
    bool mine = false; // this CTA looks for the token
    if (k.mode == kResidual) {
        const int w0 = c * (kChunk / R::kPer) + static_cast<int>(threadIdx.x);
        long long sum = 0;
#pragma unroll 1
        for (int s = 0; s < R::kWords; ++s) {
            const uint4 w = k.x.load(w0 + s * kVerifyThreads);
#pragma unroll
            for (int e = 0; e < R::kPer; ++e)
                sum += k.units(R::value(w, e), k.x.index(w0 + s * kVerifyThreads) + e);
        }
        sum = warp_sum(sum);
        if (lane == 0)
            wsum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kVerifyThreads / 32; ++i)
                sum += wsum[i];
            __stcg(p.residual + static_cast<long long>(b) * p.chunks + c, sum);
            const unsigned before = atomic_add_acq_rel_gpu(p.seq_done + b, 1u);
            last_one = before == static_cast<unsigned>(p.chunks - 1);
            if (last_one)
                p.seq_done[b] = 0u;
        }
        __syncthreads();
        if (!last_one)
            return;
        __threadfence();
        mine = true;
    }
    if (warp == 0) {
        long long target = 0;
        int at = -1;
        if (k.mode == kResidual)
            at = target_chunk(p.chunks, u, [&](int i) { return __ldcg(p.residual + static_cast<long long>(b) * p.chunks + i); },
                              target);
        else if (k.mode == kWithoutDraft) {
            float hi, lo;
            weight(k.x.at(k.except), k.top, k.ref, k.cut, k.exponent, k.s, k.entry, hi, lo);
            const long long w = fixed(hi, lo, kRowUnits);
            const int home = (k.except + k.x.lead) / kChunk;
            at = target_chunk(p.chunks, u, [&](int i) {
                const long long g = __ldcg(&st[i].sum);
                return i != home ? g : g > w ? g - w : 0;
            }, target);
        }
        const bool whole = at < 0; // nothing left beside the draft: the target's own distribution
        if (whole)
            at = target_chunk(p.chunks, u, [&](int i) { return __ldcg(&st[i].sum); }, target);
        if (lane == 0) {
            schunk = at;
            starget = target;
            swhole = whole;
        }
    }
    __syncthreads();
    if (swhole)
        k.mode = kFromTarget;
    if (!mine && schunk != c)
        return;
    const int token = look<kBf16>(k, schunk, starget, wsum, found);
    if (warp == 0) {
        float hi, lo;
        weight(token >= 0 ? k.x.at(token) : k.top, k.top, k.ref, k.cut, k.exponent, k.s, k.entry, hi, lo);
        if (lane == 0) {
            p.tokens[row0 + n] = token;
            p.probs[row0 + n] = token < 0 ? NAN
                                          : static_cast<float>((static_cast<double>(hi) + static_cast<double>(lo)) *
                                                               static_cast<double>(kRowUnits) / static_cast<double>(sr.total));
        }
    }
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct VerifyWorkspace {
    size_t counters_bytes, chunk_off, row_off, residual_off, total;
    int chunks;
};

VerifyWorkspace verify_workspace(int B, int L, int V)
{
    auto up256 = [](size_t b) { return (b + 255) / 256 * 256; };
    const size_t rows = static_cast<size_t>(B) * (L + 1);
    VerifyWorkspace w;
    w.chunks = (V + 7 + kChunk - 1) / kChunk; // a row may start up to seven logits into its first word
    w.counters_bytes = (rows + 2 * static_cast<size_t>(B)) * 4;
    w.chunk_off = kCountersOff + counters_region(w.counters_bytes);
    w.row_off = w.chunk_off + up256(rows * w.chunks * sizeof(ChunkStat));
    w.residual_off = w.row_off + up256(rows * sizeof(RowStat));
    w.total = w.residual_off + up256(static_cast<size_t>(B) * w.chunks * 8);
    return w;
}
static_assert((kVerifyMaxRows + 2 * kVerifyMaxRows) * 4 <= kCountersRegion, "every size's counters lie in the shared region");
static_assert(sizeof(ChunkStat) == 16 && sizeof(RowStat) == 32, "workspace layout");

fp8bs_status check_verify(int B, int L, int V)
{
    if (B < 1 || L < 0 || V < 1)
        return FP8BS_ERR_INVALID_ARG;
    if (L > kVerifyMaxDraft || V > kVerifyMaxVocab || static_cast<long long>(B) * (L + 1) > kVerifyMaxRows)
        return FP8BS_ERR_UNSUPPORTED_SHAPE;
    return FP8BS_OK;
}

} // namespace

} // namespace fp8bs

using namespace fp8bs;

extern "C" {

fp8bs_status speculative_verify_workspace_size(int B, int L, int V, size_t *bytes)
{
    if (!bytes)
        return FP8BS_ERR_INVALID_ARG;
    *bytes = 0;
    fp8bs_status st = check_verify(B, L, V);
    if (st != FP8BS_OK)
        return st;
    *bytes = verify_workspace(B, L, V).total;
    return FP8BS_OK;
}

fp8bs_status speculative_verify(const void *logits, fp8bs_dtype logits_type, int ldl, const int32_t *draft,
                                const int32_t *draft_len, const float *draft_probs, int ldq,
                                const float *accept_u, const float *sample_u, const float *temperature, int B, int L,
                                int V, int32_t *tokens, int32_t *accepted, float *probs, void *workspace,
                                size_t workspace_bytes, unsigned flags, void *stream)
{
    if (!logits || !sample_u || !tokens || !accepted || !probs || !workspace ||
        (logits_type != FP8BS_F32 && logits_type != FP8BS_BF16))
        return FP8BS_ERR_INVALID_ARG;
    fp8bs_status st = check_verify(B, L, V);
    if (st != FP8BS_OK)
        return st;
    if (ldl < V || (L > 0 && (!draft || !accept_u)) || (L == 0 && (draft || accept_u || draft_len || draft_probs)) ||
        (draft_probs && ldq < V) || (flags & ~FP8BS_FLAG_OVERLAP_PREV) != 0)
        return FP8BS_ERR_INVALID_ARG;
    if (!aligned(logits, logits_type == FP8BS_BF16 ? 2 : 4) || !aligned(draft, 4) || !aligned(draft_len, 4) ||
        !aligned(draft_probs, 4) || !aligned(accept_u, 4) || !aligned(sample_u, 4) || !aligned(temperature, 4) ||
        !aligned(tokens, 4) || !aligned(accepted, 4) || !aligned(probs, 4) || !aligned(workspace, 256))
        return FP8BS_ERR_MISALIGNED;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != FP8BS_OK)
        return st;
    const VerifyWorkspace w = verify_workspace(B, L, V);
    if (workspace_bytes < w.total)
        return FP8BS_ERR_WORKSPACE_TOO_SMALL;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    VerifyParams p = {};
    p.B = B;
    p.L = L;
    p.V = V;
    p.chunks = w.chunks;
    p.logits = static_cast<const uint8_t *>(logits);
    p.ldl = ldl;
    p.draft = draft;
    p.draft_len = draft_len;
    p.q = draft_probs;
    p.ldq = ldq;
    p.accept_u = accept_u;
    p.sample_u = sample_u;
    p.temperature = temperature;
    p.tokens = tokens;
    p.accepted = accepted;
    p.probs = probs;
    p.row_done = reinterpret_cast<unsigned *>(ws + kCountersOff);
    p.stopped = p.row_done + static_cast<size_t>(B) * (L + 1);
    p.seq_done = p.stopped + B;
    p.chunk = reinterpret_cast<ChunkStat *>(ws + w.chunk_off);
    p.row = reinterpret_cast<RowStat *>(ws + w.row_off);
    p.residual = reinterpret_cast<long long *>(ws + w.residual_off);
    p.runs = dev.runs;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kVerifyThreads, 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(B) * (L + 1) * w.chunks), 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = (flags & FP8BS_FLAG_OVERLAP_PREV) ? 1 : 0;
    const bool bf = logits_type == FP8BS_BF16;
    st = launch_status(cudaLaunchKernelEx(&cfg, bf ? verify_stats_kernel<true> : verify_stats_kernel<false>, p));
    if (st != FP8BS_OK)
        return st;
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(B) * w.chunks), 1, 1);
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, bf ? verify_choose_kernel<true> : verify_choose_kernel<false>, p));
}

} // extern "C"
