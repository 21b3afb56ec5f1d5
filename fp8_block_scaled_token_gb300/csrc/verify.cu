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
// part of a row, relative to a power of two near its largest) and 2^-41 (a row): integer
// sums have no order, which makes the result bitwise reproducible.
//
// w(x) = 2^((x - ref) c), c = log2(e) / T as two fp32 numbers: z = x c in two
// numbers, 2^z as in pair_math.cuh, weights relative to a power of two.  ref is 0
// while the largest logit's z is below 4096 (nothing is subtracted, and sums
// relative to powers of two add up without another exponential).  Beyond, |ref| is
// no smaller than |x| for every x that counts, so that t = fl(x - ref) and e = x -
// (t + ref) are exact (fast two-sum) and z = t c + e c.
//
// verify_rows_kernel: a warp per part of 1,024 logits of a row, rows in the order
// of their positions.  Maximum, then the sum of the weights, from registers: one
// read, and nothing that another warp has to wait for.  The last CTA of a row puts
// the parts together and decides the draft.  A row that is not accepted leaves its
// position in the sequence's word, and CTAs of later positions that start after
// that have nothing to do.  The last row of a sequence knows where it stops and
// draws the token: it finds the part and looks through it.
// verify_residual_kernel (with the draft's probabilities): for the sequences that
// stopped at a rejected draft, a warp sums max(p - q, 0) over 256 logits at a time;
// a sequence's last CTA finds the 256 and looks through them.  Nothing waits.
//
// 64 sequences of 8 rows of 248,320 take 115 us (196 with a CTA's 8,192 logits and one
// weight at a time, the token drawn by a second kernel), four times what their needed bytes
// take: 19 instructions a logit, at 60 % of the issue slots with the barriers of the CTAs'
// arrivals in between, and 28 % of the memory's rate; 8 sequences 30 us, one 14.5, a
// row of 1,000 9.0, one of 248,320 9.6, which are chains of loads, sums and arrivals.
#include <cmath>

#include "fp8bs_testing.h"
#include "internal.h"
#include "pair_math.cuh"
#include "ptx.cuh"

namespace fp8bs {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
// CTAs to an SM.  4 instead: 64 rows of 248,320 at once 21.9 us, not 21.3, and 512 rows the same 115; but 5 rows 14.2,
// not 14.5, 64 rows with the residual 29.7, not 30.3, and 256 fp32 rows of 128,000 52, not 57.5 (at 48 registers the
// rows' kernel spills 128 bytes for fp32 logits, 24 for bf16)
constexpr int kVerifyCtas = 5;
constexpr int kPart = 1024;         // logits that a warp sums
constexpr int kMostParts = 4;       // of a warp, one after the other
constexpr int kBit = 256;           // logits that a warp sums for the residual
constexpr int kVerifyMaxDraft = 31;
constexpr int kVerifyMaxRows = 4096;
constexpr int kVerifyMaxVocab = 1 << 20;
constexpr int kMaxParts = kVerifyMaxVocab / kPart + 1;
constexpr float kPartUnits = 281474976710656.0f;  // 2^48
constexpr float kRowUnits = 2199023255552.0f;     // 2^41: a row's total stays below 2^62

struct alignas(16) PartStat {
    float top;       // largest logit; NaN where the part holds a NaN or +infinity
    int exponent;    // the sum's unit is 2^(exponent - 48)
    long long sum;   // T = 0: the index of `top`
};

struct alignas(16) RowStat {
    int verdict;     // 1 accepted, 0 not (or no draft at this position), 2 no distribution
    int exponent;    // weights are relative to 2^exponent
    float top;       // largest logit
    int best;        // T = 0: its index
    long long total; // of the weights, in row units
    float prob;      // of the drafted token
    int position;    // sequence's stop: where, -1 with nothing left to draw
    Pair sum;        // the total as two numbers
    int pad[2];
};

struct VerifyParams {
    int B, L, V;
    int parts, chunks;                       // of a row: a CTA's parts are a chunk
    int parts_each;                          // of a warp
    int bits, runs_each, bit_ctas;           // the residual's: of a row, of a warp, CTAs of a row
    unsigned first_wave;                     // CTAs that start at once, before any row can have stopped
    const uint8_t *logits;
    long long ldl; // logits
    const int32_t *draft, *draft_len;
    const float *q;
    long long ldq;
    const float *accept_u, *sample_u, *temperature;
    int32_t *tokens, *accepted;
    float *probs;
    unsigned *row_done, *stopped, *seq_done; // zero between calls
    PartStat *part;                          // [rows][parts]
    long long *in_row;                       // [rows][parts]: the part's sum in row units
    RowStat *row;
    RowStat *stop;                           // [B]
    long long *residual;                     // [B][bits]
    unsigned long long *runs;
};

// Temperature and reference of one row (or part), and a lane's table entry.
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

// The reference for logits up to `top`: 0, or no smaller in magnitude than any
// logit above the cutoff.
__device__ __forceinline__ float reference(float top, const Scale &s)
{
    if (fabsf(top) * s.ch <= 4096.0f)
        return 0.0f;
    return top >= 0.0f ? top + 128.0f * s.T : top - 128.0f * s.T;
}
__device__ __forceinline__ float cutoff(float top, float T) { return top - 64.0f * T; } // weights below 2^-92 count as 0

// z = (x - ref) c for x above the cutoff.
__device__ __forceinline__ void exponent_of(float x, float ref, const Scale &s, float &zh, float &zl)
{
    const float t = x - ref;
    const float e = x - (t + ref);
    zh = t * s.ch;
    zl = fmaf(e, s.ch, fmaf(t, s.cl, fmaf(t, s.ch, -zh)));
}

// The same with reference 0 and x at the cutoff at least, in fewer operations: the
// rounding to n + j/32 and the rest straight from the product, which an fma holds
// exactly; p the cubic nearest to the power series on |y| <= 2^-6 (2^-33).
constexpr float kPow1 = 0x1.62e430p-1f, kPow2 = 0x1.ebfd1cp-3f, kPow3 = 0x1.c6b168p-5f;
__device__ __forceinline__ int pow_direct(float x, const Scale &s, float2 entry, float &th, float &rest)
{
    const float u = fmaf(x, s.ch, kShift);
    const int bits = __float_as_int(u);
    const float y = fmaf(x, s.cl, fmaf(x, s.ch, kShift - u));
    th = __shfl_sync(0xffffffffu, entry.x, bits & 31);
    const float tl = __shfl_sync(0xffffffffu, entry.y, bits & 31);
    rest = fmaf(fmaf(fmaf(y, kPow3, kPow2), y, kPow1), y, tl);
    return (bits - kShiftBits) >> 5;
}

// th, rest and the bits of n of pow_split for x - ref.
__device__ __forceinline__ float4 pow_far(float x, float ref, float ch, float cl, float2 entry)
{
    float zh, zl, th, rest;
    exponent_of(x, ref, {ch, cl, 0.0f}, zh, zl);
    const int n = pow_split(zh, zl, entry, th, rest);
    return make_float4(th, rest, __int_as_float(n), 0.0f);
}

// The weight of x relative to 2^exponent as hi + lo (0 below the cutoff); a
// whole warp calls it.
__device__ __forceinline__ void weight(float x, float top, float ref, float cut, int exponent, const Scale &s,
                                       float2 entry, float &hi, float &lo)
{
    const bool live = x >= cut;
    float th, rest;
    int n;
    if (ref == 0.0f) {
        n = pow_direct(live ? x : top, s, entry, th, rest);
    } else {
        const float4 r = pow_far(live ? x : top, ref, s.ch, s.cl, entry);
        th = r.x;
        rest = r.y;
        n = __float_as_int(r.z);
    }
    hi = live ? __uint_as_float(__float_as_uint(th) + (static_cast<uint32_t>(n - exponent) << 23)) : 0.0f;
    lo = hi * rest;
}

__device__ __forceinline__ long long fixed(float hi, float lo, float units)
{
    return __float2ll_rn(hi * units) + __float2ll_rn(lo * units);
}

// The same for hi and lo between -4 and 4 and row units, without the conversions to 64
// bits, which go through the 64-bit pipe: adding 12 leaves a number's multiples of
// 2^-20 in the sum's low bits, adding 1.5 * 2^-18 those of 2^-41 of what is left.
__device__ __forceinline__ long long row_units(float hi, float lo)
{
    const float a = hi + 12.0f, b = lo + 12.0f;
    const float c = ((hi - (a - 12.0f)) + (lo - (b - 12.0f))) + 5.72204590e-06f;
    constexpr int kA = 0x41400000, kC = 0x36C00000; // the bits of 12 and of 1.5 * 2^-18
    const int whole = (__float_as_int(a) - kA) + (__float_as_int(b) - kA);
    return static_cast<long long>(whole) * 2097152 + (__float_as_int(c) - kC);
}

// row_units of (hi + lo) - (bh + bl), 0 where that is not positive or b is not below
// 4: the whole multiples of 2^-20 of hi and bh apart, their rests with lo - bl.
__device__ __forceinline__ long long difference_units(float hi, float lo, float bh, float bl)
{
    const float a = hi + 12.0f, b = bh + 12.0f, t = lo - bl, d = t + 12.0f;
    const float c = ((hi - (a - 12.0f)) - (bh - (b - 12.0f))) + (t - (d - 12.0f)) + 5.72204590e-06f;
    constexpr int kA = 0x41400000, kC = 0x36C00000;
    const int whole = (__float_as_int(a) - __float_as_int(b)) + (__float_as_int(d) - kA);
    const long long g = static_cast<long long>(whole) * 2097152 + (__float_as_int(c) - kC);
    return bh < 4.0f && g > 0 ? g : 0;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ long long warp_scan(long long v) // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (static_cast<int>(threadIdx.x & 31) >= o)
            v += t;
    }
    return v;
}

// Two fp32 numbers as one operand of the packed instructions.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 pmul(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 padd(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 pfma(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 psub(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A thread's sum of weights: `high` in multiples of 2^-16 below 64, `low` below 1.
__device__ __forceinline__ long long sum_units(float high, float low0, float low1)
{
    // in units of 2^-48, by 32-bit conversions: low's multiples of 2^-30, then the rest
    const float a = rintf(low0 * 1073741824.0f), b = rintf(low1 * 1073741824.0f);
    const float c = fmaf(a, -9.31322575e-10f, low0), d = fmaf(b, -9.31322575e-10f, low1);
    const int mid = __float2int_rn(a) + __float2int_rn(b);
    const int rest = __float2int_rn(c * kPartUnits) + __float2int_rn(d * kPartUnits);
    return (static_cast<long long>(__float2int_rn(high * 65536.0f)) << 32) + static_cast<long long>(mid) * 262144 + rest;
}

// Sums of weights relative to 2^exponent, each below 2 and at most 32 of them a
// thread: `high` holds their multiples of 2^-16 exactly, `low` what is left.
//
// Two logits at a time with reference 0, in packed instructions (half of what
// weight() takes for each).  What lies below the cutoff counts as at it, 2^-92, which
// leaves no trace in the sums.
struct WeightSum {
    f32x2 high, low;
    f32x2 ch, cl;
    float cut;
    uint32_t th; // the lane's table entry with the exponent's and index's offset taken off
    float tl;

    __device__ __forceinline__ WeightSum(float cut_, int exponent, const Scale &s, float2 entry)
    {
        high = low = pack(0.0f, 0.0f);
        ch = pack(s.ch, s.ch);
        cl = pack(s.cl, s.cl);
        cut = cut_;
        th = __float_as_uint(entry.x) - ((threadIdx.x & 31u) << 18) - (static_cast<uint32_t>(exponent) << 23);
        tl = entry.y;
    }
    __device__ __forceinline__ void add(float x0, float x1)
    {
        const f32x2 shift = pack(kShift, kShift), top = pack(192.0f, 192.0f);
        const f32x2 x = pack(fmaxf(x0, cut), fmaxf(x1, cut));
        const f32x2 u = pfma(x, ch, shift);
        const f32x2 y = pfma(x, cl, pfma(x, ch, psub(shift, u)));
        float u0, u1;
        unpack(u, u0, u1);
        const uint32_t b0 = __float_as_uint(u0), b1 = __float_as_uint(u1);
        const uint32_t t0 = __shfl_sync(0xffffffffu, th, b0), t1 = __shfl_sync(0xffffffffu, th, b1);
        const f32x2 r = pack(__shfl_sync(0xffffffffu, tl, b0), __shfl_sync(0xffffffffu, tl, b1));
        const f32x2 rest = pfma(pfma(pfma(y, pack(kPow3, kPow3), pack(kPow2, kPow2)), y, pack(kPow1, kPow1)), y, r);
        // the bits of u are kShiftBits + 32 n + j: shifted, n is at the exponent and j at bits 18 to 22
        const f32x2 hi = pack(__uint_as_float((b0 << 18) + t0), __uint_as_float((b1 << 18) + t1));
        const f32x2 q = psub(padd(hi, top), top);
        high = padd(high, q);
        low = pfma(hi, rest, padd(low, psub(hi, q)));
    }
    __device__ __forceinline__ long long units() const
    {
        float h0, h1, l0, l1;
        unpack(high, h0, h1);
        unpack(low, l0, l1);
        return sum_units(h0 + h1, l0, l1);
    }
};
static_assert((static_cast<uint32_t>(kShiftBits) << 18) == 0u, "kShiftBits leaves the shifted word");

// The word at `at` whose first logit has index i: -infinity for what is not in the
// row of V, whose memory is not read.  Out of line: a row's first and last word.
template <bool kBf16> __device__ __noinline__ uint4 edge_word(const uint8_t *at, int i, int V)
{
    constexpr int kPer = kBf16 ? 8 : 4, kBits = 128 / kPer;
    unsigned long long w0 = kBf16 ? 0xFF80FF80FF80FF80ull : 0xFF800000FF800000ull, w1 = w0;
#pragma unroll 1
    for (int e = 0; e < kPer; ++e)
        if (i + e >= 0 && i + e < V) {
            // the bits in which it differs from -infinity
            const uint32_t b = kBf16 ? *reinterpret_cast<const uint16_t *>(at + e * 2) ^ 0xFF80u
                                     : *reinterpret_cast<const uint32_t *>(at + e * 4) ^ 0xFF800000u;
            const unsigned long long v = static_cast<unsigned long long>(b) << (e * kBits & 63);
            w0 ^= e < kPer / 2 ? v : 0ull;
            w1 ^= e < kPer / 2 ? 0ull : v;
        }
    return make_uint4(static_cast<uint32_t>(w0), static_cast<uint32_t>(w0 >> 32), static_cast<uint32_t>(w1),
                      static_cast<uint32_t>(w1 >> 32));
}

// One row's logits, in 16-byte words counted from the aligned address at or
// before its first.
template <bool kBf16> struct Row {
    static constexpr int kPer = kBf16 ? 8 : 4;                     // logits of a word
    static constexpr int kWords = kPart / kPer / 32;               // words of a lane of a part
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
    __device__ __forceinline__ uint4 whole(int word) const // all of whose logits are in the row
    {
        return *reinterpret_cast<const uint4 *>(words + static_cast<long long>(word) * 16);
    }
    // A word; -infinity for what is not in the row (whose memory is not read).
    __device__ __forceinline__ uint4 load(int word) const
    {
        const int i = index(word);
        return i >= 0 && i + kPer <= V ? whole(word) : edge(word);
    }
    __device__ __forceinline__ uint4 edge(int word) const { return edge_word<kBf16>(words + static_cast<long long>(word) * 16, index(word), V); }
    static __device__ __forceinline__ float value(const uint4 &w, int e)
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        if (!kBf16)
            return __uint_as_float(a[e & 3]);
        return __uint_as_float((e & 1) ? a[(e >> 1) & 3] & 0xFFFF0000u : a[(e >> 1) & 3] << 16);
    }
    static __device__ __forceinline__ float largest(const uint4 &w) // of a word; NaN where one is
    {
        if (kBf16) {
            const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w));
            return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        }
        return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                       max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
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

// sum * f, both in units of their own, as units of 2^(-41) of the row: sum is in
// units of 2^(k - 41), f = th (1 + rest) in [1, 2).
__device__ __forceinline__ long long rescale(long long sum, float th, float rest, int k)
{
    // f in units of 2^-62: th's 24 bits as they are, th * rest (below 2^-5) in units of 2^-36
    const unsigned long long f = (static_cast<unsigned long long>((__float_as_uint(th) & 0x7FFFFFu) | 0x800000u) << 39) +
                                 (static_cast<unsigned long long>(__float2uint_rn(fmaxf(th * rest, 0.0f) * 68719476736.0f)) << 26) -
                                 (static_cast<unsigned long long>(__float2uint_rn(fmaxf(-th * rest, 0.0f) * 68719476736.0f)) << 26);
    const int shift = -k - 2;
    if (shift > 63)
        return 0;
    const unsigned long long v = __umul64hi(static_cast<unsigned long long>(sum), f);
    return static_cast<long long>(shift >= 0 ? v >> shift : v << -shift);
}

// The factor that takes sums of a part (largest logit ctop, exponent cexp) to
// row units, as th, rest and k of rescale; false where the part is below the
// row's cutoff.  A whole warp calls it.
__device__ __forceinline__ bool to_row(float ctop, int cexp, float ref, float cut, int exponent, const Scale &s,
                                       float2 entry, float &th, float &rest, int &k)
{
    const bool live = ctop >= cut;
    // the part's reference seen from the row's, by a two-sum without conditions
    const float cref = live ? reference(ctop, s) : ref;
    const float d = cref - ref, bb = d - cref;
    const float e = (cref - (d - bb)) + (-ref - bb);
    const float zh = d * s.ch;
    const float zl = fmaf(e, s.ch, fmaf(d, s.cl, fmaf(d, s.ch, -zh)));
    k = pow_split(zh, zl, entry, th, rest) + cexp - exponent + 41 - 48;
    return live;
}

// a b < c, of numbers that are not negative.
__device__ __forceinline__ bool less(Pair a, Pair b, Pair c)
{
    const float p = a.hi * b.hi;
    const float e = fmaf(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi);
    return (p - c.hi) + (e - c.lo) < 0.0f;
}

__device__ __forceinline__ Pair pair_of(long long v) // to 48 bits
{
    const float hi = __ll2float_rn(v);
    return {hi, __ll2float_rn(v - __float2ll_rn(hi))};
}

// What a CTA shares.
struct RowShared {
    float top[kVerifyWarps];
    int best[kVerifyWarps];
    long long sum[kVerifyWarps];
    long long in_row[kMaxParts];   // this row's parts
    RowStat row;                   // this row, then the one that the sequence stops at
    long long target;
    int skip, last_chunk, last_row, draw_now, part, found, end;
};

__device__ __forceinline__ PartStat load_stat(const PartStat *st)
{
    const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(st));
    return {__uint_as_float(w.x), static_cast<int>(w.y),
            static_cast<long long>(static_cast<unsigned long long>(w.w) << 32 | w.z)};
}

// The row's parts put together, and the verdict on its draft; the whole CTA.
template <bool kBf16>
__device__ __forceinline__ void finish_row(const VerifyParams &p, int b, int j, int len, const Row<kBf16> &x, RowShared &sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = static_cast<long long>(b) * (p.L + 1) + j;
    const PartStat *const st = p.part + row * p.parts;
    const float T = temperature(p, b);
    const float2 entry = kPow32[lane];
    const long long d = static_cast<long long>(b) * p.L + j;
    const int t = j < len ? p.draft[d] : -1;
    const bool inside = t >= 0 && t < p.V;
    const float xt = inside ? x.at(t) : -INFINITY;
    const float qt = j >= len || !inside ? 0.0f : p.q == nullptr ? 1.0f : p.q[d * p.ldq + t];
    const float ut = j < len ? p.accept_u[d] : 0.0f;
    const PartStat first = static_cast<int>(threadIdx.x) < p.parts ? load_stat(st + threadIdx.x) : PartStat{-INFINITY, 0, 0};
    float top = first.top;
#pragma unroll 1
    for (int i = threadIdx.x + kVerifyThreads; i < p.parts; i += kVerifyThreads)
        top = max_nan(top, __ldcg(&st[i].top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        sh.top[warp] = top;
    __syncthreads();
    top = sh.top[0];
#pragma unroll
    for (int i = 1; i < kVerifyWarps; ++i)
        top = max_nan(top, sh.top[i]);
    RowStat r = {};
    r.top = top;
    r.position = j;
    if (!(top > -INFINITY && top < INFINITY) || !good_temperature(T)) {
        r.verdict = 2;
    } else if (T == 0.0f) {
        int best = 0x7fffffff;
#pragma unroll 1
        for (int i = threadIdx.x; i < p.parts; i += kVerifyThreads)
            if (__ldcg(&st[i].top) == top)
                best = min(best, static_cast<int>(__ldcg(&st[i].sum)));
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0)
            sh.best[warp] = best;
        __syncthreads();
        r.best = sh.best[0];
#pragma unroll
        for (int i = 1; i < kVerifyWarps; ++i)
            r.best = min(r.best, sh.best[i]);
        r.prob = t == r.best ? 1.0f : 0.0f;
        r.verdict = inside && ut * qt < r.prob ? 1 : 0;
    } else {
        const Scale s = make_scale(T);
        const float ref = reference(top, s), cut = cutoff(top, T);
        float zh, zl, th, rest;
        exponent_of(top, ref, s, zh, zl);
        r.exponent = pow_exponent(zh);
        long long sum = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < p.parts; i0 += kVerifyThreads) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            const PartStat v = i0 == 0 ? first : i < p.parts ? load_stat(st + i) : PartStat{-INFINITY, 0, 0};
            int k;
            const bool live = to_row(v.top, v.exponent, ref, cut, r.exponent, s, entry, th, rest, k);
            const long long g = live ? rescale(v.sum, th, rest, k) : 0;
            if (i < p.parts) {
                __stcg(p.in_row + row * p.parts + i, g);
                sh.in_row[i] = g;
                sum += g;
            }
        }
        sum = warp_sum(sum);
        if (lane == 0)
            sh.sum[warp] = sum;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVerifyWarps; ++i)
            r.total += sh.sum[i];
        r.sum = pair_of(r.total);
        if (j < len) {
            float hi, lo;
            weight(xt, top, ref, cut, r.exponent, s, entry, hi, lo);
            const Pair w = {hi * kRowUnits, lo * kRowUnits};
            const float uq = ut * qt;
            r.verdict = inside && less({uq, fmaf(ut, qt, -uq)}, r.sum, w) ? 1 : 0;
            r.prob = divide(fast_two_sum(w.hi, w.lo), r.sum).hi;
        }
    }
    if (threadIdx.x == 0) {
        p.row[row] = r;
        sh.row = r;
        if (r.verdict != 1)
            atomicMax(p.stopped + b, static_cast<unsigned>(64 - j));
    }
}

__device__ __forceinline__ float probability(float hi, float lo, Pair total)
{
    return divide(fast_two_sum(hi * kRowUnits, lo * kRowUnits), total).hi;
}

// floor(u * total), at most total - 1; 0 where u is NaN or not positive.
__device__ __forceinline__ long long target_of(float u, long long total)
{
    if (!(u > 0.0f))
        return 0;
    if (u >= 1.0f)
        return total - 1;
    const uint32_t b = __float_as_uint(u);
    const unsigned long long m = (b >> 23) == 0u ? b : (b & 0x7FFFFFu) | 0x800000u; // u = m 2^-shift
    const int shift = 150 - static_cast<int>((b >> 23) == 0u ? 1u : b >> 23);         // 24 or more
    const unsigned long long t = static_cast<unsigned long long>(total);
    const unsigned long long lo = t * m, hi = __umul64hi(t, m);
    const unsigned long long v = shift < 64 ? lo >> shift | hi << (64 - shift) : shift < 128 ? hi >> (shift - 64) : 0ull;
    return static_cast<long long>(v);
}

// Position of the target weight u * (sum of `sum(i)`, i < n) and what is left of it
// there, to sh.part and sh.target; -1 where the sum is not positive.  The whole CTA
// calls it, a thread for n / 256 positions in a row.
template <class Sum> __device__ __forceinline__ void find_target(int n, float u, Sum sum, RowShared &sh)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int each = (n + kVerifyThreads - 1) / kVerifyThreads;
    const int first = static_cast<int>(threadIdx.x) * each;
    long long mine = 0;
#pragma unroll 1
    for (int i = first; i < first + each && i < n; i += 4) {
        long long g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            g[k] = i + k < first + each && i + k < n ? sum(i + k) : 0;
        mine += (g[0] + g[1]) + (g[2] + g[3]);
    }
    long long upto = warp_scan(mine);
    if (lane == 31)
        sh.sum[warp] = upto;
    if (threadIdx.x == 0)
        sh.part = -1;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < kVerifyWarps; ++i) {
        upto += i < warp ? sh.sum[i] : 0;
        total += sh.sum[i];
    }
    if (total > 0) {
        const long long target = target_of(u, total);
        long long at = upto - mine;
        if (at <= target && target < upto) {
#pragma unroll 1
            for (int i = first; i < first + each && i < n; i += 4) {
                long long g[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    g[k] = i + k < first + each && i + k < n ? sum(i + k) : 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (at <= target && target < at + g[k]) {
                        sh.part = i + k;
                        sh.target = target - at;
                    }
                    at += g[k];
                }
            }
        }
    }
    __syncthreads();
}

// A row's weights in row units.
template <bool kBf16> struct Weights {
    Row<kBf16> x;
    Scale s;
    float top, ref, cut;
    int exponent;
    float2 entry;

    __device__ __forceinline__ Weights(const VerifyParams &p, long long row, const RowStat &r, float T)
        : x(p, row), s(make_scale(T)), top(r.top), ref(reference(r.top, s)), cut(cutoff(r.top, T)), exponent(r.exponent),
          entry(kPow32[threadIdx.x & 31])
    {
    }
    __device__ __forceinline__ void pair(float v, float &hi, float &lo) const // whole warps
    {
        weight(v, top, ref, cut, exponent, s, entry, hi, lo);
    }
};

// Where the cumulative sum of a CTA's weights passes `target`: g, kN a thread, of the
// logits from i0 on, in order.  Where rounding leaves none (sums were taken in finer
// units), the last one with a weight, of those with one unit or more if there are
// any.  The thread that has it writes it and its probability (weights hi + lo, whose
// total is r.sum).  All threads call it; false where no logit has a weight.
template <int kN>
__device__ __forceinline__ bool look(const VerifyParams &p, long long to, const RowStat &r, const long long (&g)[kN],
                                     const float (&hi)[kN], const float (&lo)[kN], int i0, long long target, RowShared &sh)
{
    constexpr int kWhole = 2 * kVerifyMaxVocab; // above every index
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.found = 0x7fffffff;
        sh.end = -1;
    }
    long long mine = 0;
    int last = -1;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        mine += g[e];
        if (g[e] > 0)
            last = i0 + e + kWhole;
        else if (hi[e] > 0.0f && last < kWhole)
            last = i0 + e;
    }
    long long upto = warp_scan(mine);
    if (lane == 31)
        sh.sum[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVerifyWarps; ++i)
        upto += i < warp ? sh.sum[i] : 0;
    if (upto - mine <= target && target < upto) {
        long long at = upto;
#pragma unroll
        for (int e = kN - 1; e >= 0; --e) { // from behind: the first that passes is written last
            if (at > target)
                sh.found = i0 + e;
            at -= g[e];
        }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last >= 0)
        atomicMax(&sh.end, last);
    __syncthreads();
    const int token = sh.found != 0x7fffffff ? sh.found : sh.end >= kWhole ? sh.end - kWhole : sh.end;
    if (token >= i0 && token < i0 + kN) {
        float h = hi[0], l = lo[0];
#pragma unroll
        for (int e = 1; e < kN; ++e) {
            h = token == i0 + e ? hi[e] : h;
            l = token == i0 + e ? lo[e] : l;
        }
        p.tokens[to] = token;
        p.probs[to] = probability(h, l, r.sum);
    }
    return token >= 0;
}

// Draws the token of row `r` (of sequence b, at r.position) from its own weights,
// without that of logit `except` where it is in the row.  The whole CTA calls it;
// `own`: the parts' sums lie in sh.in_row.
template <bool kBf16>
__device__ __forceinline__ void draw(const VerifyParams &p, int b, const RowStat &r, float T, float u, int except, bool own,
                                     RowShared &sh)
{
    const long long row = static_cast<long long>(b) * (p.L + 1) + r.position;
    const Weights<kBf16> w(p, row, r, T);
    const long long *const in_row = p.in_row + row * p.parts;
    auto sum = [&](int i) { return own ? sh.in_row[i] : __ldcg(in_row + i); };
    int without = except >= 0 && except < p.V ? except : -1, home = -1;
    long long less_by = 0;
    if (without >= 0) {
        float h, l;
        w.pair(w.x.at(without), h, l);
        less_by = row_units(h, l);
        home = (without + w.x.lead) / kPart;
    }
#pragma unroll 1
    for (;;) { // the second time from everything, where nothing is left beside it
        find_target(p.parts, u, [&](int i) {
            const long long g = sum(i);
            return i != home ? g : g > less_by ? g - less_by : 0;
        }, sh);
        const int part = sh.part;
        if (part >= 0 || without < 0) {
            constexpr int kN = kPart / kVerifyThreads; // logits of a thread
            const long long target = sh.target;
            const int i0 = (part < 0 ? 0 : part) * kPart - w.x.lead + static_cast<int>(threadIdx.x) * kN; // (a row's total is positive)
            float v[kN], hi[kN], lo[kN];
            long long g[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e)
                v[e] = i0 + e >= 0 && i0 + e < p.V && i0 + e != without ? w.x.at(i0 + e) : -INFINITY;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                w.pair(v[e], hi[e], lo[e]);
                g[e] = row_units(hi[e], lo[e]);
            }
            if (look(p, row, r, g, hi, lo, i0, target, sh) || without < 0)
                break;
        }
        __syncthreads();
        without = home = -1;
    }
}

// A CTA per (position, sequence, chunk), in that order.
template <bool kBf16>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas) verify_rows_kernel(const VerifyParams p)
{
    using R = Row<kBf16>;
    __shared__ RowShared sh;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_VERIFY_ROWS, 1ull);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float2 entry = kPow32[lane];
    grid_launch_dependents();
    grid_dependency_wait();
    const int c = static_cast<int>(blockIdx.x % p.chunks);
    const int rank = static_cast<int>(blockIdx.x / p.chunks);
    const int j = rank / p.B, b = rank - j * p.B;
    const int len = drafted(p, b);
    if (j > len)
        return;
    bool skip = false;
    if (blockIdx.x >= p.first_wave && j > 0) {
        if (threadIdx.x == 0)
            sh.skip = behind_a_stop(p, b, j) ? 1 : 0;
        __syncthreads();
        skip = sh.skip != 0;
    }
    const long long row = static_cast<long long>(b) * (p.L + 1) + j;
    const R x(p, row);
    const float T = temperature(p, b);
    if (!skip) {
        const bool drawing = good_temperature(T) && T != 0.0f;
        const Scale sc = make_scale(drawing ? T : 1.0f);
        int part = (c * kVerifyWarps + warp) * p.parts_each;
        const int end = min(part + p.parts_each, p.parts);
#pragma unroll 1
        for (; part < end; ++part) {
            const int w0 = part * (kPart / R::kPer) + lane;
            uint4 raw[R::kWords];
            const int first = x.index(part * (kPart / R::kPer));
            if (first >= 0 && first + kPart <= p.V) {
#pragma unroll
                for (int s = 0; s < R::kWords; ++s)
                    raw[s] = x.whole(w0 + s * 32);
            } else {
#pragma unroll
                for (int s = 0; s < R::kWords; ++s)
                    raw[s] = x.edge(w0 + s * 32);
            }
            float top = R::largest(raw[0]);
#pragma unroll
            for (int s = 1; s < R::kWords; ++s)
                top = max_nan(top, R::largest(raw[s]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            PartStat out = {top, 0, 0};
            if (!(top > -INFINITY && top < INFINITY)) {
                // no sum
            } else if (!drawing) {
                int best = 0x7fffffff;
#pragma unroll
                for (int s = R::kWords - 1; s >= 0; --s)
#pragma unroll
                    for (int e = R::kPer - 1; e >= 0; --e)
                        if (R::value(raw[s], e) == top)
                            best = x.index(w0 + s * 32) + e;
                out.sum = __reduce_min_sync(0xffffffffu, best);
            } else {
                const float ref = reference(top, sc), cut = cutoff(top, T);
                float zh, zl;
                exponent_of(top, ref, sc, zh, zl);
                out.exponent = pow_exponent(zh);
                long long sum;
                if (ref == 0.0f) {
                    WeightSum sums(cut, out.exponent, sc, entry);
#pragma unroll
                    for (int s = 0; s < R::kWords; ++s)
#pragma unroll
                        for (int e = 0; e < R::kPer; e += 2)
                            sums.add(R::value(raw[s], e), R::value(raw[s], e + 1));
                    sum = sums.units();
                } else {
                    sum = 0;
#pragma unroll 1
                    for (int i = 0; i < kPart / 32; ++i) {
                        const int at = first + i * 32 + lane;
                        float hi, lo;
                        weight(at >= 0 && at < p.V ? x.at(at) : -INFINITY, top, ref, cut, out.exponent, sc, entry, hi, lo);
                        sum += fixed(hi, lo, kPartUnits);
                    }
                }
                out.sum = warp_sum(sum);
            }
            if (lane == 0) {
                const unsigned long long v = static_cast<unsigned long long>(out.sum);
                __stcg(reinterpret_cast<uint4 *>(p.part + row * p.parts + part),
                       make_uint4(__float_as_uint(out.top), static_cast<uint32_t>(out.exponent), static_cast<uint32_t>(v),
                                  static_cast<uint32_t>(v >> 32)));
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sh.last_chunk = 1;
        if (p.chunks > 1) {
            sh.last_chunk = atomic_add_acq_rel_gpu(p.row_done + row, 1u) == static_cast<unsigned>(p.chunks - 1);
            if (sh.last_chunk != 0)
                p.row_done[row] = 0u;
        }
        // where a part was left out, this sees why
        sh.skip = sh.last_chunk != 0 && j > 0 && behind_a_stop(p, b, j) ? 1 : 0;
    }
    __syncthreads();
    // (the arrival of thread 0 acquires the others' writes, and the barrier passes that on)
    if (sh.last_chunk == 0)
        return;
    const bool finish = sh.skip == 0;
    const float u = p.sample_u[b];
    if (finish)
        finish_row<kBf16>(p, b, j, len, x, sh);
    __syncthreads();
    if (len > 0) {
        if (threadIdx.x == 0) {
            sh.last_row = atomic_add_acq_rel_gpu(p.seq_done + b, 1u) == static_cast<unsigned>(len);
            if (sh.last_row != 0)
                p.seq_done[b] = 0u;
        }
        __syncthreads();
        if (sh.last_row == 0)
            return;
    }
    // the sequence's last row: where it stops, and its token
    const long long row0 = static_cast<long long>(b) * (p.L + 1);
    if (warp == 0) {
        // the first position that was not accepted (position len never is); rows behind it may be old
        const int v = lane > len ? 0 : finish && lane == j ? sh.row.verdict : __ldcg(&p.row[row0 + lane].verdict);
        const int n = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, v != 1))) - 1;
        if (lane < n) {
            p.tokens[row0 + lane] = p.draft[static_cast<long long>(b) * p.L + lane];
            p.probs[row0 + lane] = finish && lane == j ? sh.row.prob : __ldcg(&p.row[row0 + lane].prob);
        } else if (lane > n && lane <= p.L) {
            p.tokens[row0 + lane] = -1;
            p.probs[row0 + lane] = 0.0f;
        }
        __syncwarp();
        if (lane == 0) {
            p.accepted[b] = n;
            p.stopped[b] = 0u;
            if (!(finish && n == j)) {
                const uint4 *const from = reinterpret_cast<const uint4 *>(p.row + row0 + n);
                uint4 *const to = reinterpret_cast<uint4 *>(&sh.row);
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    to[i] = __ldcg(from + i);
            }
            const bool done = sh.row.verdict == 2 || T == 0.0f; // no distribution, or no choice
            const bool later = !done && p.q != nullptr && n < len;
            if (done) {
                p.tokens[row0 + n] = sh.row.verdict == 2 ? -1 : sh.row.best;
                p.probs[row0 + n] = sh.row.verdict == 2 ? NAN : 1.0f;
            }
            if (p.q != nullptr) {
                RowStat s = sh.row;
                s.position = later ? n : -1;
                p.stop[b] = s;
            }
            sh.draw_now = !done && !later;
        }
    }
    __syncthreads();
    if (sh.draw_now == 0)
        return;
    const RowStat r = sh.row;
    const int except = r.position < len ? p.draft[static_cast<long long>(b) * p.L + r.position] : -1;
    draw<kBf16>(p, b, r, T, u, except, finish && r.position == j, sh);
}

// A CTA per (sequence, runs_each times kBit logits a warp): the weights max(p - q, 0)
// where a draft was rejected.
template <bool kBf16> __global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas) verify_residual_kernel(const VerifyParams p)
{
    using R = Row<kBf16>;
    constexpr int kN = kBit / 32; // logits of a lane, one after the other
    __shared__ RowShared sh;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        atomicAdd(p.runs + FP8BS_RUNS_VERIFY_RESIDUAL, 1ull);
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = static_cast<int>(blockIdx.x / p.bit_ctas), c = static_cast<int>(blockIdx.x % p.bit_ctas);
    const float T = temperature(p, b), u = p.sample_u[b];
    const uint4 *const from = reinterpret_cast<const uint4 *>(p.stop + b);
    RowStat r;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        reinterpret_cast<uint4 *>(&r)[i] = __ldcg(from + i);
    if (r.position < 0)
        return;
    const Weights<kBf16> w(p, static_cast<long long>(b) * (p.L + 1) + r.position, r, T);
    const float *const q = p.q + (static_cast<long long>(b) * p.L + r.position) * p.ldq;
    const Pair W = {r.sum.hi * (1.0f / kRowUnits), r.sum.lo * (1.0f / kRowUnits)};
    auto residual = [&](float hi, float lo, float qi) {
        const float bh = qi * W.hi;
        return difference_units(hi, lo, bh, fmaf(qi, W.lo, fmaf(qi, W.hi, -bh)));
    };
    long long *const sums = p.residual + static_cast<long long>(b) * p.bits;
#pragma unroll 1
    for (int n = 0; n < p.runs_each; ++n) {
        const int bit = (c * p.runs_each + n) * kVerifyWarps + warp;
        if (bit >= p.bits)
            break;
        const int word = (bit * kBit + lane * kN) / R::kPer;
        const int i0 = w.x.index(word);
        uint4 v[kN / R::kPer];
        float qi[kN];
#pragma unroll
        for (int s = 0; s < kN / R::kPer; ++s)
            v[s] = w.x.load(word + s);
        if (i0 >= 0 && i0 + kN <= p.V && (reinterpret_cast<uintptr_t>(q + i0) & 15) == 0) {
#pragma unroll
            for (int e = 0; e < kN; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(q + i0 + e);
                qi[e] = f.x;
                qi[e + 1] = f.y;
                qi[e + 2] = f.z;
                qi[e + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e)
                qi[e] = i0 + e >= 0 && i0 + e < p.V ? q[i0 + e] : 0.0f;
        }
        long long sum = 0;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            float hi, lo;
            w.pair(R::value(v[e / R::kPer], e % R::kPer), hi, lo);
            sum += residual(hi, lo, qi[e]);
        }
        sum = warp_sum(sum);
        if (lane == 0)
            __stcg(sums + bit, sum);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sh.last_chunk = atomic_add_acq_rel_gpu(p.seq_done + b, 1u) == static_cast<unsigned>(p.bit_ctas - 1);
        if (sh.last_chunk != 0)
            p.seq_done[b] = 0u;
    }
    __syncthreads();
    if (sh.last_chunk == 0)
        return;
    find_target(p.bits, u, [&](int i) { return __ldcg(sums + i); }, sh);
    const int bit = sh.part;
    const long long target = sh.target;
    if (bit < 0) { // p nowhere above q: from p
        __syncthreads();
        draw<kBf16>(p, b, r, T, u, -1, false, sh);
        return;
    }
    static_assert(kBit == kVerifyThreads, "a logit a thread");
    const int i = bit * kBit - w.x.lead + static_cast<int>(threadIdx.x);
    const bool inside = i >= 0 && i < p.V;
    float hi[1], lo[1];
    w.pair(inside ? w.x.at(i) : -INFINITY, hi[0], lo[0]);
    const long long g[1] = {residual(hi[0], lo[0], inside ? q[i] : 0.0f)};
    look(p, static_cast<long long>(b) * (p.L + 1) + r.position, r, g, hi, lo, i, target, sh);
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct VerifyWorkspace {
    size_t counters_bytes, part_off, in_row_off, row_off, stop_off, residual_off, total;
    int parts, bits;
};

VerifyWorkspace verify_workspace(int B, int L, int V)
{
    auto up256 = [](size_t b) { return (b + 255) / 256 * 256; };
    const size_t rows = static_cast<size_t>(B) * (L + 1);
    VerifyWorkspace w;
    w.parts = (V + 7 + kPart - 1) / kPart; // a row may start up to seven logits into its first word
    w.bits = (V + 7 + kBit - 1) / kBit;
    w.counters_bytes = (rows + 2 * static_cast<size_t>(B)) * 4;
    w.part_off = kCountersOff + counters_region(w.counters_bytes);
    w.in_row_off = w.part_off + up256(rows * w.parts * sizeof(PartStat));
    w.row_off = w.in_row_off + up256(rows * w.parts * 8);
    w.stop_off = w.row_off + up256(rows * sizeof(RowStat));
    w.residual_off = w.stop_off + up256(static_cast<size_t>(B) * sizeof(RowStat));
    w.total = w.residual_off + up256(static_cast<size_t>(B) * w.bits * 8);
    return w;
}
static_assert((kVerifyMaxRows + 2 * kVerifyMaxRows) * 4 <= kCountersRegion, "every size's counters lie in the shared region");
static_assert(kMaxParts * kPart >= kVerifyMaxVocab + 7, "parts of a row");
static_assert(sizeof(PartStat) == 16 && sizeof(RowStat) == 48, "workspace layout");

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
    // parts of a warp: more than one where the GPU is filled three times over all the same (512 rows of 248,320 in
    // 115 us, 124 with one; two, for 64 rows, 31.7 us instead of 30.3; four, for 5 rows, 17.4 instead of 14.5)
    const long long rows = static_cast<long long>(B) * (L + 1);
    p.parts = w.parts;
    p.parts_each = 1;
    while (p.parts_each < kMostParts && rows * w.parts >= 2ll * p.parts_each * 3 * kVerifyWarps * kVerifyCtas * dev.sms)
        p.parts_each *= 2;
    // the same for the residual, where a CTA's first loads and its arrival are most of its time (512 rows: 130 us with one
    // run each, 117 with two, 115 with four; 64 rows 30.3, 30.4, 32.9; 5 rows 14.5, 14.9, 16.3)
    p.bits = w.bits;
    p.runs_each = 1;
    const int runs = (w.bits + kVerifyWarps - 1) / kVerifyWarps;
    while (p.runs_each < kMostParts && static_cast<long long>(B) * runs >= 2ll * p.runs_each * kVerifyCtas * dev.sms)
        p.runs_each *= 2;
    p.bit_ctas = (runs + p.runs_each - 1) / p.runs_each;
    p.chunks = (w.parts + p.parts_each * kVerifyWarps - 1) / (p.parts_each * kVerifyWarps);
    p.first_wave = static_cast<unsigned>(dev.sms * kVerifyCtas);
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
    p.part = reinterpret_cast<PartStat *>(ws + w.part_off);
    p.in_row = reinterpret_cast<long long *>(ws + w.in_row_off);
    p.row = reinterpret_cast<RowStat *>(ws + w.row_off);
    p.stop = reinterpret_cast<RowStat *>(ws + w.stop_off);
    p.residual = reinterpret_cast<long long *>(ws + w.residual_off);
    p.runs = dev.runs;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kVerifyThreads, 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(rows * p.chunks), 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = (flags & FP8BS_FLAG_OVERLAP_PREV) ? 1 : 0;
    const bool bf = logits_type == FP8BS_BF16;
    st = launch_status(cudaLaunchKernelEx(&cfg, bf ? verify_rows_kernel<true> : verify_rows_kernel<false>, p));
    if (st != FP8BS_OK || !draft_probs)
        return st;
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(B) * p.bit_ctas), 1, 1);
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, bf ? verify_residual_kernel<true> : verify_residual_kernel<false>, p));
}

} // extern "C"
