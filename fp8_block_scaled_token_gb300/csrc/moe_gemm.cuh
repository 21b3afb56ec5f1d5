// moe_gemm.cuh -- the two grouped products of an expert layer for up to 64
// tokens, E4M3 with 128x128 weight-block and 1x128 activation scales.
//
//   up:   g, u = W13[e] a   (gate rows 0..I-1, up rows I..2I-1 of expert e),
//         h = g / (1 + exp(-g)) * u, one fp32 scale per token and 128 of I,
//         E4M3 codes
//   down: y = sum over chosen experts of w * W2[e] h
//
// A few tokens choose from many experts, so nearly every expert product has
// one to a few rows and the layer's time is the active experts' weight bytes.
// Both products therefore multiply every active expert's weights by ALL the
// tokens (16, 32 or 64 columns of the MMA's N, which cost no memory traffic
// worth counting): no gather, no padding per expert, every weight byte is read
// once, and a token that did not choose an expert has weight 0 there.
//   up   is one product with N concatenated over the active experts:
//        unit = (active expert a, 128 of I, 128 of H), a gate tile and an up
//        tile of weights a unit;
//   down is one product with K concatenated over the active experts:
//        unit = (128 of H, active expert a, 128 of I); the experts' sum is
//        the K sum, with the token's weight folded into the scale of its
//        intermediate, so nothing is combined afterwards.
// Units are dealt to the CTAs in equal contiguous ranges (stream-K, plan.cuh)
// over the number of active experts, which the kernels read on the device.  A
// tile shared by CTAs is summed in contributor order by the last one to
// arrive: results repeat bit for bit, and no CTA waits for another.
//
// Measured (8 tokens, 64 experts, top 4, H = 5,120, I = 1,280): the up product
// reads its 341 MB at 7.0 TB/s between its first and last MMA, the down
// product 171 MB at 6.4; before, between and after them lie the routing (9 us
// until the first weights can be named), 4 us and 3 us.  64 tokens and 64
// experts of (5,120, 1,408): the layer 238-240 us, 0.85 of the measured copy
// bandwidth; there one CTA fills an SM and the next product cannot start
// early.  Row-major weights, whose tiles are 128 runs of 128 bytes, take 91.4 us
// instead of 90.1 (8 tokens) and 244.6 instead of 238.2 (64).
//
// Warp 0 streams the tiles (TMA), warp 1 issues tcgen05.mma, the others
// promote each unit's accumulators by their scales into fp32 registers, as in
// gemm_kernel.cuh.  Every wait is bounded.
#pragma once

#include <cuda_bf16.h>

#include "fp8bs_testing.h"
#include "moe.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace fp8bs {

enum MoePhase : int { kMoeUp = 0, kMoeDown = 1 };

struct MoeGemmParams {
    int M, H, I, E;
    int stages;
    const unsigned *masks; // [groups][kMoeMaxExperts / 32] experts that each group of tokens chose
    unsigned *chosen;      // 1 while the masks are known to be complete: up sets it, down clears it
    int groups;
    const float *wtok;     // [E][NPAD]
    const float *ws;       // weight block scales: s13 [E][2I/128][H/128] or s2 [E][H/128][I/128]
    const float *xs;       // up: activation scales [H/128][M]
    uint8_t *hq;           // up: codes out, [active][NPAD][I]
    float *hs;             // scales times weights, [active][I/128][NPAD]: up writes, down reads
    uint16_t *y;           // down: bf16 [M][H]
    unsigned *status, *counters;
    float *slots;          // [2 * grid (up: 3 * grid)][tiles a unit][NPAD * 128]
    int w_tiled;
    int max_active;
    int test_skip_unit;
    unsigned long long timeout_ns;
    unsigned long long *runs;
};

template <int NPAD, int PHASE> struct MoeCfg {
    static_assert(NPAD == 16 || NPAD == 32 || NPAD == 64, "token tile");
    static constexpr int kTiles = PHASE == kMoeUp ? 2 : 1;  // weight tiles a unit
    static constexpr int kWBytes = 128 * 128;
    static constexpr int kBBytes = NPAD * 128;
    static constexpr int kStageBytes = kTiles * kWBytes + kBBytes;
    static constexpr int kMaxStages = 12;
    static constexpr int kAcc = PHASE == kMoeDown && NPAD == 16 ? 8 : 4;
    static constexpr int kAccCols = kTiles * NPAD;
    static constexpr int kTmemCols = kAcc * kAccCols; // 128 (16 tokens), 256 / 128 (32), 512 / 256 (64)
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols >= 32 && kTmemCols <= 512, "tensor memory");
    // Up to 32 tokens two CTAs per SM, so that the next kernel's CTA streams
    // its first weights while this one finishes (32 tokens, 128 experts of
    // (2,048, 768), top 8: 103.6 us, one CTA of twice the ring 106.3; 20 tokens,
    // 16 of (512, 256), top 2: 17.0 and 17.9); at 64 two groups of epilogue
    // warps, whose registers leave no room for a second CTA.
    static constexpr int kMinBlocks = NPAD <= 32 ? 2 : 1;
    static constexpr int kColGroups = NPAD == 64 ? 2 : 1;
    static constexpr int kCols = NPAD / kColGroups;
    static_assert(kCols <= 32, "a lane holds one token's scale");
    static constexpr int kEpiWarps = 4 * kColGroups;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kMaxRegs = NPAD == 16 ? 160 : 168;
    static constexpr int kHeader = 3072; // barriers and flags, then [1024, 3072) the active experts
    static constexpr int kProdFloats = kEpiWarps * 2 * kTiles * kCols; // per warp, by unit parity
    static constexpr uint32_t kIdesc = idesc_e4m3_f32(128, NPAD);
    static_assert((2 * kMaxStages + 2 * kAcc + 1) * 8 + 16 <= 1024, "header layout");
    static constexpr int smem_bytes(int stages)
    {
        return 1024 + kHeader + stages * kStageBytes + kProdFloats * 4;
    }
};

template <int NPAD, int PHASE>
__global__ void __maxnreg__((MoeCfg<NPAD, PHASE>::kMaxRegs))
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_b,
                    const MoeGemmParams p)
{
    using C = MoeCfg<NPAD, PHASE>;
    constexpr bool kUp = PHASE == kMoeUp;
    constexpr int kTriggerLead = 6; // as in gemm_kernel.cuh
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + C::kMaxStages;
    uint64_t *tfull = empty + C::kMaxStages;
    uint64_t *tempty = tfull + C::kAcc;
    uint64_t *mma_done = tempty + C::kAcc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *last_flag = abort_flag + 1;
    volatile int *active_count = last_flag + 1;
    int *act = reinterpret_cast<int *>(smem + 1024);            // [kMoeMaxExperts]
    const int S = p.stages;
    uint8_t *ring = smem + C::kHeader;
    float *prod = reinterpret_cast<float *>(ring + S * C::kStageBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    if (threadIdx.x == 0) {
        if (cta == 0)
            atomicAdd(p.runs + FP8BS_RUNS_MOE_GEMM(PHASE, NPAD), 1ull);
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::kAcc; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], C::kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        *last_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_b);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    // The list of active experts, ascending, from the masks that the routing
    // kernel left: the up product's predecessor, which it waits for here.  The
    // down product, which is to stream its first weights while the up product
    // finishes, takes them over from the up product's first CTA: that one has
    // waited, and publishes so before it lets this grid start (release here,
    // acquire there).  A CTA that does not find the word set waits for the whole
    // up product: the last of the down product's CTAs may, after the first has
    // finished and cleared it.
    if (kUp) {
        grid_dependency_wait();
        if (cta == 0 && threadIdx.x == 0)
            store_release_gpu(p.chosen, 1u);
    }
    if (warp == 2) {
        if (!kUp && !__all_sync(0xffffffffu, load_acquire_gpu(p.chosen) != 0u))
            grid_dependency_wait();
        unsigned word = 0; // lane w: experts 32 w .. 32 w + 31
        if (lane < (p.E + 31) / 32) {
#pragma unroll
            for (int g = 0; g < kMoeMaxTokens / kMoeTokenGroup; ++g)
                word |= g < p.groups ? __ldcg(p.masks + g * (kMoeMaxExperts / 32) + lane) : 0u;
        }
        int before = 0; // active experts of the words so far
#pragma unroll 1
        for (int w = 0; 32 * w < p.E; ++w) {
            const unsigned bits = __shfl_sync(0xffffffffu, word, w);
            const int at = before + __popc(bits & ((1u << lane) - 1u));
            if ((bits >> lane & 1u) && at < p.max_active)
                act[at] = 32 * w + lane;
            before += __popc(bits);
        }
        if (lane == 0)
            *active_count = before < p.max_active ? before : p.max_active;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const int A = *active_count;

    // K blocks of one expert, tiles of 128 output rows (up: of one expert's I)
    const int kg1 = kUp ? p.H / 128 : p.I / 128;
    const int nj = kUp ? p.I / 128 : p.H / 128;
    const int kg = kUp ? kg1 : A * kg1;           // units per output tile
    const int tiles = kUp ? A * nj : nj;
    const long long units = static_cast<long long>(tiles) * kg;
    // A tile's exchange takes time in proportion to its contributors n, its
    // product kg / n: small layers use sqrt(kg) contributors a tile, not every
    // SM.  Down, tokens x experts x (H, I), with the cap and without: 20 x 16 x
    // (512, 256) 18.3 and 23.5 us, 50 x 24 x (896, 640) 32.5 and 35.0, one token
    // and 2 experts of (2,048, 1,408) 17.8 and 18.8; large layers have fewer
    // than that anyway.  Up: 40 x 8 x (1,280, 384) 20.8 and 22.7, but one token
    // and 2 experts of (512, 256) 13.7 and 13.5: from 32 columns only.
    const int contributors = static_cast<int>(ceilf(sqrtf(static_cast<float>(kg))));
    const int most = (kUp && NPAD == 16) || tiles * contributors > static_cast<int>(gridDim.x)
                         ? static_cast<int>(gridDim.x) : tiles * contributors;
    const int ctas = plan_ctas(units, most); // CTAs past the units have none
    const bool has = cta < ctas;
    // plan.cuh's functions, in 32 bits where they fit (64-bit divisions on the
    // way to the first load are most of a microsecond)
    const bool narrow = units <= 0xffffffffll / static_cast<long long>(gridDim.x + 1);
    const unsigned units32 = static_cast<unsigned>(units), ctas32 = static_cast<unsigned>(ctas);
    auto range_begin = [&](int c) {
        return narrow ? static_cast<long long>(units32 * static_cast<unsigned>(c) / ctas32) : plan_begin(units, ctas, c);
    };
    auto owner = [&](long long u) {
        return narrow ? static_cast<int>(((static_cast<unsigned>(u) + 1u) * ctas32 + units32 - 1u) / units32) - 1
                      : plan_owner(units, ctas, u);
    };
    const long long u0 = has ? range_begin(cta) : 0;
    const int nunits = has ? static_cast<int>(range_begin(cta + 1) - u0) : 0;
    const int tile0 = !has ? 0 : narrow ? static_cast<int>(static_cast<unsigned>(u0) / static_cast<unsigned>(kg))
                                        : static_cast<int>(u0 / kg);
    const int ku0 = has ? static_cast<int>(u0 - static_cast<long long>(tile0) * kg) : 0; // unit within the tile

    // A unit's place: output tile, active expert, K block of that expert.
    struct Unit {
        int ku, a, j, kb; // unit within the tile, active expert, tile of 128 rows within its matrix, K block
    };
    auto first_unit = [&]() {
        Unit u;
        u.ku = ku0;
        u.a = kUp ? tile0 / nj : ku0 / kg1;
        u.j = kUp ? tile0 % nj : tile0;
        u.kb = kUp ? ku0 : ku0 % kg1;
        return u;
    };
    auto step = [&](Unit &u) {
        if (kUp) {
            u.kb = ++u.ku;
            if (u.ku == kg) {
                u.ku = u.kb = 0;
                if (++u.j == nj) {
                    u.j = 0;
                    ++u.a;
                }
            }
        } else {
            ++u.ku;
            if (++u.kb == kg1) {
                u.kb = 0;
                ++u.a;
            }
            if (u.ku == kg) {
                u.ku = u.a = 0;
                ++u.j;
            }
        }
    };
    // Weight tile of a unit (its t-th), counted in 128-row tiles from the start of the weights.
    auto weight_tile = [&](const Unit &u, int t) {
        const long long e = act[u.a];
        return kUp ? e * 2 * nj + t * nj + u.j : e * nj + u.j;
    };
    auto unit_ok = [&](const Unit &u) {
        return FP8BS_CHECK(u.a >= 0 && u.a < A && u.j >= 0 && u.j < nj && u.kb >= 0 && u.kb < kg1 && act[u.a] >= 0 &&
                           act[u.a] < p.E);
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint64_t pol_w = l2_policy_evict_first();
            const uint64_t pol_b = l2_policy_evict_last();
            uint32_t armed_mask = 0, armed_parity = 0;
            auto weight_x = [&](const Unit &u) { return p.w_tiled ? 0 : u.kb * 128; };
            auto weight_y = [&](const Unit &u, int t) {
                const long long wt = weight_tile(u, t);
                return static_cast<int>(p.w_tiled ? (wt * kg1 + u.kb) * 128 : wt * 128);
            };
            auto load_w = [&](int s, const Unit &u) {
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t)
                    tma_load_2d(ring + s * C::kStageBytes + t * C::kWBytes, &tm_w, &full[s], weight_x(u),
                                weight_y(u, t), pol_w);
            };
            auto load_b = [&](int s, const Unit &u) {
                tma_load_2d(ring + s * C::kStageBytes + C::kTiles * C::kWBytes, &tm_b, &full[s], u.kb * 128,
                            kUp ? 0 : u.a * NPAD, pol_b);
            };
            Unit u = first_unit();
            const int pre = nunits < S ? nunits : S;
            for (int i = 0; i < pre; ++i, step(u)) {
                if (i == p.test_skip_unit || !unit_ok(u))
                    continue;
                mbar_arrive_expect_tx(&full[i], C::kStageBytes);
                armed_mask |= 1u << i;
                load_w(i, u);
            }
            if (!kUp)
                grid_dependency_wait(); // the intermediate
            Unit ub = first_unit();
            for (int i = 0; i < pre; ++i, step(ub))
                if (armed_mask & (1u << i))
                    load_b(i, ub);
            int s = pre % S;
            uint32_t ph = static_cast<uint32_t>(pre / S) & 1u;
            bool triggered = false;
            for (int i = pre; i < nunits; ++i) {
                if (!triggered && i >= nunits - kTriggerLead) {
                    grid_launch_dependents();
                    triggered = true;
                }
                if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, kErrTimeoutProducer, p.timeout_ns))
                    break;
                if (i != p.test_skip_unit && unit_ok(u)) {
                    mbar_arrive_expect_tx(&full[s], C::kStageBytes);
                    armed_mask |= 1u << s;
                    armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
                    load_w(s, u);
                    load_b(s, u);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
                step(u);
            }
            if (!triggered)
                grid_launch_dependents();
            // Nothing may still be landing in shared memory when the CTA exits.
            for (int i = 0; i < S; ++i) {
                if (!(armed_mask & (1u << i)))
                    continue;
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_test(&full[i], (armed_parity >> i) & 1u)) {
                    if (globaltimer_ns() - t0 > p.timeout_ns) {
                        atomicOr(p.status, kErrTimeoutDrain);
                        break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // (the whole warp runs the loop and one lane issues, as the 4-bit
        // product's: the operands' values are uniform, and the next stage's
        // barrier is looked at before this one's MMAs are issued)
        const bool leader = elect_one();
        int acc = 0, s = 0;
        uint32_t acc_ph = 0, ph = 0;
        bool ready = false;
        for (int i = 0; i < nunits; ++i) {
            bool ok = mbar_wait(&tempty[acc], acc_ph ^ 1u, abort_flag, p.status, kErrTimeoutMma, p.timeout_ns);
            if (!ready)
                ok = ok && mbar_wait(&full[s], ph, abort_flag, p.status, kErrTimeoutMma, p.timeout_ns);
            if (!__all_sync(0xffffffffu, ok))
                break;
            tc_fence_after_sync();
            const int s1 = s + 1 == S ? 0 : s + 1;
            const uint32_t ph1 = s + 1 == S ? ph ^ 1u : ph;
            ready = __all_sync(0xffffffffu, i + 1 < nunits && mbar_peek(&full[s1], ph1));
            if (leader) {
                const uint32_t stage = smem_u32(ring) + static_cast<uint32_t>(s * C::kStageBytes);
                const uint64_t b_desc = sw128_kmajor_desc(stage + C::kTiles * C::kWBytes);
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t) {
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::kAccCols + t * NPAD);
                    const uint64_t a_desc = sw128_kmajor_desc(stage + t * C::kWBytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8f6f4(d_tmem, a_desc + 2 * k, b_desc + 2 * k, C::kIdesc, k > 0 ? 1u : 0u);
                }
                mma_commit(&empty[s]);
                mma_commit(&tfull[acc]);
            }
            __syncwarp();
            if (++acc == C::kAcc) {
                acc = 0;
                acc_ph ^= 1u;
            }
            s = s1;
            ph = ph1;
        }
        if (leader) {
            // every MMA complete before the tensor memory is released
            mma_commit(mma_done);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_test(mma_done, 0)) {
                if (globaltimer_ns() - t0 > p.timeout_ns) {
                    atomicOr(p.status, kErrTimeoutDrain);
                    break;
                }
            }
        }
    } else {
        // ------------------------------------------------ promotion / epilogue
        const int quarter = warp & 3; // TMEM lanes this warp may read
        const int row = quarter * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const int col0 = ((warp - 2) >> 2) * C::kCols; // this thread's token columns
        const int mcnt = p.M - col0;                   // of them that exist (may exceed kCols)
        float acc[C::kTiles][C::kCols];
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
            for (int m = 0; m < C::kCols; ++m)
                acc[t][m] = 0.0f;
        int accb = 0;
        uint32_t acc_ph = 0;
        Unit u = first_unit();
        int tile = tile0, seg_first = ku0;
        // Contributors of the (at most two) tiles this CTA shares, as in gemm_kernel.cuh.
        struct SplitPlan {
            int c_first, c_last, slot_first;
        };
        auto make_plan = [&](int t) {
            const long long tf = static_cast<long long>(t) * kg;
            SplitPlan sp;
            sp.c_first = owner(tf);
            sp.c_last = owner(tf + kg - 1);
            sp.slot_first = 2 * sp.c_first + (range_begin(sp.c_first) == tf ? 0 : 1);
            return sp;
        };
        const int tile_b = tile0 + (has ? (ku0 + nunits - 1) / kg : 0);
        SplitPlan plan_a = {0, 0, 0}, plan_b = {0, 0, 0};
        if (nunits > 0) {
            plan_a = make_plan(tile0);
            plan_b = tile_b != tile0 ? make_plan(tile_b) : plan_a;
        }
        // The weight blocks' scales of the first 32 units to L1 (a lane a unit):
        // in a short range their first use would wait for memory unit by unit.
        if (warp == 2 && lane < nunits) {
            const int ku = ku0 + lane, t = tile0 + ku / kg, r = ku % kg;
            Unit v;
            v.ku = r;
            v.a = kUp ? t / nj : r / kg1;
            v.j = kUp ? t % nj : t;
            v.kb = kUp ? r : r % kg1;
            if (unit_ok(v))
#pragma unroll
                for (int q = 0; q < C::kTiles; ++q)
                    prefetch_l1(p.ws + weight_tile(v, q) * kg1 + v.kb);
        }
        if (!kUp)
            grid_dependency_wait();
        // Scales of the units to promote, loaded kAhead units ahead: the weight
        // blocks', and this lane's token's.
        struct Scales {
            float w[C::kTiles], a;
        };
        constexpr int kAhead = 2;
        Scales nx[kAhead];
        auto load_scales = [&](const Unit &v) {
            Scales r = {};
            if (!unit_ok(v))
                return r;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
                r.w[t] = p.ws[weight_tile(v, t) * kg1 + v.kb];
            if (lane < C::kCols && lane < mcnt)
                r.a = kUp ? __ldcg(p.xs + v.kb * p.M + col0 + lane)
                          : __ldcg(p.hs + (static_cast<long long>(v.a) * kg1 + v.kb) * NPAD + col0 + lane);
            return r;
        };
        Unit un = u; // the unit whose scales are loaded next
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            nx[q] = Scales{};
            if (q < nunits)
                nx[q] = load_scales(un);
            step(un);
        }
        float *const wprod = prod + (warp - 2) * 2 * C::kTiles * C::kCols;
        // up: the tokens' weights for the unit's expert, this lane's tokens
        // lane and lane + 32; read when the expert changes, used at a tile's end
        float w_tok[2] = {0.0f, 0.0f};
        auto load_weights = [&](int a) {
            const float *wt = p.wtok + static_cast<long long>(act[a]) * NPAD;
#pragma unroll
            for (int q = 0; q < (NPAD + 31) / 32; ++q)
                w_tok[q] = lane + 32 * q < p.M ? __ldcg(wt + lane + 32 * q) : 0.0f;
        };
        if (kUp && nunits > 0 && unit_ok(u))
            load_weights(u.a);

        // down: finished sums of one output tile (thread = row `row` of it)
        auto store_y = [&]() {
            const int n = u.j * 128 + row;
#pragma unroll
            for (int m = 0; m < C::kCols; ++m)
                if (m < mcnt)
                    p.y[static_cast<long long>(col0 + m) * p.H + n] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(acc[0][m]));
        };
        // up: one pair of tiles from its contributors' partials in the slots:
        // h, its scale and codes, a warp a token (128 rows, four a lane).  The
        // chosen tokens are dealt to the warps in turn; the
        // others get zero codes (written, not multiplied in: an unchosen
        // expert's sums may be infinite).  The loops stay rolled: this code
        // runs once or twice a CTA, and unrolled over the tokens its
        // instruction fetches alone took 11 us.
        constexpr int kSlot = C::kTiles * NPAD * 128;
        auto finish_up = [&](int c_first, int c_last, int slot_first) {
            const int ew = warp - 2;
            unsigned long long chosen = __ballot_sync(0xffffffffu, w_tok[0] != 0.0f);
            if constexpr (NPAD > 32)
                chosen |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, w_tok[1] != 0.0f)) << 32;
            const long long hrow = static_cast<long long>(u.a) * NPAD;
            float *const hs = p.hs + (static_cast<long long>(u.a) * nj + u.j) * NPAD;
            uint8_t *const hq = p.hq + hrow * p.I + u.j * 128 + 4 * lane;
#pragma unroll 1
            for (int m = ew; m < p.M; m += C::kEpiWarps) {
                if (chosen >> m & 1ull)
                    continue;
                *reinterpret_cast<uint32_t *>(hq + static_cast<long long>(m) * p.I) = 0u;
                if (lane == 0)
                    __stcg(hs + m, 0.0f);
            }
            // the warp's chosen tokens: numbers ew, ew + kEpiWarps, ... of the
            // set bits; four contributors' partials in flight at a time
            int rank = 0;
#pragma unroll 1
            for (; chosen != 0ull; chosen &= chosen - 1ull) {
                if (rank++ % C::kEpiWarps != ew)
                    continue;
                const int m = __ffsll(static_cast<long long>(chosen)) - 1;
                float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, up[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const float *const src = p.slots + m * 128 + 4 * lane;
#pragma unroll 1
                for (int c0 = c_first; c0 <= c_last; c0 += 4) {
                    float4 vg[4], vu[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + q <= c_last ? c0 + q : c_last;
                        const float *s = src + static_cast<long long>(c == c_first ? slot_first : 2 * c) * kSlot;
                        vg[q] = __ldcg(reinterpret_cast<const float4 *>(s));
                        vu[q] = __ldcg(reinterpret_cast<const float4 *>(s + NPAD * 128));
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (c0 + q <= c_last) {
                            add2(h[0], h[1], vg[q].x, vg[q].y);
                            add2(h[2], h[3], vg[q].z, vg[q].w);
                            add2(up[0], up[1], vu[q].x, vu[q].y);
                            add2(up[2], up[3], vu[q].z, vu[q].w);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    h[q] = __fdiv_rn(h[q], 1.0f + expf(-h[q])) * up[q];
                const float s = group_scale(warp_max(abs_max4(h[0], h[1], h[2], h[3])));
                *reinterpret_cast<uint32_t *>(hq + static_cast<long long>(m) * p.I) =
                    quantize4(h[0], h[1], h[2], h[3], s);
                const float w = __shfl_sync(0xffffffffu, NPAD > 32 && m >= 32 ? w_tok[1] : w_tok[0], m & 31);
                if (lane == 0)
                    __stcg(hs + m, s * w);
            }
        };

        // down: a tile's sum over its contributors, a warp a token (four rows
        // a lane).  The time is the L2's round trips: kTok tokens of kCon
        // contributors, 12 KB a warp, are in flight at a time, and the loops
        // over more of either stay rolled.  (Thread = row, six contributors of
        // eight tokens, took 41.6 us where this takes 35.0, a layer of 50 tokens
        // with 22 contributors a tile; bulk copies into the idle ring, eight in
        // flight, 40.6.  Four tokens of six contributors: 13 tokens 29.7 us, not
        // 30.0, but one token of 128 experts 22.1, not 21.5.)
        auto finish_down = [&](int c_first, int c_last, int slot_first) {
            constexpr int kTok = 2, kCon = 12;
            const int ew = warp - 2;
            uint16_t *const y = p.y + u.j * 128 + 4 * lane;
            const bool y_wide = (reinterpret_cast<uintptr_t>(p.y) & 7u) == 0; // (the entry asks for two bytes)
#pragma unroll 1
            for (int m0 = ew; m0 < p.M; m0 += kTok * C::kEpiWarps) {
                float sum[kTok][4] = {};
#pragma unroll 1
                for (int c0 = c_first; c0 <= c_last; c0 += kCon) {
                    float4 v[kCon][kTok];
#pragma unroll
                    for (int q = 0; q < kCon; ++q) {
                        const int c = c0 + q;
                        const float *const src =
                            p.slots + static_cast<long long>(c == c_first ? slot_first : 2 * c) * kSlot + 4 * lane;
#pragma unroll
                        for (int t = 0; t < kTok; ++t) {
                            const int m = m0 + t * C::kEpiWarps;
                            v[q][t] = c <= c_last && m < p.M ? __ldcg(reinterpret_cast<const float4 *>(src + m * 128))
                                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < kCon; ++q)
                        if (c0 + q <= c_last)
#pragma unroll
                            for (int t = 0; t < kTok; ++t) {
                                add2(sum[t][0], sum[t][1], v[q][t].x, v[q][t].y);
                                add2(sum[t][2], sum[t][3], v[q][t].z, v[q][t].w);
                            }
                }
#pragma unroll
                for (int t = 0; t < kTok; ++t) {
                    if (m0 + t * C::kEpiWarps >= p.M)
                        break;
                    uint16_t *const to = y + static_cast<long long>(m0 + t * C::kEpiWarps) * p.H;
                    ushort4 b;
                    b.x = __bfloat16_as_ushort(__float2bfloat16_rn(sum[t][0]));
                    b.y = __bfloat16_as_ushort(__float2bfloat16_rn(sum[t][1]));
                    b.z = __bfloat16_as_ushort(__float2bfloat16_rn(sum[t][2]));
                    b.w = __bfloat16_as_ushort(__float2bfloat16_rn(sum[t][3]));
                    if (y_wide)
                        *reinterpret_cast<ushort4 *>(to) = b;
                    else
                        to[0] = b.x, to[1] = b.y, to[2] = b.z, to[3] = b.w;
                }
            }
        };

        for (int i = 0; i < nunits; ++i) {
            const bool seg_end = (i == nunits - 1) || (u.ku == kg - 1);
            // s_w * s_a of this unit's tokens, per warp (double-buffered by
            // parity: rewritten only after every lane passed the next __syncwarp)
            float *pr = wprod + (i & 1) * C::kTiles * C::kCols;
            // down: the tokens that chose this unit's expert.  The others' codes
            // and scales are 0, but 0 times a weight or a block scale that is not
            // finite is NaN, and an expert's is to reach no token beside its own.
            // (A NaN among a row's 128 weights makes all its columns NaN, the
            // first among them, so the sums are looked through only then:
            // doing it always took 250 us where 64 tokens take 239.)
            const unsigned chose = kUp ? 0u : __ballot_sync(0xffffffffu, nx[0].a != 0.0f);
            if (lane < C::kCols) {
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t)
                    pr[t * C::kCols + lane] = kUp || nx[0].a != 0.0f ? nx[0].w[t] * nx[0].a : 0.0f;
            }
            __syncwarp();
            Unit nu = u;
            step(nu);
#pragma unroll
            for (int q = 0; q + 1 < kAhead; ++q)
                nx[q] = nx[q + 1];
            if (i + kAhead < nunits)
                nx[kAhead - 1] = load_scales(un);
            step(un);
            mbar_wait(&tfull[accb], acc_ph, abort_flag, p.status, kErrTimeoutEpilogue, p.timeout_ns);
            // (a wait that gave up carries on in bounds, as in gemm_kernel.cuh)
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + lane_addr + static_cast<uint32_t>(accb * C::kAccCols + col0);
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
                uint32_t r[C::kCols];
                tmem_issue(taddr + t * NPAD, r);
                tmem_wait(r);
                if (!kUp && isnan(__uint_as_float(r[0])))
#pragma unroll
                    for (int q = 0; q < C::kCols; ++q)
                        r[q] = chose >> q & 1u ? r[q] : 0u;
#pragma unroll
                for (int q = 0; q < C::kCols / 4; ++q) {
                    const float4 sc = reinterpret_cast<const float4 *>(pr + t * C::kCols)[q];
                    fma2(acc[t][4 * q], acc[t][4 * q + 1], sc.x, sc.y, __uint_as_float(r[4 * q]),
                         __uint_as_float(r[4 * q + 1]));
                    fma2(acc[t][4 * q + 2], acc[t][4 * q + 3], sc.z, sc.w, __uint_as_float(r[4 * q + 2]),
                         __uint_as_float(r[4 * q + 3]));
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&tempty[accb]);
            if (++accb == C::kAcc) {
                accb = 0;
                acc_ph ^= 1u;
            }
            if (seg_end) {
                const bool whole = seg_first == 0 && u.ku == kg - 1;
                if (!kUp && whole) {
                    store_y();
                } else {
                    // shared tile: publish this CTA's partial; the last
                    // contributor to arrive sums all of them in order (up:
                    // also for a whole tile, by way of a slot of its own)
                    SplitPlan pl = tile == tile0 ? plan_a : plan_b;
                    if (kUp && whole)
                        pl.c_first = pl.c_last = cta, pl.slot_first = 2 * static_cast<int>(gridDim.x) + cta;
                    auto slot_of = [&](int c) { return c == pl.c_first ? pl.slot_first : 2 * c; };
                    const bool ex_ok =
                        FP8BS_CHECK(pl.c_first >= 0 && pl.c_first <= cta && cta <= pl.c_last && pl.c_last < ctas &&
                                    slot_of(cta) < (kUp ? 3 : 2) * static_cast<int>(gridDim.x) && tile >= 0 && tile < tiles);
                    float *mine = p.slots + static_cast<long long>(slot_of(cta)) * kSlot + col0 * 128 + row;
#pragma unroll
                    for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
                        for (int m = 0; m < C::kCols; ++m)
                            if (m < mcnt && ex_ok)
                                __stcg(mine + (t * NPAD + m) * 128, acc[t][m]);
                    named_bar_sync(1, 32 * C::kEpiWarps);
                    if (!(kUp && whole)) {
                        if (warp == 2 && lane == 0) {
                            const unsigned prev = ex_ok ? atomic_add_acq_rel_gpu(&p.counters[tile], 1u) : 0u;
                            *last_flag = (ex_ok && prev == static_cast<unsigned>(pl.c_last - pl.c_first)) ? 1 : 0;
                        }
                        named_bar_sync(1, 32 * C::kEpiWarps);
                    }
                    if (kUp && (whole || *last_flag)) {
                        if (ex_ok)
                            finish_up(pl.c_first, pl.c_last, pl.slot_first);
                        if (warp == 2 && lane == 0 && !whole)
                            p.counters[tile] = 0u; // ready for the next call
                    } else if (!kUp && *last_flag) {
                        finish_down(pl.c_first, pl.c_last, pl.slot_first);
                        if (warp == 2 && lane == 0)
                            p.counters[tile] = 0u;
                    }
                    named_bar_sync(1, 32 * C::kEpiWarps); // last_flag and the whole tiles' slot may be written again
                }
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
                    for (int m = 0; m < C::kCols; ++m)
                        acc[t][m] = 0.0f;
                ++tile;
                seg_first = 0;
                if (kUp && i + 1 < nunits && nu.a != u.a && unit_ok(nu))
                    load_weights(nu.a);
            }
            u = nu;
        }
        // No token chose any expert: the layer's output is zero.
        if (!kUp && A == 0) {
            const long long n = static_cast<long long>(p.M) * p.H;
            for (long long i = static_cast<long long>(cta) * (32 * C::kEpiWarps) + (threadIdx.x - 64); i < n;
                 i += static_cast<long long>(gridDim.x) * (32 * C::kEpiWarps))
                p.y[i] = 0;
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (!kUp && cta == 0 && threadIdx.x == 0)
        store_release_gpu(p.chosen, 0u); // (this thread has waited for the up product)
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

template <int NPAD, int PHASE>
fp8bs_status launch_moe_gemm(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    using C = MoeCfg<NPAD, PHASE>;
    static unsigned long long attr_done = 0;
    constexpr bool kUp = PHASE == kMoeUp;
    constexpr int kSmemLimit = 227 * 1024;
    auto kernel = moe_gemm_kernel<NPAD, PHASE>;
    // (two CTAs: the up product's and the down product's together fit an SM)
    int stages = (C::kMinBlocks == 2 ? (kUp ? 108 : 104) * 1024 : 204 * 1024) / C::kStageBytes;
    stages = stages > C::kMaxStages ? C::kMaxStages : stages;
    const int smem = C::smem_bytes(stages);
    fp8bs_status st = ensure_smem_attr(reinterpret_cast<const void *>(kernel), kSmemLimit, dev.device, &attr_done);
    if (st != FP8BS_OK)
        return st;
    const int max_active = L.E < L.M * L.top_k ? L.E : L.M * L.top_k;
    const uint64_t rows = static_cast<uint64_t>(L.E) * (kUp ? 2 * L.I : L.H);
    const uint64_t cols = static_cast<uint64_t>(kUp ? L.H : L.I);
    CUtensorMap tm_w, tm_b;
    const void *wp = kUp ? L.w13 : L.w2;
    if (L.flags & FP8BS_FLAG_WEIGHTS_TILED)
        st = make_tmap_2d(&tm_w, wp, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows / 128 * cols, 128, 128, 128, 128);
    else
        st = make_tmap_2d(&tm_w, wp, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, cols, cols, 128, 128);
    if (st == FP8BS_OK)
        st = kUp ? make_tmap_2d(&tm_b, L.workspace + w.xq_off, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                                static_cast<uint64_t>(L.M), cols, cols, 128, NPAD)
                 : make_tmap_2d(&tm_b, L.workspace + w.hq_off, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                                static_cast<uint64_t>(max_active) * NPAD, cols, cols, 128, NPAD);
    if (st != FP8BS_OK)
        return st;
    MoeGemmParams p = {};
    p.M = L.M;
    p.H = L.H;
    p.I = L.I;
    p.E = L.E;
    p.stages = stages;
    p.masks = reinterpret_cast<const unsigned *>(L.workspace + w.masks_off);
    p.chosen = reinterpret_cast<unsigned *>(L.workspace + w.chosen_off);
    p.groups = L.wr != nullptr ? (L.M + kMoeTokenGroup - 1) / kMoeTokenGroup : 1; // (a given choice: one)
    p.wtok = reinterpret_cast<const float *>(L.workspace + w.wtok_off);
    p.ws = kUp ? L.s13 : L.s2;
    p.xs = reinterpret_cast<const float *>(L.workspace + w.xs_off);
    p.hq = L.workspace + w.hq_off;
    p.hs = reinterpret_cast<float *>(L.workspace + w.hs_off);
    p.y = static_cast<uint16_t *>(L.y);
    p.status = reinterpret_cast<unsigned *>(L.workspace);
    p.counters = reinterpret_cast<unsigned *>(L.workspace + (kUp ? w.counters_up_off : w.counters_down_off));
    p.slots = reinterpret_cast<float *>(L.workspace + w.slots_off);
    p.w_tiled = (L.flags & FP8BS_FLAG_WEIGHTS_TILED) ? 1 : 0;
    p.max_active = max_active;
    p.test_skip_unit = L.test_skip_phase == PHASE ? L.test_skip_unit : -1;
    p.timeout_ns = L.timeout_ns;
    p.runs = dev.runs;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.sms), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1; // follows this layer's own kernel, and waits for it
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_b, p));
}

template <int PHASE> fp8bs_status launch_moe_phase(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev)
{
    switch (moe_token_pad(L.M)) {
    case 16:
        return launch_moe_gemm<16, PHASE>(L, w, dev);
    case 32:
        return launch_moe_gemm<32, PHASE>(L, w, dev);
    default:
        return launch_moe_gemm<64, PHASE>(L, w, dev);
    }
}

} // namespace fp8bs
