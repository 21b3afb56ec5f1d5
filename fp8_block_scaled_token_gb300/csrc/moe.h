// moe.h -- host-side plumbing of the mixture-of-experts layer (moe.cu,
// moe_route.cu, moe_scored.cu, moe_up.cu, moe_down.cu); not part of the public ABI.
#pragma once

#include "internal.h"

namespace fp8bs {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxGroups = 32;
constexpr int kMoeMaxSplits = 4; // of H in the router's product under scores
constexpr int kMoeTokenGroup = 8; // tokens that one routing CTA multiplies an expert's router row with

inline int moe_token_pad(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// Workspace of one expert layer.  [0, 256) the status word; the routing
// words and the arrival counters are zero between calls and where no
// operator's data lies (internal.h).  The routing alone uses what comes before
// masks_off.
constexpr size_t kMoeRouteOff = 832;
struct MoeWorkspace {
    size_t route_off;         // arrival counters of the kMoeMaxTokens / kMoeTokenGroup groups of tokens, then a
                              // bit mask of the experts (kMoeMaxExperts / 32 words) for a given choice
    size_t chosen_off;        // 1 from the gate/up product's start to the down product's end: the masks are complete
    size_t logits_off;        // [M][E] router logits; under scores [splits of H][M][E] partial sums
    size_t counters_up_off;   // arrival counters of the (active expert, 128 of I) pairs
    size_t counters_down_off; // arrival counters of the 128-row tiles of H
    size_t counters_bytes;    // of both
    size_t masks_off;         // [groups of tokens][kMoeMaxExperts / 32] bit masks of the experts they chose
    size_t ids_off;           // [M][top_k] chosen experts, where the caller keeps none
    size_t topw_off;          // [M][top_k] their weights
    size_t wtok_off;          // [E][NPAD] weight of each token for each expert, 0 where not chosen
    size_t xq_off, xs_off;    // activations: codes [M][H], scales [H/128][M]
    size_t hq_off, hs_off;    // intermediate: codes [active][NPAD][I], scales times weights [active][I/128][NPAD]
    size_t slots_off;         // partials, [3 * SMs][2][NPAD * 128] fp32
    size_t total;
};

// How experts are scored and grouped; scored = false is the plain top_k of the logits.
struct MoeScores {
    bool scored = false;
    int planes() const { return scored ? kMoeMaxSplits : 1; }
    bool sigmoid = false;
    const float *bias = nullptr; // [E], or nullptr
    int groups = 1, top_groups = 1, group_best = 1;
    float scale = 1.0f;
};

struct MoeLaunch {
    int M, H, I, E, top_k;
    const void *x;
    int ldx;
    const void *wr;          // router weights [E][H], or nullptr: ids and topw are given
    int wr_type;
    int renorm;
    MoeScores scores;        // of moe_route_grouped and fp8_moe_layer_grouped
    const uint8_t *w13, *w2; // tiled or row-major E4M3
    const float *s13, *s2;
    int32_t *ids;
    float *topw;
    void *y;
    uint8_t *workspace;
    unsigned flags;
    cudaStream_t stream;
    unsigned long long timeout_ns;
    int test_skip_unit = -1;  // -1, or a unit whose stage the producer of phase test_skip_phase never fills
    int test_skip_phase = 0;  // 0 = gate/up, 1 = down
};

// planes: of [M][E] logits, 1 under the plain choice and kMoeMaxSplits under scores.  The size queries report the
// larger layout, which both calls may use; each call asks for its own.
MoeWorkspace moe_workspace(int M, int H, int I, int E, int top_k, int sms, int planes);
fp8bs_status launch_moe_scored(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev);
fp8bs_status launch_moe_route(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev);
fp8bs_status launch_moe_up(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev);
fp8bs_status launch_moe_down(const MoeLaunch &L, const MoeWorkspace &w, const DeviceInfo &dev);

} // namespace fp8bs
