// moe.cu -- entry points of the mixture-of-experts layer: argument checks on
// the host, the workspace's layout, and the three launches (routing or plan,
// gate/up product, down product).
#include <cmath>

#include "fp8bs_testing.h"
#include "moe.h"

namespace fp8bs {

MoeWorkspace moe_workspace(int M, int H, int I, int E, int top_k, int sms, int planes)
{
    auto up256 = [](size_t b) { return (b + 255) / 256 * 256; };
    const size_t npad = static_cast<size_t>(moe_token_pad(M));
    const size_t active = static_cast<size_t>(E < M * top_k ? E : M * top_k);
    MoeWorkspace w;
    w.route_off = kMoeRouteOff;
    w.chosen_off = kMoeRouteOff + (kMoeMaxTokens / kMoeTokenGroup + kMoeMaxExperts / 32) * 4;
    w.counters_down_off = kCountersOff;
    w.counters_up_off = w.counters_down_off + static_cast<size_t>(H / 128) * 4;
    w.counters_bytes = static_cast<size_t>(H / 128) * 4 + active * (I / 128) * 4;
    w.logits_off = kCountersOff + counters_region(w.counters_bytes);
    w.masks_off = w.logits_off + up256(static_cast<size_t>(M) * E * 4 * planes);
    w.ids_off = w.masks_off + static_cast<size_t>(kMoeMaxTokens / kMoeTokenGroup) * (kMoeMaxExperts / 32) * 4;
    w.topw_off = w.ids_off + up256(static_cast<size_t>(M) * top_k * 4);
    w.wtok_off = w.topw_off + up256(static_cast<size_t>(M) * top_k * 4);
    w.xq_off = w.wtok_off + up256(static_cast<size_t>(E) * npad * 4);
    w.xs_off = w.xq_off + up256(static_cast<size_t>(M) * H);
    w.hq_off = w.xs_off + up256(static_cast<size_t>(M) * (H / 128) * 4);
    w.hs_off = w.hq_off + up256(active * npad * I);
    w.slots_off = w.hs_off + up256(active * (I / 128) * npad * 4);
    w.total = w.slots_off + static_cast<size_t>(3) * sms * 2 * npad * 128 * 4;
    return w;
}

namespace {

// The routing words lie behind the GEMMs' greedy keys and counter (64 64-bit
// words and one 32-bit word from byte 256), which like them are zero between calls.
static_assert(kMoeRouteOff >= 256 + 64 * 8 + 4 &&
                  kMoeRouteOff + (kMoeMaxTokens / kMoeTokenGroup + kMoeMaxExperts / 32 + 1) * 4 <= kCountersOff,
              "routing words");
static_assert(kMoeMaxTokens / kMoeTokenGroup * (kMoeMaxExperts / 32) * 4 % 256 == 0, "masks");

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What the choice and the products share: token, expert and K counts.
fp8bs_status check_tokens(int M, int H, int E, int top_k)
{
    if (M < 1 || H < 1 || E < 1 || top_k < 1)
        return FP8BS_ERR_INVALID_ARG;
    if (M > kMoeMaxTokens || E > kMoeMaxExperts || top_k > kMoeMaxTopK || top_k > E || H % 128 != 0 || H > (1 << 24))
        return FP8BS_ERR_UNSUPPORTED_SHAPE;
    return FP8BS_OK;
}

fp8bs_status check_experts(int M, int H, int I, int E, int top_k)
{
    fp8bs_status st = check_tokens(M, H, E, top_k);
    if (st != FP8BS_OK)
        return st;
    if (I < 1)
        return FP8BS_ERR_INVALID_ARG;
    // 128x128 weight tiles of each matrix within the tensor maps' 31-bit row coordinates
    if (I % 128 != 0 || I > (1 << 24) ||
        static_cast<long long>(E) * 2 * (I / 128) * (H / 128) >= (1ll << 24))
        return FP8BS_ERR_UNSUPPORTED_SHAPE;
    return FP8BS_OK;
}

constexpr unsigned kMoeFlags = FP8BS_FLAG_OVERLAP_PREV | FP8BS_FLAG_WEIGHTS_TILED;

fp8bs_status run_experts(MoeLaunch &L, size_t workspace_bytes)
{
    DeviceInfo dev;
    fp8bs_status st = current_device(&dev);
    if (st != FP8BS_OK)
        return st;
    const MoeWorkspace w = moe_workspace(L.M, L.H, L.I, L.E, L.top_k, dev.sms, L.scores.planes());
    if (workspace_bytes < w.total)
        return FP8BS_ERR_WORKSPACE_TOO_SMALL;
    if (L.ids == nullptr)
        L.ids = reinterpret_cast<int32_t *>(L.workspace + w.ids_off);
    if (L.topw == nullptr)
        L.topw = reinterpret_cast<float *>(L.workspace + w.topw_off);
    st = zero_far_counters(L.workspace, w.counters_bytes, L.stream);
    if (st == FP8BS_OK)
        st = launch_moe_route(L, w, dev);
    if (st == FP8BS_OK)
        st = launch_moe_up(L, w, dev);
    if (st == FP8BS_OK)
        st = launch_moe_down(L, w, dev);
    return st;
}

// Scores, groups and the router's weights of a grouped choice.
fp8bs_status set_scores(MoeLaunch &L, const void *wr, fp8bs_dtype wr_type, const float *bias, fp8bs_score scoring,
                        int groups, int top_groups, int group_best, int renormalize, float scale)
{
    if (!wr || (wr_type != FP8BS_F32 && wr_type != FP8BS_BF16) ||
        (scoring != FP8BS_SCORE_SOFTMAX && scoring != FP8BS_SCORE_SIGMOID) || groups < 1 || top_groups < 1 ||
        top_groups > groups || group_best < 1 || group_best > 2 || !std::isfinite(scale))
        return FP8BS_ERR_INVALID_ARG;
    if (groups > kMoeMaxGroups || L.E % groups != 0 || L.top_k > top_groups * (L.E / groups) ||
        (top_groups < groups && group_best > L.E / groups))
        return FP8BS_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(wr, 16) || !aligned(bias, 4))
        return FP8BS_ERR_MISALIGNED;
    L.wr = wr;
    L.wr_type = wr_type;
    L.renorm = renormalize != 0;
    L.scores.scored = true;
    L.scores.sigmoid = scoring == FP8BS_SCORE_SIGMOID;
    L.scores.bias = bias;
    L.scores.groups = groups;
    L.scores.top_groups = top_groups;
    L.scores.group_best = group_best;
    L.scores.scale = scale;
    return FP8BS_OK;
}

MoeLaunch route_call(const void *x, int ldx, int M, int H, int E, int top_k, int32_t *ids, float *weights,
                     void *workspace, unsigned flags, void *stream)
{
    MoeLaunch L = {};
    L.M = M;
    L.H = H;
    L.E = E;
    L.top_k = top_k;
    L.x = x;
    L.ldx = ldx;
    L.ids = ids;
    L.topw = weights;
    L.workspace = static_cast<uint8_t *>(workspace);
    L.flags = flags;
    L.stream = static_cast<cudaStream_t>(stream);
    return L;
}

fp8bs_status check_route(const MoeLaunch &L)
{
    if (!L.x || !L.ids || !L.topw || !L.workspace)
        return FP8BS_ERR_INVALID_ARG;
    fp8bs_status st = check_tokens(L.M, L.H, L.E, L.top_k);
    if (st != FP8BS_OK)
        return st;
    if (L.ldx < L.H || (L.flags & ~FP8BS_FLAG_OVERLAP_PREV) != 0)
        return FP8BS_ERR_INVALID_ARG;
    if (!aligned(L.x, 16) || L.ldx % 8 != 0 || !aligned(L.ids, 4) || !aligned(L.topw, 4) || !aligned(L.workspace, 256))
        return FP8BS_ERR_MISALIGNED;
    return FP8BS_OK;
}

fp8bs_status run_route(const MoeLaunch &L, size_t workspace_bytes)
{
    DeviceInfo dev;
    fp8bs_status st = current_device(&dev);
    if (st != FP8BS_OK)
        return st;
    // the routing's part depends on M, E and the planes alone
    const MoeWorkspace w = moe_workspace(L.M, 128, 128, L.E, 1, dev.sms, L.scores.planes());
    if (workspace_bytes < w.masks_off)
        return FP8BS_ERR_WORKSPACE_TOO_SMALL;
    return launch_moe_route(L, w, dev);
}

fp8bs_status check_layer(const MoeLaunch &L)
{
    if (!L.x || !L.w13 || !L.s13 || !L.w2 || !L.s2 || !L.y || !L.workspace)
        return FP8BS_ERR_INVALID_ARG;
    fp8bs_status st = check_experts(L.M, L.H, L.I, L.E, L.top_k);
    if (st != FP8BS_OK)
        return st;
    if (L.ldx < L.H || (L.flags & ~kMoeFlags) != 0)
        return FP8BS_ERR_INVALID_ARG;
    if (!aligned(L.x, 16) || L.ldx % 8 != 0 || !aligned(L.w13, 16) || !aligned(L.w2, 16) || !aligned(L.s13, 4) ||
        !aligned(L.s2, 4) || !aligned(L.y, 2) || !aligned(L.ids, 4) || !aligned(L.topw, 4) ||
        !aligned(L.workspace, 256))
        return FP8BS_ERR_MISALIGNED;
    return FP8BS_OK;
}

} // namespace

} // namespace fp8bs

using namespace fp8bs;

extern "C" {

fp8bs_status moe_route_workspace_size(int M, int E, size_t *bytes)
{
    if (!bytes)
        return FP8BS_ERR_INVALID_ARG;
    *bytes = 0;
    fp8bs_status st = check_tokens(M, 128, E, 1);
    if (st != FP8BS_OK)
        return st;
    *bytes = moe_workspace(M, 128, 128, E, 1, 1, kMoeMaxSplits).masks_off;
    return FP8BS_OK;
}

fp8bs_status moe_route(const void *x, int ldx, const void *wr, fp8bs_dtype wr_type, int M, int H, int E, int top_k,
                       int renormalize, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes,
                       unsigned flags, void *stream)
{
    if (!wr || (wr_type != FP8BS_F32 && wr_type != FP8BS_BF16))
        return FP8BS_ERR_INVALID_ARG;
    MoeLaunch L = route_call(x, ldx, M, H, E, top_k, ids, weights, workspace, flags, stream);
    L.wr = wr;
    L.wr_type = wr_type;
    L.renorm = renormalize != 0;
    fp8bs_status st = check_route(L);
    if (st == FP8BS_OK && !aligned(wr, 16))
        st = FP8BS_ERR_MISALIGNED;
    return st != FP8BS_OK ? st : run_route(L, workspace_bytes);
}

fp8bs_status moe_route_grouped(const void *x, int ldx, const void *wr, fp8bs_dtype wr_type, const float *bias, int M,
                               int H, int E, int top_k, fp8bs_score scoring, int groups, int top_groups,
                               int group_best, int renormalize, float scale, int32_t *ids, float *weights,
                               void *workspace, size_t workspace_bytes, unsigned flags, void *stream)
{
    MoeLaunch L = route_call(x, ldx, M, H, E, top_k, ids, weights, workspace, flags, stream);
    fp8bs_status st = check_route(L);
    if (st == FP8BS_OK)
        st = set_scores(L, wr, wr_type, bias, scoring, groups, top_groups, group_best, renormalize, scale);
    return st != FP8BS_OK ? st : run_route(L, workspace_bytes);
}

fp8bs_status fp8_moe_workspace_size(int M, int H, int I, int E, int top_k, size_t *bytes)
{
    if (!bytes)
        return FP8BS_ERR_INVALID_ARG;
    *bytes = 0;
    fp8bs_status st = check_experts(M, H, I, E, top_k);
    if (st != FP8BS_OK)
        return st;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != FP8BS_OK)
        return st;
    *bytes = moe_workspace(M, H, I, E, top_k, dev.sms, kMoeMaxSplits).total;
    return FP8BS_OK;
}

fp8bs_status fp8_moe_experts(const void *x, int ldx, const int32_t *ids, const float *weights, const uint8_t *w13,
                             const float *s13, const uint8_t *w2, const float *s2, void *y, int M, int H, int I, int E,
                             int top_k, void *workspace, size_t workspace_bytes, unsigned flags, void *stream)
{
    if (!ids || !weights)
        return FP8BS_ERR_INVALID_ARG;
    MoeLaunch L = {};
    L.M = M;
    L.H = H;
    L.I = I;
    L.E = E;
    L.top_k = top_k;
    L.x = x;
    L.ldx = ldx;
    L.ids = const_cast<int32_t *>(ids); // read only: no router weights
    L.topw = const_cast<float *>(weights);
    L.test_skip_unit = -1;
    L.w13 = w13;
    L.s13 = s13;
    L.w2 = w2;
    L.s2 = s2;
    L.y = y;
    L.workspace = static_cast<uint8_t *>(workspace);
    L.flags = flags;
    L.stream = static_cast<cudaStream_t>(stream);
    L.timeout_ns = kDefaultTimeoutNs;
    fp8bs_status st = check_layer(L);
    return st != FP8BS_OK ? st : run_experts(L, workspace_bytes);
}

fp8bs_status fp8_moe_layer(const void *x, int ldx, const void *wr, fp8bs_dtype wr_type, int renormalize,
                           const uint8_t *w13, const float *s13, const uint8_t *w2, const float *s2, void *y,
                           int32_t *ids, float *weights, int M, int H, int I, int E, int top_k, void *workspace,
                           size_t workspace_bytes, unsigned flags, void *stream)
{
    if (!wr || (wr_type != FP8BS_F32 && wr_type != FP8BS_BF16))
        return FP8BS_ERR_INVALID_ARG;
    MoeLaunch L = {};
    L.M = M;
    L.H = H;
    L.I = I;
    L.E = E;
    L.top_k = top_k;
    L.x = x;
    L.ldx = ldx;
    L.wr = wr;
    L.wr_type = wr_type;
    L.renorm = renormalize != 0;
    L.ids = ids;
    L.topw = weights;
    L.test_skip_unit = -1;
    L.w13 = w13;
    L.s13 = s13;
    L.w2 = w2;
    L.s2 = s2;
    L.y = y;
    L.workspace = static_cast<uint8_t *>(workspace);
    L.flags = flags;
    L.stream = static_cast<cudaStream_t>(stream);
    L.timeout_ns = kDefaultTimeoutNs;
    fp8bs_status st = check_layer(L);
    if (st == FP8BS_OK && !aligned(wr, 16))
        st = FP8BS_ERR_MISALIGNED;
    return st != FP8BS_OK ? st : run_experts(L, workspace_bytes);
}

fp8bs_status fp8_moe_layer_grouped(const void *x, int ldx, const void *wr, fp8bs_dtype wr_type, const float *bias,
                                   fp8bs_score scoring, int groups, int top_groups, int group_best, int renormalize,
                                   float scale, const uint8_t *w13, const float *s13, const uint8_t *w2,
                                   const float *s2, void *y, int32_t *ids, float *weights, int M, int H, int I, int E,
                                   int top_k, void *workspace, size_t workspace_bytes, unsigned flags, void *stream)
{
    MoeLaunch L = {};
    L.M = M;
    L.H = H;
    L.I = I;
    L.E = E;
    L.top_k = top_k;
    L.x = x;
    L.ldx = ldx;
    L.ids = ids;
    L.topw = weights;
    L.test_skip_unit = -1;
    L.w13 = w13;
    L.s13 = s13;
    L.w2 = w2;
    L.s2 = s2;
    L.y = y;
    L.workspace = static_cast<uint8_t *>(workspace);
    L.flags = flags;
    L.stream = static_cast<cudaStream_t>(stream);
    L.timeout_ns = kDefaultTimeoutNs;
    fp8bs_status st = check_layer(L);
    if (st == FP8BS_OK)
        st = set_scores(L, wr, wr_type, bias, scoring, groups, top_groups, group_best, renormalize, scale);
    return st != FP8BS_OK ? st : run_experts(L, workspace_bytes);
}

// Test hook (declared in include/fp8bs_testing.h).
fp8bs_status fp8bs_testhook_moe_stall(const void *x, int ldx, const int32_t *ids, const float *weights,
                                      const uint8_t *w13, const float *s13, const uint8_t *w2, const float *s2,
                                      void *y, int M, int H, int I, int E, int top_k, void *workspace,
                                      size_t workspace_bytes, unsigned flags, int phase, int skip_unit,
                                      unsigned long long timeout_ns, void *stream)
{
    if (!ids || !weights || phase < 0 || phase > 1 || skip_unit < 0 || timeout_ns == 0 ||
        timeout_ns > 10ull * kDefaultTimeoutNs)
        return FP8BS_ERR_INVALID_ARG;
    MoeLaunch L = {};
    L.M = M;
    L.H = H;
    L.I = I;
    L.E = E;
    L.top_k = top_k;
    L.x = x;
    L.ldx = ldx;
    L.ids = const_cast<int32_t *>(ids);
    L.topw = const_cast<float *>(weights);
    L.w13 = w13;
    L.s13 = s13;
    L.w2 = w2;
    L.s2 = s2;
    L.y = y;
    L.workspace = static_cast<uint8_t *>(workspace);
    L.flags = flags;
    L.stream = static_cast<cudaStream_t>(stream);
    L.timeout_ns = timeout_ns;
    L.test_skip_unit = skip_unit;
    L.test_skip_phase = phase;
    fp8bs_status st = check_layer(L);
    return st != FP8BS_OK ? st : run_experts(L, workspace_bytes);
}

} // extern "C"
