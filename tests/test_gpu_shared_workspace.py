"""One workspace for calls of different shapes and entry points, as a decode
step's layers share it: what has to be zero between calls (status word, greedy
keys, routing words, arrival counters) lies where no call keeps its data.

More than 16,384 tiles: the counters past those lie where smaller shapes keep
data, and the call zeroes them.

The order matters: a call with few tiles first, whose split-K partials are
written, then one with many, whose counters reach further.
"""
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from fp8_block_scaled_token_gb300 import synth

pytestmark = pytest.mark.gpu

K = 1280


def _fp8(M, N, seed, kind):
    x = synth.activations(M, K, seed=seed, device="cuda")
    w = synth.weights(N, K, seed=seed + 50, device="cuda")
    if kind == "bf16":
        wb = w.to(torch.bfloat16)
        return fb.bf16_gemm_ref_workspace_size(M, N, K), lambda work: (fb.bf16_gemm_ref(x, wb, workspace=work),)
    if kind == "mx":
        a, q = fb.fp8_mx_quant_act(x), fb.fp8_mx_quant_weights(w)
        return fb.fp8_mx_gemm_workspace_size(M, N, K), lambda work: (fb.fp8_mx_gemm(*a, *q, N, workspace=work),)
    if kind == "fp4":
        q = fb.fp4_quant_weights(w)
        return fb.fp4_gemm_workspace_size(M, N, K), lambda work: (fb.fp4_gemm_fused(x, *q, N, workspace=work),)
    q = fb.fp8_quant_weight_blocks(w, tiled=True)
    size = fb.fp8_blockscaled_gemm_workspace_size(M, N, K)
    if kind == "greedy":
        return size, lambda work: fb.fp8_blockscaled_gemm_fused_greedy(x, *q, workspace=work, n=N)
    return size, lambda work: (fb.fp8_blockscaled_gemm_fused(x, *q, workspace=work, n=N),)


def _moe(M, E, k, H, I, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def w(*shape):
        return torch.randn(shape, generator=g, device="cuda") * 0.05
    x, wr = w(M, H).to(torch.bfloat16), w(E, H)
    q = (*fb.fp8_quant_weight_blocks(w(E * 2 * I, H), tiled=True), *fb.fp8_quant_weight_blocks(w(E * H, I), tiled=True))
    return fb.fp8_moe_workspace_size(M, H, I, E, k), lambda work: fb.fp8_moe_layer(x, wr, k, *q, workspace=work)


def _check(calls):
    alone = [call(fb.make_workspace(size)) for size, call in calls]
    work = fb.make_workspace(max(size for size, _ in calls))
    for _ in range(2):
        for (_, call), want in zip(calls, alone):
            for a, b in zip(call(work), want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert fb.workspace_status(work) == 0
    assert not work[:1024 + 65536].any(), "status, greedy keys, routing words and counters back at zero"


@pytest.mark.parametrize("kind", ["fp8", "greedy", "mx", "bf16", "fp4"])
def test_shapes_of_one_entry_point(kind):
    """10 tiles, then 68 and 272, whose counters go past the first's."""
    _check([_fp8(8, 1280, 1, kind), _fp8(8, 8704, 2, kind), _fp8(1, 640, 3, kind), _fp8(40, 34816, 4, kind)])


def test_expert_layers_of_different_sizes():
    _check([_moe(2, 4, 2, 256, 128, 1), _moe(16, 64, 6, 512, 256, 2), _moe(64, 32, 4, 256, 384, 3)])


def test_all_entry_points():
    _check([_fp8(8, 1280, 1, "fp8"), _moe(5, 40, 3, 512, 256, 2), _fp8(8, 8704, 3, "greedy"), _fp8(8, 8704, 4, "fp4"),
            _moe(30, 16, 4, 1280, 128, 5), _fp8(8, 8704, 6, "mx"), _fp8(4, 1280, 7, "greedy"), _fp8(8, 8704, 8, "bf16")])


def test_routing_alone_shares_too():
    x = synth.activations(20, 512, seed=1, device="cuda")
    wr = synth.weights(100, 512, seed=2, device="cuda")
    _check([(fb.moe_route_workspace_size(20, 100), lambda work: fb.moe_route(x, wr, 4, workspace=work)),
            _fp8(8, 8704, 3, "fp8"), _moe(5, 40, 3, 512, 256, 2)])


FAR = 20000 * 128  # rows: 20,000 tiles, two or four K blocks each, so that CTAs share tiles past 16,384


def _far(kind):
    x = synth.activations(8, 512 if kind == "fp4" else 256, seed=5, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    w = torch.randn((FAR, x.shape[1]), generator=g, device="cuda", dtype=torch.bfloat16)
    if kind == "fp4":
        q = fb.fp4_quant_weights(w)
        return fb.fp4_gemm_workspace_size(8, FAR, 512), lambda work, y: fb.fp4_gemm_fused(x, *q, FAR, y=y, workspace=work)
    if kind == "mx":
        a, q = fb.fp8_mx_quant_act(x), fb.fp8_mx_quant_weights(w)
        return fb.fp8_mx_gemm_workspace_size(8, FAR, 256), lambda work, y: fb.fp8_mx_gemm(*a, *q, FAR, y=y, workspace=work)
    if kind == "bf16":
        return fb.bf16_gemm_ref_workspace_size(8, FAR, 256), lambda work, y: fb.bf16_gemm_ref(x, w, y=y, workspace=work)
    q = fb.fp8_quant_weight_blocks(w, tiled=True)
    return (fb.fp8_blockscaled_gemm_workspace_size(8, FAR, 256),
            lambda work, y: fb.fp8_blockscaled_gemm_fused(x, *q, y=y, workspace=work, n=FAR))


def _check_far(size, call, small):
    want = call(fb.make_workspace(size), None)
    work = fb.make_workspace(max(size, small[0]))
    small_want = [t.clone() for t in small[1](work)]
    for _ in range(2):
        work[1024 + 65536:] = 0xA5                                 # what a small shape's data may hold
        y = torch.full_like(want, float("nan"))
        call(work, y)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        for a, b in zip(small[1](work), small_want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert fb.workspace_status(work) == 0 and not work[:1024 + 65536].any()


@pytest.mark.parametrize("kind", ["fp8", "mx", "bf16", "fp4"])
def test_more_tiles_than_the_shared_counters(kind):
    size, call = _far(kind)
    _check_far(size, call, _fp8(8, 1280, 1, "fp8"))


def test_more_expert_tiles_than_the_shared_counters():
    """64 tokens that name every one of 512 experts, 40 tiles of I each."""
    M, E, k, H, I = 64, 512, 8, 256, 5120
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    q = []
    for rows, K in ((E * 2 * I, H), (E * H, I)):
        q += fb.fp8_quant_weight_blocks(torch.randn((rows, K), generator=g, device="cuda", dtype=torch.bfloat16), tiled=True)
    ids = torch.randperm(E, generator=g, device="cuda").to(torch.int32).view(M, k)
    w = torch.rand((M, k), generator=g, device="cuda")
    _check_far(fb.fp8_moe_workspace_size(M, H, I, E, k),
               lambda work, y: fb.fp8_moe_experts(x, ids, w, *q, experts=E, y=y, workspace=work), _fp8(8, 1280, 1, "fp8"))
