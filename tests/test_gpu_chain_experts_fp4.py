"""Chains in which each layer reads what the one before wrote, with
FLAG_OVERLAP_PREV throughout and one shared workspace: 4-bit layers, expert
layers, and both among the FP8 and MX layers.  A kernel that read its input, the
choice of the experts or the workspace before the previous kernel's writes would
see the previous pass's, which had another input.  Every output must be bitwise
that of the same calls one at a time, each waited for, with workspaces of their
own and no flag.
"""
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb

pytestmark = pytest.mark.gpu


class Weights:
    """Random weights of scale 1/sqrt(K), so that a chain's values stay near 1."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def __call__(self, rows, K):
        return torch.randn((rows, K), generator=self.gen, device="cuda") * K ** -0.5

    def fp4(self, rows, K, fmt):
        q = fb.fp4_quant_weights(self(rows, K), fmt)
        return lambda x, **kw: (fb.fp4_gemm_fused(x, *q, rows, fmt, **kw),)

    def fp4_two_calls(self, rows, K, fmt):
        q = fb.fp4_quant_weights(self(rows, K), fmt)

        def call(x, workspace=None, flags=0):
            return (fb.fp4_gemm(*fb.fp4_quant_act(x, fmt, flags=flags), *q, rows, K, fmt, workspace=workspace, flags=flags),)
        return call

    def fp8(self, rows, K):
        q = fb.fp8_quant_weight_blocks(self(rows, K), tiled=True)
        return lambda x, **kw: (fb.fp8_blockscaled_gemm_fused(x, *q, n=rows, **kw),)

    def mx(self, rows, K):
        q = fb.fp8_mx_quant_weights(self(rows, K))

        def call(x, workspace=None, flags=0):
            return (fb.fp8_mx_gemm(*fb.fp8_mx_quant_act(x, flags=flags), *q, rows, workspace=workspace, flags=flags),)
        return call

    def _experts(self, E, H, I):
        return (*fb.fp8_quant_weight_blocks(self(E * 2 * I, H) * 2, tiled=True),
                *fb.fp8_quant_weight_blocks(self(E * H, I) * 4, tiled=True))

    def layer(self, E, k, H, I):
        q, wr = self._experts(E, H, I), self(E, H) * 2
        return lambda x, **kw: fb.fp8_moe_layer(x, wr, k, *q, **kw)

    def route_and_experts(self, E, k, H, I):
        q, wr = self._experts(E, H, I), self(E, H) * 2

        def call(x, **kw):
            ids, w = fb.moe_route(x, wr, k, **kw)
            return fb.fp8_moe_experts(x, ids, w, *q, experts=E, **kw), ids, w
        return call


H = 1024


def _fp4_chain(seed):
    w = Weights(seed)
    return [w.fp4(2048, H, fb.FP4_NV), w.fp4(640, 2048, fb.FP4_MX), w.fp4_two_calls(5120, 640, fb.FP4_NV),
            w.fp4_two_calls(H, 5120, fb.FP4_MX), w.fp4(H, H, fb.FP4_NV)]


def _expert_chain(seed):
    w = Weights(seed)
    return [w.layer(16, 2, H, 256), w.layer(60, 6, H, 128), w.route_and_experts(24, 3, H, 384), w.layer(8, 1, H, 128)]


def _mixed_chain(seed):
    w = Weights(seed)
    return [w.fp8(H, H), w.fp4(2048, H, fb.FP4_NV), w.fp4(H, 2048, fb.FP4_MX), w.layer(32, 4, H, 256), w.mx(H, H),
            w.route_and_experts(16, 2, H, 256), w.fp8(2560, H), w.fp4(H, 2560, fb.FP4_NV), w.layer(12, 2, H, 128),
            w.fp8(H, H)]


CHAINS = [(_fp4_chain, M) for M in (1, 8, 33, 130, 512)] + \
         [(c, M) for c in (_expert_chain, _mixed_chain) for M in (1, 8, 20, 50)]


def _apart(chain, x):
    """Every layer's outputs, one call at a time."""
    out = []
    for call in chain:
        torch.cuda.synchronize()
        out.append(call(x))
        x = out[-1][0]
    torch.cuda.synchronize()
    assert not x.isnan().any()
    return out


def _inputs(M, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    return [torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(n)]


def _same(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        for s, t in zip(a, b):
            assert torch.equal(s.view(torch.int16), t.view(torch.int16)), "layer %d" % i


@pytest.mark.parametrize("make,M", CHAINS)
def test_chained_layers(make, M):
    chain, xs = make(7), _inputs(M, 4)
    want = [_apart(chain, x) for x in xs]
    work = fb.make_workspace(64 << 20)

    def run(x):
        out = []
        for call in chain:
            out.append(call(x, workspace=work, flags=fb.FLAG_OVERLAP_PREV))
            x = out[-1][0]
        return out
    for _ in range(2):                                             # eagerly, without a wait between the passes
        got = [run(x) for x in xs]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            _same(g, w)
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                                  # the same buffers, with another input each time
        out = run(x)
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        _same(out, want[i])
    assert fb.workspace_status(work) == 0
