"""The operators between a step's layers with the layers, as a speculative-
verify step runs them: norm and cast -> FP8 projection -> norm -> scored expert
layer -> norm and MX cast -> MX layer -> norm -> output layer -> verification of
the drafts, in one chain under FLAG_OVERLAP_PREV with one shared workspace, eager
and as a replayed graph.  A kernel that read its input or the workspace before the
previous kernel's writes would see the last pass's, which had another input.
Every output must be bitwise that of the same calls one at a time, each waited
for, with workspaces of their own and no flag.
"""
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb

pytestmark = pytest.mark.gpu

H, V, E, I, K_TOP = 1024, 5000, 32, 256, 4


class Step:
    def __init__(self, B, L, seed):
        self.B, self.L, self.M = B, L, B * (L + 1)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(rows, K, scale=1.0):
            return torch.randn((rows, K), generator=g, device="cuda") * scale * K ** -0.5
        self.proj = fb.fp8_quant_weight_blocks(w(H, H), tiled=True)
        self.mx = fb.fp8_mx_quant_weights(w(H, H))
        self.out = fb.fp8_quant_weight_blocks(w(V, H, 3.0), tiled=True)
        self.router, self.bias = w(E, H, 2.0), torch.randn(E, generator=g, device="cuda") * 0.05
        self.experts = (*fb.fp8_quant_weight_blocks(w(E * 2 * I, H, 2.0), tiled=True),
                        *fb.fp8_quant_weight_blocks(w(E * H, I, 4.0), tiled=True))
        self.gammas = [torch.rand(H, generator=g, device="cuda") + 0.5 for _ in range(4)]
        self.gen = g

    def inputs(self):
        """Another pass's embedding rows, drafts and random numbers."""
        def r(*shape):
            return torch.rand(shape, generator=self.gen, device="cuda")
        q = torch.softmax(torch.randn((self.B * self.L, V), generator=self.gen, device="cuda") * 3.0, dim=1)
        draft = torch.multinomial(q, 1, generator=self.gen).view(self.B, self.L).to(torch.int32)
        return dict(x=torch.randn((self.M, H), generator=self.gen, device="cuda").to(torch.bfloat16), q=q, draft=draft,
                    accept_u=r(self.B, self.L) * 0.02, sample_u=r(self.B), temperature=r(self.B) + 0.5)

    def sizes(self):
        M = self.M
        return [fb.fp8_blockscaled_gemm_workspace_size(M, H, H), fb.fp8_moe_workspace_size(M, H, I, E, K_TOP),
                fb.fp8_mx_gemm_workspace_size(M, H, H), fb.fp8_blockscaled_gemm_workspace_size(M, V, H),
                fb.speculative_verify_workspace_size(self.B, self.L, V)]

    def run(self, t, work, flags=0, wait=lambda: None):
        """All outputs; work: one workspace for all, or None for new ones."""
        kept = []

        def keep(*out):
            wait()
            kept.extend(o for o in out if o is not None)
            return out
        a, s, h, _ = keep(*fb.fp8_rmsnorm_quant_act(t["x"], self.gammas[0], residual=t["x"], flags=flags))
        y, = keep(fb.fp8_blockscaled_gemm(a, s, *self.proj, workspace=work, flags=flags, n=H))
        _, _, h, n = keep(*fb.fp8_rmsnorm_quant_act(y, self.gammas[1], residual=h, store_y=True, flags=flags))
        y, _, _ = keep(*fb.fp8_moe_layer_grouped(n, self.router, K_TOP, *self.experts, bias=self.bias, groups=8, top_groups=3,
                                                 scale=1.5, workspace=work, flags=flags))
        keep(*fb.moe_route_grouped(n, self.router, K_TOP, scoring=fb.SCORE_SOFTMAX, groups=4, top_groups=2, group_best=1,
                                   workspace=work, flags=flags))
        a, s, h, _ = keep(*fb.fp8_mx_rmsnorm_quant_act(y, self.gammas[2], residual=h, flags=flags))
        y, = keep(fb.fp8_mx_gemm(a, s, *self.mx, H, workspace=work, flags=flags))
        a, s, h, _ = keep(*fb.fp8_rmsnorm_quant_act(y, self.gammas[3], residual=h, residual_out=h, flags=flags))
        logits, = keep(fb.fp8_blockscaled_gemm(a, s, *self.out, workspace=work, flags=flags, n=V))
        keep(*fb.speculative_verify(logits, t["sample_u"], draft=t["draft"], accept_u=t["accept_u"], draft_probs=t["q"],
                                    temperature=t["temperature"], workspace=work, flags=flags))
        keep(*fb.speculative_verify(logits[:self.B], t["sample_u"], workspace=work, flags=flags))
        return kept


def _same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("B,L", [(1, 1), (1, 7), (8, 7), (12, 2)])
def test_a_step_overlapped_and_replayed_gives_the_bits_of_single_calls(B, L):
    step = Step(B, L, seed=B * 10 + L)
    passes = [step.inputs() for _ in range(4)]
    want = [step.run(t, None, wait=torch.cuda.synchronize) for t in passes]
    assert not all(torch.equal(a, b) for a, b in zip(want[0], want[1]))
    work = fb.make_workspace(max(step.sizes()))
    for _ in range(3):
        got = [step.run(t, work, flags=fb.FLAG_OVERLAP_PREV) for t in passes]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            _same(g, w)
    t = {k: v.clone() for k, v in passes[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run(t, work, flags=fb.FLAG_OVERLAP_PREV)
    for p, w in zip(passes + passes[:1], want + want[:1]):
        for k in t:
            t[k].copy_(p[k])
        graph.replay()
        torch.cuda.synchronize()
        _same(out, w)
    assert fb.workspace_status(work) == 0 and not work[:1024 + 65536].any()


def test_two_streams_at_once_with_workspaces_of_their_own():
    steps = [Step(4, 3, seed=1), Step(8, 7, seed=2)]
    inputs = [s.inputs() for s in steps]
    want = [s.run(t, None, wait=torch.cuda.synchronize) for s, t in zip(steps, inputs)]
    works = [fb.make_workspace(max(s.sizes())) for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, (s, t) in enumerate(zip(steps, inputs)):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.run(t, works[i], flags=fb.FLAG_OVERLAP_PREV))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            _same(one, w)


def test_the_output_layers_logits_are_what_the_verification_reads():
    """At temperature 0 the drafts are accepted as far as they are the greedy
    choice of the same layer, and the next token is that choice."""
    B, L = 6, 3
    step = Step(B, L, seed=9)
    t = step.inputs()
    token, _, logits = fb.fp8_blockscaled_gemm_fused_greedy(t["x"], *step.out, n=V)
    greedy = token.view(B, L + 1)
    draft = greedy[:, :L].contiguous()
    draft[1, 0] += 1
    draft[2, 2] -= 1
    got, accepted, probs = fb.speculative_verify(logits, t["sample_u"], draft=draft, accept_u=t["accept_u"],
                                                 temperature=torch.zeros(B, device="cuda"))
    n = [L, 0, 2] + [L] * (B - 3)
    assert accepted.tolist() == n
    for b in range(B):
        assert torch.equal(got[b, :n[b] + 1], greedy[b, :n[b] + 1]) and (got[b, n[b] + 1:] == -1).all()
        assert (probs[b, :n[b] + 1] == 1).all() and (probs[b, n[b] + 1:] == 0).all()
