"""The expert-block example runs, and its step agrees with the same layers put
together from other calls of the library: the choice and the experts apart, the
4-bit cast and product apart, and the output layer's greedy choice from stored
logits."""
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from examples import expert_block

pytestmark = pytest.mark.gpu


def test_step_agrees_with_the_layers_apart():
    tokens, hidden, inter, experts, top_k, vocab = 5, 512, 256, 12, 3, 1000
    tail = expert_block.Tail(tokens, hidden, inter, experts, top_k, vocab, blocks=2, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16)
    token, chosen = tail.step(x)
    tail.check()
    for block, ids in zip(tail.blocks, chosen):
        a = fb.fp4_quant_act(x)
        x = x + fb.fp4_gemm(*a, *block.proj, hidden, hidden)
        ids2, w = fb.moe_route(x, block.router, top_k)
        assert torch.equal(ids2, ids)
        x = x + fb.fp8_moe_experts(x, ids2, w, *block.w13, *block.w2, experts=experts)
    y = fb.fp8_blockscaled_gemm_fused(x, *tail.out, n=vocab)
    assert torch.equal(token.long(), y.float().argmax(dim=1))


def test_main_runs(capsys):
    token, chosen = expert_block.main(["--tokens", "3", "--hidden", "256", "--inter", "128", "--experts", "8", "--top-k",
                                       "2", "--vocab", "512", "--blocks", "2", "--steps", "3"])
    assert token.shape == (3,) and len(chosen) == 2
    assert "MB of weights read" in capsys.readouterr().out
