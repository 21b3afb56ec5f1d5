"""A decode step's tail on one GPU, from its public calls: a 4-bit projection
with a residual, an expert layer with a residual, and the FP8 output layer with
the greedy choice of the next token.

    python examples/expert_block.py [--tokens 8] [--hidden 2048] [--experts 64] [--top-k 6]
                                    [--inter 768] [--vocab 32768] [--blocks 4] [--steps 20]

Weights are random, quantised once by the library; the workspaces are made
once; the step is captured in a CUDA graph and replayed, so what is timed is
the GPU's work.  Prints the time of a step and the bytes of weights it read.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_token_gb300 as fb  # noqa: E402


class Block:
    """One block's packed weights and workspaces."""

    def __init__(self, tokens, hidden, inter, experts, top_k, gen):
        def w(*shape):
            return torch.randn(shape, generator=gen, device="cuda") * 0.02
        self.tokens, self.hidden, self.top_k = tokens, hidden, top_k
        self.proj = fb.fp4_quant_weights(w(hidden, hidden))
        self.router = w(experts, hidden)
        self.w13 = fb.fp8_quant_weight_blocks(w(experts * 2 * inter, hidden), tiled=True)
        self.w2 = fb.fp8_quant_weight_blocks(w(experts * hidden, inter), tiled=True)
        self.proj_work = fb.make_workspace(fb.fp4_gemm_workspace_size(tokens, hidden, hidden))
        self.moe_work = fb.make_workspace(fb.fp8_moe_workspace_size(tokens, hidden, inter, experts, top_k))

    def __call__(self, x):
        """(x after the projection and the expert layer, the experts chosen)."""
        x = x + fb.fp4_gemm_fused(x, *self.proj, self.hidden, workspace=self.proj_work)
        y, ids, _ = fb.fp8_moe_layer(x, self.router, self.top_k, *self.w13, *self.w2, workspace=self.moe_work)
        return x + y, ids


class Tail:
    """Some blocks and the output layer."""

    def __init__(self, tokens, hidden, inter, experts, top_k, vocab, blocks, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.blocks = [Block(tokens, hidden, inter, experts, top_k, gen) for _ in range(blocks)]
        self.vocab = vocab
        self.out = fb.fp8_quant_weight_blocks(torch.randn((vocab, hidden), generator=gen, device="cuda") * 0.02, tiled=True)
        self.out_work = fb.make_workspace(fb.fp8_blockscaled_gemm_workspace_size(tokens, vocab, hidden))

    def step(self, x):
        """(next token of each row, the experts chosen in each block)."""
        chosen = []
        for block in self.blocks:
            x, ids = block(x)
            chosen.append(ids)
        token, _, _ = fb.fp8_blockscaled_gemm_fused_greedy(x, *self.out, store_y=False, workspace=self.out_work, n=self.vocab)
        return token, chosen

    def check(self):
        """Raises if a kernel of any layer gave up waiting."""
        for work in [self.out_work] + [w for b in self.blocks for w in (b.proj_work, b.moe_work)]:
            if fb.workspace_status(work):
                raise RuntimeError("a kernel reported a time-out")


def weight_bytes(tail, chosen):
    """Bytes of weights one step reads: of the experts, only the chosen ones."""
    total = sum(t.numel() * t.element_size() for t in tail.out)
    for block, ids in zip(tail.blocks, chosen):
        share = len(torch.unique(ids)) / block.router.shape[0]
        total += sum(t.numel() * t.element_size() for t in block.proj)
        total += block.router.numel() * 4
        total += share * sum(t.numel() * t.element_size() for t in (*block.w13, *block.w2))
    return total


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 8), ("hidden", 2048), ("experts", 64), ("top-k", 6), ("inter", 768),
                        ("vocab", 32768), ("blocks", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    tail = Tail(a.tokens, a.hidden, a.inter, a.experts, a.top_k, a.vocab, a.blocks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=gen, device="cuda").to(torch.bfloat16)
    token, chosen = tail.step(x)  # also the first call of everything, before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_token, _ = tail.step(x)
    for _ in range(3):
        graph.replay()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    tail.check()
    assert torch.equal(graph_token, token), "the replayed step chose other tokens"
    ms = start.elapsed_time(end) / a.steps
    read = weight_bytes(tail, chosen)
    print("%d blocks, %d tokens: %.1f us a step, %.0f MB of weights read, %.2f TB/s" % (
        a.blocks, a.tokens, ms * 1e3, read / 1e6, read / ms / 1e9))
    print("tokens:", token.tolist())
    return token, chosen


if __name__ == "__main__":
    main()
