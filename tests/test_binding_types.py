"""The binding of the expert and 4-bit layers names an argument that is no
tensor in a TypeError, as the other entry points do."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb

NO_TENSORS = [[[1.0, 2.0]], np.zeros((2, 128), np.float32), None, 3, "x"]


@pytest.mark.parametrize("bad", NO_TENSORS)
def test_the_first_argument(bad):
    for call, name in ((lambda: fb.fp4_quant_weights(bad), "w"), (lambda: fb.fp4_quant_act(bad), "x"),
                       (lambda: fb.fp4_gemm_fused(bad, None, None, None, 128), "x"),
                       (lambda: fb.fp4_gemm(bad, None, None, None, None, None, 128, 128), "aq"),
                       (lambda: fb.fp4_dequant_weights(bad, None, None, 128, 128), "wq"),
                       (lambda: fb.moe_route(bad, None, 1), "x"),
                       (lambda: fb.fp8_moe_layer(bad, None, 1, None, None, None, None), "x"),
                       (lambda: fb.fp8_moe_experts(bad, None, None, None, None, None, None), "x")):
        with pytest.raises(TypeError, match="^%s must be" % name):
            call()


def test_a_tensor_on_the_cpu_is_refused_as_such():
    for call in (lambda: fb.fp4_quant_weights(torch.zeros(128, 128)),
                 lambda: fb.fp4_quant_act(torch.zeros(2, 128, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", NO_TENSORS)
def test_every_other_argument(bad):
    H, I, E, k = 256, 128, 4, 2
    x = torch.zeros((2, H), dtype=torch.bfloat16, device="cuda")
    wr = torch.zeros((E, H), device="cuda")
    w13 = fb.fp8_quant_weight_blocks(torch.zeros((E * 2 * I, H), device="cuda"), tiled=True)
    w2 = fb.fp8_quant_weight_blocks(torch.zeros((E * H, I), device="cuda"), tiled=True)
    ids = torch.zeros((2, k), dtype=torch.int32, device="cuda")
    packed = dict(zip(("wq", "ws_atoms", "w_rows"), fb.fp4_quant_weights(torch.zeros((128, H), device="cuda"))))
    act = dict(zip(("aq", "as_atoms", "a_rows"), fb.fp4_quant_act(x)))
    experts = dict(w13=w13[0], s13=w13[1], w2=w2[0], s2=w2[1])
    calls = [(fb.fp8_moe_layer, dict(x=x, wr=wr, top_k=k, **experts), ["y", "ids", "weights", "workspace"]),
             (fb.fp8_moe_experts, dict(x=x, ids=ids, weights=ids.float(), experts=E, **experts), ["y", "workspace"]),
             (fb.moe_route, dict(x=x, wr=wr, top_k=k), ["ids", "weights", "workspace"]),
             (fb.fp4_gemm_fused, dict(x=x, n=128, **packed), ["y", "workspace"]),
             (fb.fp4_gemm, dict(n=128, k=H, **act, **packed), ["y", "workspace"]),
             (fb.fp4_dequant_weights, dict(n=128, k=H, **packed), ["w"]),
             (fb.fp4_quant_act, dict(x=x), ["xq", "xs_atoms", "x_rows"]),
             (fb.fp4_quant_weights, dict(w=wr), ["wq", "ws_atoms", "w_rows"])]
    for fn, good, optional in calls:
        fn(**good)
        for name in [n for n in good if n not in ("n", "k", "top_k", "experts")] + optional:
            if bad is None and (name in optional or name in ("a_rows", "w_rows")):
                continue  # may be left out
            with pytest.raises(TypeError, match="^%s must be" % name):
                fn(**{**good, name: bad})
