"""The expert layer and the 4-bit layer of a decode step: cases, plain forms
and 64-bit values, for measuring the library's kernels.

``run`` computes an operator in its plain form (elementary torch operations
in fp32, rounded once at the end) or, where ``own`` is true, through the
public entry points of fp8_block_scaled_token_gb300.  ``exact`` gives the
same outputs from the definitions in 64 bits, written apart from the plain
form.  Three operators:

* ``moe``: router product, top-k choice, experts' gate/up product, SwiGLU,
  re-quantisation, down product and weighted sum, for up to 64 tokens, with
  E4M3 weights in 128x128 blocks (the tiled layout).
* ``fp4``: a linear layer with microscaled 4-bit weights and activations
  (the cast of the activations, then the product), up to 512 tokens.
* ``fp4_quant``: weights to microscaled 4 bits, and the values they stand for.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases
_LISTED = [
    # smallest expert layer: one token, few small experts; latency only
    dict(name="moe_m1_small", op="moe", M=1, E=8, k=2, H=512, I=256, wr="bf16", renorm=True),
    # one decoding sequence through many fine-grained experts
    dict(name="moe_m1_e128", op="moe", M=1, E=128, k=8, H=2048, I=768, wr="bf16", renorm=True),
    # a speculative-verify batch of 8 rows at the repository's hidden size
    dict(name="moe_m8_h5120", op="moe", M=8, E=64, k=4, H=5120, I=1280, wr="bf16", renorm=True),
    # odd numbers of tokens, experts and blocks; fp32 router; weights over all experts
    dict(name="moe_m13_odd", op="moe", M=13, E=43, k=3, H=1408, I=640, wr="f32", renorm=False),
    # the largest batch: every expert is read
    dict(name="moe_m64_h5120", op="moe", M=64, E=64, k=6, H=5120, I=1408, wr="bf16", renorm=True),
    # smallest 4-bit layer: one token
    dict(name="fp4_m1_small", op="fp4", fmt="nv", M=1, N=640, K=512),
    # the square attention projection of a decode step
    dict(name="fp4_m8_square", op="fp4", fmt="nv", M=8, N=5120, K=5120),
    # the MLP up projection, 16 rows
    dict(name="fp4_m16_mlp_up", op="fp4", fmt="nv", M=16, N=34816, K=5120),
    # ragged rows and a K that ends inside a 256-wide block, power-of-two scales
    dict(name="fp4_mx_m37_ragged", op="fp4", fmt="mx", M=37, N=5003, K=17376),
    # chunked prefill: compute-bound
    dict(name="fp4_m512_mlp_up", op="fp4", fmt="nv", M=512, N=34816, K=5120),
    # weights of one MLP down projection to 4 bits and back
    dict(name="fp4_quant_mlp_down", op="fp4_quant", fmt="nv", N=5120, K=17408, w="bf16"),
    # a small ragged fp32 weight, power-of-two scales
    dict(name="fp4_quant_mx_ragged", op="fp4_quant", fmt="mx", N=1000, K=2080, w="f32"),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm (never 3072)."""
    while True:
        v = max(1, _log_int(rng, lo / step, hi / step)) * step
        if v != 3072 and 2 * v != 3072:
            return v


def draw(rng):
    op = rng.choice(["moe", "fp4", "fp4", "fp4_quant"])
    if op == "moe":
        while True:
            c = dict(op=op, M=_log_int(rng, 1, 64), E=_log_int(rng, 4, 160), H=_blocks(rng, 256, 5120, 128),
                     I=_blocks(rng, 128, 2048, 128), wr=rng.choice(["bf16", "f32"]), renorm=rng.random() < 0.5)
            c["k"] = min(c["E"], rng.randint(1, 8))
            if c["E"] * c["H"] * c["I"] <= 64 * 5120 * 1408:  # the largest listed layer's weights
                return c
    fmt = rng.choice(["nv", "mx"])
    while True:
        n = _log_int(rng, 64, 34816)
        k = _blocks(rng, 128, 17408, 32)
        if n == 3072 or n * k > 34816 * 5120:
            continue
        if op == "fp4":
            return dict(op=op, fmt=fmt, M=_log_int(rng, 1, 512), N=n, K=k)
        if n * k <= 5120 * 17408:
            return dict(op=op, fmt=fmt, N=n, K=k, w=rng.choice(["bf16", "f32"]))


def work(case):
    if case["op"] == "moe":
        M, E, k, H, I = (case[n] for n in ("M", "E", "k", "H", "I"))
        active = E * (1.0 - (1.0 - k / E) ** M)  # experts that some token chose, in the mean
        wr = 4 if case["wr"] == "f32" else 2
        return {"bytes": active * 3 * I * H * (1 + 4 / 16384) + E * H * wr + 4 * M * H + 8 * M * k,
                "flops": 2.0 * M * k * 3 * I * H + 2.0 * M * E * H}
    N, K = case["N"], case["K"]
    packed = N * K / 2 + N * K / (16 if case["fmt"] == "nv" else 32)
    if case["op"] == "fp4":
        M = case["M"]
        return {"bytes": packed + 2.0 * M * K + 2.0 * M * N, "flops": 2.0 * M * N * K}
    # the weights read, the packed form written and read, the values written
    return {"bytes": N * K * (4 if case["w"] == "f32" else 2) + 2 * packed + 4.0 * N * K, "flops": 2.0 * N * K}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, M, K):
    """bf16 N(0, 1) with one value in a thousand twenty times as large."""
    x = torch.randn((M, K), generator=g, device="cuda")
    big = torch.rand((M, K), generator=g, device="cuda") < 0.001
    return torch.where(big, x * 20.0, x).to(torch.bfloat16)


def _fp8_blocks(g, rows, K, std):
    """Codes in the tiled layout ([row tile * K block, 128, 128] uint8) and
    fp32 block scales of a random weight matrix, made tile by tile: N(0, std^2)
    values scaled so that each block's largest reaches 448."""
    tiles = (rows // 128) * (K // 128)
    codes = torch.empty((tiles, 128, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((tiles,), device="cuda")
    step = 16384
    for t in range(0, tiles, step):
        n = min(step, tiles - t)
        w = torch.randn((n, 128, 128), generator=g, device="cuda").mul_(std)
        s = w.abs().amax(dim=(1, 2)) / 448.0
        codes[t:t + n] = (w / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[t:t + n] = s
    return codes, scales.view(rows // 128, K // 128)




def _e2m1_codes(q):
    """4-bit codes (uint8) of the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to even, saturating."""
    a = q.abs()
    m = (a > 0.25).to(torch.uint8)
    m += a >= 0.75
    m += a > 1.25
    m += a >= 1.75
    m += a > 2.5
    m += a >= 3.5
    m += a > 5.0
    return m + 8 * ((q < 0) & (m > 0)).to(torch.uint8)


def _pow2(e):
    """2^e as fp32, exact, from int32 exponents in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 0x400000).to(torch.int32).view(torch.float32)


def _fp4_rows(v, fmt):
    """fp32 rows [R, K] (K a multiple of 32) -> codes uint8 [R, K], scale bytes
    uint8 [R, K/16 or K/32], row scales fp32 [R]: the definition in fp32."""
    R, K = v.shape
    if fmt == "nv":
        b = v.view(R, K // 16, 16)
        r = v.abs().amax(dim=1) / torch.full((), 2688.0, device=v.device)
        r = torch.where(r < 2.0 ** -126, torch.ones_like(r), r)
        s = (b.abs().amax(dim=2) / torch.full((), 6.0, device=v.device)) / r[:, None]
        s = s.clamp(max=448.0).to(torch.float8_e4m3fn)
        d = s.float() * r[:, None]
        q = torch.where(d[:, :, None] > 0, b / d[:, :, None], torch.zeros_like(b))
        return _e2m1_codes(q).view(R, K), s.view(torch.uint8), r
    b = v.view(R, K // 32, 32)
    am = b.abs().amax(dim=2)
    e = torch.where(am > 0, torch.frexp(am)[1] - 3, torch.zeros_like(am, dtype=torch.int32)).clamp(-127, 127)
    q = b * _pow2(-e)[:, :, None]
    return _e2m1_codes(q).view(R, K), (e + 127).to(torch.uint8), torch.ones((R,), device=v.device)


def _atom_order(rows_scales, per):
    """Scale bytes [rows, blocks] -> [row tiles * atoms, 512]: per 128 rows and
    `per` = 4 consecutive blocks, row r's block j at 16 (r % 32) + 4 (r / 32) + j."""
    R, B = rows_scales.shape
    rt, at = -(-R // 128), B // per
    p = torch.zeros((rt * 128, B), dtype=torch.uint8, device=rows_scales.device)
    p[:R] = rows_scales
    return p.view(rt, 4, 32, at, per).permute(0, 3, 2, 1, 4).reshape(rt * at, 512).contiguous()


def _pack_weights(v, fmt):
    """fp32 W [N, K] -> the packed operand: codes uint8 [row tiles * ceil(K/256), 128, 128]
    (two codes a byte, the lower k in the lower four bits), scale atoms, row scales [N]."""
    N, K = v.shape
    Kp = -(-K // 256) * 256
    codes = torch.zeros((-(-N // 128) * 128, Kp), dtype=torch.uint8, device=v.device)
    blk = 16 if fmt == "nv" else 32
    sb = torch.zeros((N, Kp // blk), dtype=torch.uint8, device=v.device)
    r = torch.empty((N,), device=v.device)
    for n in range(0, N, 4096):
        c, s, rr = _fp4_rows(v[n:n + 4096].float(), fmt)
        codes[n:n + c.shape[0], :K] = c
        sb[n:n + c.shape[0], :K // blk] = s
        r[n:n + c.shape[0]] = rr
    byts = codes[:, 0::2] | (codes[:, 1::2] << 4)
    rt, kt = byts.shape[0] // 128, Kp // 256
    tiles = byts.view(rt, 128, kt, 128).permute(0, 2, 1, 3).reshape(rt * kt, 128, 128).contiguous()
    return tiles, _atom_order(sb, 4), r


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "moe":
        M, E, H, I = (case[n] for n in ("M", "E", "H", "I"))
        wr = torch.randn((E, H), generator=g, device="cuda").mul_(1.5 / math.sqrt(H))
        w13, s13 = _fp8_blocks(g, E * 2 * I, H, 0.02)
        w2, s2 = _fp8_blocks(g, E * H, I, 0.02)
        return dict(case=dict(case), x=_activations(g, M, H), wr=wr if case["wr"] == "f32" else wr.to(torch.bfloat16),
                    w13=w13, s13=s13, w2=w2, s2=s2)
    N, K = case["N"], case["K"]
    w = torch.randn((N, K), generator=g, device="cuda").mul_(0.02)
    w *= torch.where(torch.rand((N, K), generator=g, device="cuda") < 0.01, 8.0, 1.0)
    if case["op"] == "fp4_quant":
        return dict(case=dict(case), w=w.to(torch.bfloat16) if case["w"] == "bf16" else w)
    wq, wa, wrow = _pack_weights(w, case["fmt"])
    return dict(case=dict(case), x=_activations(g, case["M"], K), wq=wq, wa=wa, wrow=wrow)


# ------------------------------------------------------------- plain forms
def _dequant_fp8(tiles, s):
    """Tiled codes and block scales -> fp32 [rows, K]."""
    rt, kt = s.shape
    v = tiles.view(torch.float8_e4m3fn).view(rt, kt, 128, 128).float() * s[:, :, None, None]
    return v.permute(0, 2, 1, 3).reshape(rt * 128, kt * 128)


def _fp8_cast(v):
    """Values after one fp32 scale per 128 consecutive values and the E4M3 rounding."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 128, 128)
    am = b.abs().amax(dim=-1, keepdim=True)
    s = torch.where(am > 0, am / torch.full((), 448.0, device=v.device), torch.ones_like(am))
    return ((b / s).to(torch.float8_e4m3fn).float() * s).reshape(v.shape)


def _plain_moe(st):
    c = st["case"]
    E, k, I = c["E"], c["k"], c["I"]
    x = st["x"].float()
    logits = x @ st["wr"].float().t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.exp(top - top[:, :1])
    w = w[:, :k] / (w[:, :k] if c["renorm"] else w).sum(dim=1, keepdim=True)
    ids = ids[:, :k]
    w13 = _dequant_fp8(st["w13"], st["s13"]).view(E, 2 * I, -1)
    gu = torch.matmul(_fp8_cast(x)[None], w13.transpose(1, 2))           # [E, M, 2I]
    del w13
    gate, up = gu[..., :I], gu[..., I:]
    h = _fp8_cast(gate / (1.0 + torch.exp(-gate)) * up)
    d = torch.matmul(h, _dequant_fp8(st["w2"], st["s2"]).view(E, -1, I).transpose(1, 2))  # [E, M, H]
    m = torch.arange(x.shape[0], device=x.device)
    y = (d[ids, m[:, None]] * w[:, :, None]).sum(dim=1)
    return dict(y=y.to(torch.bfloat16), ids=ids.to(torch.int32), weights=w)


def _e2m1_values(codes):
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                     device=codes.device)
    return t[codes.int()]


def _scale_values(sb, fmt):
    return sb.view(torch.float8_e4m3fn).float() if fmt == "nv" else _pow2(sb.int() - 127)


def _unpack(tiles, atoms, rows, N, K, fmt):
    """The packed weight operand -> fp32 [N, K]."""
    rt, kt = -(-N // 128), -(-K // 256)
    byts = tiles.view(rt, kt, 128, 128).permute(0, 2, 1, 3).reshape(rt * 128, kt * 128)
    v = _e2m1_values(torch.stack((byts & 15, byts >> 4), dim=2).view(rt * 128, kt * 256))
    at = atoms.shape[0] // rt
    sb = atoms.view(rt, at, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, at * 4)
    s = _scale_values(sb.contiguous(), fmt)[:N] * rows[:, None]
    return (v[:N].view(N, at * 4, -1) * s[:, :, None]).view(N, kt * 256)[:, :K]


def _fp4_values(v, fmt):
    """fp32 rows -> the values that their 4-bit form stands for."""
    codes, sb, r = _fp4_rows(v, fmt)
    s = _scale_values(sb, fmt) * r[:, None]
    return (_e2m1_values(codes).view(*s.shape, -1) * s[:, :, None]).view(v.shape)


def _plain(st):
    c = st["case"]
    if c["op"] == "moe":
        return _plain_moe(st)
    if c["op"] == "fp4_quant":
        return _fp4_values(st["w"].float(), c["fmt"])
    w = _unpack(st["wq"], st["wa"], st["wrow"], c["N"], c["K"], c["fmt"])
    return (_fp4_values(st["x"].float(), c["fmt"]) @ w.t()).to(torch.bfloat16)


# ------------------------------------------------------ the library's calls
def _own(st):
    import fp8_block_scaled_token_gb300 as fb
    c = st["case"]
    if c["op"] == "moe":
        if "work" not in st:
            st["work"] = fb.make_workspace(fb.fp8_moe_workspace_size(c["M"], c["H"], c["I"], c["E"], c["k"]))
        y, ids, w = fb.fp8_moe_layer(st["x"], st["wr"], c["k"], st["w13"], st["s13"], st["w2"], st["s2"],
                                     renormalize=c["renorm"], workspace=st["work"])
        return dict(y=y, ids=ids, weights=w)
    fmt = fb.FP4_NV if c["fmt"] == "nv" else fb.FP4_MX
    if c["op"] == "fp4_quant":
        wq, wa, wrow = fb.fp4_quant_weights(st["w"], fmt)
        return fb.fp4_dequant_weights(wq, wa, wrow, c["N"], c["K"], fmt)
    if "work" not in st:
        st["work"] = fb.make_workspace(fb.fp4_gemm_workspace_size(c["M"], c["N"], c["K"], fmt))
    return fb.fp4_gemm_fused(st["x"], st["wq"], st["wa"], st["wrow"], c["N"], fmt, workspace=st["work"])


def run(st):
    return _own(st) if own else _plain(st)


# ------------------------------------------------------------ 64-bit values
def _round_to(q, bits, emin, top):
    """float64 q to `bits` fraction bits, ties to even, least exponent emin, saturating at top."""
    a = q.abs()
    e = (torch.frexp(a)[1] - 1).clamp(min=emin)
    step = torch.exp2((e - bits).double())
    return torch.sign(q) * (torch.round(a / step) * step).clamp(max=top)


def _fl(v):
    """The fp32 roundings that the casts' definition names: a scale is an fp32
    number, and a code is that of the quotient rounded to fp32."""
    return v.float().double()


def _exact_fp8_cast(v):
    b = v.reshape(*v.shape[:-1], -1, 128)
    s = _fl(b.abs().amax(dim=-1, keepdim=True) / 448.0)
    s[s == 0] = 1.0
    return (_round_to(_fl(b / s), 3, -6, 448.0) * s).reshape(v.shape)


def _e4m3_numbers(device):
    """The values of the 256 codes, from the format's fields."""
    c = torch.arange(256, device=device)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (1.0 + f / 8.0) * torch.exp2((e - 7).double()))
    return torch.where(c >= 128, -v, v)


def _exact_expert(tiles, s, kt, e, rows):
    """float64 [rows, K] of expert e."""
    n = rows // 128
    t = _e4m3_numbers(tiles.device)[tiles[e * n * kt:(e + 1) * n * kt].int()]
    t = t.view(n, kt, 128, 128) * s[e * n:(e + 1) * n].double()[:, :, None, None]
    return t.permute(0, 2, 1, 3).reshape(rows, kt * 128)


def _exact_moe(st):
    c = st["case"]
    E, k, H, I = (c[n] for n in ("E", "k", "H", "I"))
    x = st["x"].double()
    logits = x @ st["wr"].double().t()
    top, ids = torch.topk(logits, k, dim=1)
    over = top if c["renorm"] else logits
    w = torch.exp(top - torch.logsumexp(over, dim=1, keepdim=True))
    a = _exact_fp8_cast(x)
    y = torch.zeros_like(x)
    for e in range(E):
        m, j = torch.nonzero(ids == e, as_tuple=True)
        if not m.numel():
            continue
        gu = a[m] @ _exact_expert(st["w13"], st["s13"], H // 128, e, 2 * I).t()
        h = _exact_fp8_cast(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        y.index_add_(0, m, (h @ _exact_expert(st["w2"], st["s2"], I // 128, e, H).t()) * w[m, j][:, None])
    return dict(y=y, ids=None, weights=w)


def _exact_fp4(v, fmt):
    """float64 rows -> the values that their 4-bit form stands for."""
    R, K = v.shape
    blk = 16 if fmt == "nv" else 32
    b = v.view(R, K // blk, blk)
    am = b.abs().amax(dim=2, keepdim=True)
    if fmt == "nv":
        r = _fl(v.abs().amax(dim=1) / 2688.0)[:, None, None]
        r = torch.where(r < 2.0 ** -126, torch.ones_like(r), r)
        s = _fl(_round_to(_fl(_fl(am / 6.0) / r), 3, -6, 448.0) * r)
    else:
        s = torch.where(am > 0, torch.exp2((torch.frexp(am)[1] - 3).double()), torch.ones_like(am))
    q = torch.where(s > 0, _fl(b / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(b))
    return (_round_to(q, 1, 0, 6.0) * s).view(R, K)


def _exact_packed(st, lo, hi):
    """float64 rows lo..hi of the packed weight operand (lo a multiple of 128)."""
    c = st["case"]
    kt = -(-c["K"] // 256)
    blk = 16 if c["fmt"] == "nv" else 32
    t0, t1 = lo // 128, -(-hi // 128)
    byts = st["wq"][t0 * kt:t1 * kt].view(-1, kt, 128, 128).transpose(1, 2).reshape(-1, kt * 128).int()
    code = torch.stack((byts % 16, byts // 16), dim=2).view(byts.shape[0], -1)
    mag = code % 8
    v = torch.where(mag < 2, mag * 0.5, (1.0 + (mag % 2) * 0.5) * torch.exp2((mag // 2 - 1).double()))
    v = torch.where(code >= 8, -v, v)[:, :c["K"]]
    r = torch.arange(v.shape[0], device=v.device)
    j = torch.arange(c["K"] // blk, device=v.device)
    per = st["wa"].shape[0] // (-(-c["N"] // 128))  # atoms of a row tile
    flat = st["wa"].view(-1).long()
    at = ((t0 + r[:, None] // 128) * per + j[None] // 4) * 512
    at = at + 16 * (r[:, None] % 32) + 4 * (r[:, None] % 128 // 32) + j[None] % 4
    sb = flat[at]
    s = _e4m3_numbers(v.device)[sb] if c["fmt"] == "nv" else torch.exp2((sb - 127).double())
    v = (v.view(v.shape[0], -1, blk) * s[:, :, None]).view(v.shape)[:hi - lo]
    return v * st["wrow"][lo:hi].double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "moe":
        return _exact_moe(st)
    if c["op"] == "fp4_quant":
        return torch.cat([_exact_fp4(st["w"][n:n + 4096].double(), c["fmt"]) for n in range(0, c["N"], 4096)])
    a = _exact_fp4(st["x"].double(), c["fmt"])
    return torch.cat([a @ _exact_packed(st, n, min(n + 4096, c["N"])).t() for n in range(0, c["N"], 4096)], dim=1)
