"""What stands between the linear layers of a decode or speculative-verify
step: cases, plain forms and 64-bit values, for measuring the library's kernels.

``run`` computes an operator in its plain form (elementary torch operations)
or, where ``own`` is true, through the public entry points of
fp8_block_scaled_token_gb300.  ``exact`` gives the same outputs from the
definitions in 64 bits, written apart from the plain form.  Three operators:

* ``norm``: the residual's addition, root-mean-square norm and the cast to
  E4M3, with one fp32 scale per 128 values ("fp8") or one power of two per 32
  ("mx"); codes are returned as the E4M3 numbers that they are.
* ``route``: router product, softmax or sigmoid scores, balance bias, choice of
  groups and of experts, weights.  The plain form works in 64 bits: a score next
  to the last chosen one decides by its last digits.
* ``verify``: drafted tokens against the target's probabilities from given
  random numbers, and the next token.  The plain form works in 64 bits: a step of
  the cumulative sum is a millionth of it.
"""
import math

import torch

own = False

# ------------------------------------------------------------------ cases
_LISTED = [
    # one decoding sequence, before a projection: latency only
    dict(name="norm_m1", op="norm", fmt="fp8", M=1, K=5120, res=True, y=False, gamma="bf16"),
    # an odd number of rows, fp32 weights of the norm, power-of-two scales, the embedding's rows (no residual yet)
    dict(name="norm_mx_m37", op="norm", fmt="mx", M=37, K=1408, res=False, y=True, gamma="f32"),
    # a chunk of a prompt before the expert layer's router: y as well
    dict(name="norm_m512", op="norm", fmt="fp8", M=512, K=5120, res=True, y=True, gamma="bf16"),
    # a long prompt at once: memory-bound
    dict(name="norm_m16384", op="norm", fmt="fp8", M=16384, K=5120, res=True, y=True, gamma="bf16"),
    # one decoding sequence, sigmoid scores with a bias, no groups
    dict(name="route_m1", op="route", M=1, H=2048, E=64, k=6, score="sigmoid", bias=True, G=1, tg=1, best=2, wr="bf16",
         renorm=True, scale=1.0),
    # a speculative-verify batch: sigmoid scores, bias, 4 of 8 groups by their two best
    dict(name="route_m8_groups", op="route", M=8, H=5120, E=256, k=8, score="sigmoid", bias=True, G=8, tg=4, best=2,
         wr="f32", renorm=True, scale=2.5),
    # the largest batch: softmax scores, 3 of 8 groups by their best, weights as they are
    dict(name="route_m64_softmax", op="route", M=64, H=5120, E=160, k=6, score="softmax", bias=False, G=8, tg=3, best=1,
         wr="bf16", renorm=False, scale=16.0),
    # the next token of one sequence, no draft, a small vocabulary: latency only
    dict(name="verify_sample", op="verify", B=1, L=0, V=1000, x="bf16", q=False, ragged=False, temp=True, mask=False, pad=0),
    # four drafted tokens of one sequence against the repository's output layer
    dict(name="verify_m5", op="verify", B=1, L=4, V=248320, x="bf16", q=True, ragged=False, temp=False, mask=False, pad=0),
    # drafts of several lengths without probabilities (prompt lookup), masked logits, temperatures with 0, an odd vocabulary
    dict(name="verify_ragged", op="verify", B=13, L=3, V=50001, x="f32", q=False, ragged=True, temp=True, mask=True, pad=7),
    # eight sequences of seven drafted tokens
    dict(name="verify_m64", op="verify", B=8, L=7, V=248320, x="bf16", q=True, ragged=False, temp=True, mask=False, pad=0),
    # a full server: 512 rows of logits
    dict(name="verify_m512", op="verify", B=64, L=7, V=248320, x="bf16", q=True, ragged=False, temp=False, mask=False, pad=0),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "verify"])
    if op == "norm":
        while True:
            fmt = rng.choice(["fp8", "mx"])
            c = dict(op=op, fmt=fmt, M=_log_int(rng, 1, 512 if fmt == "mx" else 16384), K=128 * _log_int(rng, 1, 136),
                     res=rng.random() < 0.7, y=rng.random() < 0.5, gamma=rng.choice(["bf16", "f32"]))
            if c["M"] * c["K"] <= 16384 * 5120:
                return c
    if op == "route":
        while True:
            G = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
            E = G * _log_int(rng, 2, 64) if G > 1 else _log_int(rng, 4, 320)
            c = dict(op=op, M=_log_int(rng, 1, 64), H=128 * _log_int(rng, 2, 40), E=E, score=rng.choice(["softmax", "sigmoid"]),
                     bias=rng.random() < 0.6, G=G, tg=rng.randint(1, G), best=rng.randint(1, 2), wr=rng.choice(["bf16", "f32"]),
                     renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]))
            c["k"] = rng.randint(1, min(12, c["tg"] * (E // G)))
            if E <= 512 and c["M"] * c["H"] * E <= 64 * 5120 * 256:
                return c
    while True:
        c = dict(op=op, B=_log_int(rng, 1, 64), L=rng.randint(0, 9), V=_log_int(rng, 256, 248320), x=rng.choice(["bf16", "f32"]),
                 q=rng.random() < 0.6, ragged=rng.random() < 0.5, temp=rng.random() < 0.5, mask=rng.random() < 0.3,
                 pad=rng.choice([0, 0, 8, 13]))
        c["q"] = c["q"] and c["L"] > 0
        if c["B"] * (c["L"] + 1) * c["V"] <= 256 * 248320:
            return c


def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        per = 2 + (4 if case["res"] else 0) + (2 if case["y"] else 0) + 1 + (1 / 32 if case["fmt"] == "mx" else 4 / 128)
        return {"bytes": M * K * per + K * (4 if case["gamma"] == "f32" else 2), "flops": 8.0 * M * K}
    if case["op"] == "route":
        M, E, H = case["M"], case["E"], case["H"]
        return {"bytes": E * H * (4 if case["wr"] == "f32" else 2) + 2.0 * M * H + 8 * M * case["k"] + (4 * E if case["bias"] else 0),
                "flops": 2.0 * M * E * H}
    B, L, V = case["B"], case["L"], case["V"]
    # the rows that a sequence needs: up to its first rejected token.  With two tokens of three accepted, as the
    # inputs below are, (1 - a^(L+1)) / (1 - a) rows in the mean, and one row of q for all but a^L of them.
    a = 2.0 / 3.0
    rows = B * (1.0 - a ** (L + 1)) / (1.0 - a)
    size = 4 if case["x"] == "f32" else 2
    return {"bytes": rows * V * size + (B * (1.0 - a ** L) * V * 4 if case["q"] else 0) + 8.0 * B * (L + 1),
            "flops": 4.0 * rows * V}


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


def _norm_state(c, g):
    M, K = c["M"], c["K"]
    gamma = torch.rand((K,), generator=g, device="cuda") * 1.5 + 0.25
    return dict(x=_activations(g, M, K), gamma=gamma if c["gamma"] == "f32" else gamma.to(torch.bfloat16), eps=1e-6,
                res=(torch.randn((M, K), generator=g, device="cuda") * 3.0).to(torch.bfloat16) if c["res"] else None)


def _route_state(c, g):
    wr = torch.randn((c["E"], c["H"]), generator=g, device="cuda").mul_(1.5 / math.sqrt(c["H"]))
    return dict(x=_activations(g, c["M"], c["H"]), wr=wr if c["wr"] == "f32" else wr.to(torch.bfloat16),
                bias=torch.randn((c["E"],), generator=g, device="cuda") * 0.05 if c["bias"] else None)


def _verify_state(c, g):
    """Logits: N(0, 2^2) and twenty tokens a row that stand out.  The draft
    model's: the same with noise; the drafted tokens are its own samples (or,
    without probabilities, one of the three likeliest of the target)."""
    B, L, V = c["B"], c["L"], c["V"]
    R = B * (L + 1)
    ld = V + c["pad"]
    x = torch.randn((R, ld), generator=g, device="cuda").mul_(2.0)
    top = torch.randint(0, V, (R, 20), generator=g, device="cuda")
    x.scatter_add_(1, top, torch.rand((R, 20), generator=g, device="cuda") * 6.0 + 6.0)
    if c["mask"]:  # what a grammar forbids
        x.masked_fill_(torch.rand((R, ld), generator=g, device="cuda") < 0.3, -math.inf)
    st = dict(accept_u=None, draft=None, q=None, draft_len=None, temp=None)
    if L:
        z = x.view(B, L + 1, ld)[:, :L, :V]
        if c["q"]:
            q = torch.randn((B, L, V), generator=g, device="cuda").mul_(0.5).add_(z)
            q.sub_(q.amax(dim=2, keepdim=True)).exp_()
            q.div_(q.sum(dim=2, keepdim=True))
            st["q"] = q.view(B * L, V)
            st["draft"] = torch.multinomial(st["q"], 1, generator=g).view(B, L).to(torch.int32)
        else:
            rank = torch.randint(0, 3, (B, L, 1), generator=g, device="cuda")
            st["draft"] = torch.topk(z, 3, dim=2)[1].gather(2, rank).view(B, L).to(torch.int32)
        st["accept_u"] = torch.rand((B, L), generator=g, device="cuda")
        if c["ragged"]:
            st["draft_len"] = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if c["temp"]:  # every fourth sequence takes the likeliest token
        t = torch.rand((B,), generator=g, device="cuda") * 0.8 + 0.6
        st["temp"] = torch.where(torch.arange(B, device="cuda") % 4 == 3, torch.zeros_like(t), t)
    st["x"] = (x if c["x"] == "f32" else x.to(torch.bfloat16))[:, :V]
    st["sample_u"] = torch.rand((B,), generator=g, device="cuda")
    return st


def prepare(case, seed):
    g = _gen(seed)
    make = {"norm": _norm_state, "route": _route_state, "verify": _verify_state}[case["op"]]
    return dict(make(case, g), case=dict(case))


# ------------------------------------------------------------- plain forms
def _atoms(byts):
    """Scale bytes [M, K/32] -> [token tiles * K/128, 512]: per 128 rows and four
    blocks, row r's block j at 16 (r % 32) + 4 (r / 32) + j; rows past M zero."""
    M, n = byts.shape
    tt = -(-M // 128)
    p = torch.zeros((tt * 128, n), dtype=torch.uint8, device=byts.device)
    p[:M] = byts
    return p.view(tt, 4, 32, n // 4, 4).permute(0, 3, 2, 1, 4).reshape(tt * (n // 4), 512).contiguous()


def _norm_out(fmt, codes, scales, h, y):
    out = dict(codes=codes, scales=scales)
    if h is not None:
        out["h"] = h
    if y is not None:
        out["y"] = y
    return out


def _pow2(e):
    """2^e as fp32, exact, from int32 exponents in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_norm(st):
    c = st["case"]
    M, K = c["M"], c["K"]
    h = st["x"].float()
    if c["res"]:
        h = (h + st["res"].float()).to(torch.bfloat16)
    f = h.float()
    u = f * st["gamma"].float()
    r = 1.0 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + st["eps"])
    v = u * r
    if c["fmt"] == "fp8":  # a group's codes do not depend on the row's r, its scale does
        b = u.view(M, K // 128, 128)
        am = b.abs().amax(dim=2)
        s = torch.where(am > 0, am / torch.full((), 448.0, device=v.device), torch.ones_like(am))
        codes = (b / s[:, :, None]).to(torch.float8_e4m3fn).view(M, K)
        s = torch.where(am > 0, s * r, s)
        s = s if M <= 16 else s.t().contiguous()
    else:
        b = v.view(M, K // 32, 32)
        am = b.abs().amax(dim=2)
        e = torch.where(am > 0, torch.frexp(am)[1] - 9, torch.zeros_like(am, dtype=torch.int32)).clamp(-126, 127)
        codes = (b * _pow2(-e)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(M, K)
        s = _atoms((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)
    return _norm_out(c["fmt"], codes, s, h if c["res"] else None, v.to(torch.bfloat16) if c["y"] else None)


def _plain_route(st):
    c = st["case"]
    M, E, G, k = c["M"], c["E"], c["G"], c["k"]
    l = st["x"].double() @ st["wr"].double().t()
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    choice = s if st["bias"] is None else s + st["bias"].double()
    if c["tg"] < G:
        group = torch.sort(choice.view(M, G, E // G), dim=2, descending=True)[0][:, :, :c["best"]].sum(dim=2)
        rank = torch.sort(torch.sort(group, dim=1, descending=True, stable=True)[1], dim=1)[1]
        choice = torch.where((rank < c["tg"])[:, :, None], choice.view(M, G, E // G), -math.inf).view(M, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return dict(ids=ids.to(torch.int32), weights=(w * c["scale"]).float())


def _plain_verify(st):
    c = st["case"]
    B, L, V = c["B"], c["L"], c["V"]
    dev = st["x"].device
    x = st["x"].double().view(B, L + 1, V)
    m = x.amax(dim=2, keepdim=True)
    if st["temp"] is None:
        p = torch.exp(x - m)
    else:
        t = st["temp"].double()[:, None, None]
        p = torch.exp((x - m) / torch.where(t > 0, t, 1.0))
        first = torch.where(x == m, torch.arange(V, device=dev), V).amin(dim=2, keepdim=True)
        p = torch.where(t > 0, p, (torch.arange(V, device=dev) == first).double())
    p /= p.sum(dim=2, keepdim=True)
    del x
    if L:
        at = torch.arange(L, device=dev)
        d = st["draft"].long()[:, :, None]
        pt = p[:, :L].gather(2, d)[:, :, 0]
        qt = 1.0 if st["q"] is None else st["q"].view(B, L, V).gather(2, d)[:, :, 0].double()
        ok = st["accept_u"].double() * qt < pt
        if st["draft_len"] is not None:
            ok &= at[None] < st["draft_len"][:, None]
        n = ok.int().cumprod(dim=1).sum(dim=1)
        lens = torch.full_like(n, L) if st["draft_len"] is None else st["draft_len"].long()
    else:
        n = torch.zeros((B,), dtype=torch.int64, device=dev)
        lens = n
    b = torch.arange(B, device=dev)
    p_n = p[b, n]
    if L:
        j = n.clamp(max=L - 1)
        if st["q"] is None:
            q_n = (torch.arange(V, device=dev)[None] == st["draft"].long()[b, j][:, None]).double()
        else:
            q_n = st["q"].view(B, L, V)[b, j].double()
        r = (p_n - q_n).clamp(min=0.0)
        r = torch.where(((n < lens) & (r.sum(dim=1) > 0))[:, None], r, p_n)
    else:
        r = p_n
    cum = r.cumsum(dim=1)
    target = st["sample_u"].double() * cum[:, -1]
    last = torch.where(r > 0, torch.arange(V, device=dev), 0).amax(dim=1)
    nxt = torch.minimum((cum <= target[:, None]).sum(dim=1), last)
    pos = torch.arange(L + 1, device=dev)[None]
    tokens = torch.where(pos == n[:, None], nxt[:, None], -1)
    probs = torch.where(pos == n[:, None], p_n.gather(1, nxt[:, None]), 0.0)
    if L:
        keep = at[None] < n[:, None]
        tokens[:, :L] = torch.where(keep, st["draft"].long(), tokens[:, :L])
        probs[:, :L] = torch.where(keep, pt, probs[:, :L])
    return dict(tokens=tokens.to(torch.int32), accepted=n.to(torch.int32), probs=probs.float())


def _plain(st):
    return {"norm": _plain_norm, "route": _plain_route, "verify": _plain_verify}[st["case"]["op"]](st)


# ------------------------------------------------------ the library's calls
def _own_norm(st, fb):
    c = st["case"]
    call = fb.fp8_rmsnorm_quant_act if c["fmt"] == "fp8" else fb.fp8_mx_rmsnorm_quant_act
    q, s, h, y = call(st["x"], st["gamma"], st["eps"], residual=st["res"], store_y=c["y"])
    if c["fmt"] == "mx":
        s = s.view(torch.float8_e8m0fnu)
    return _norm_out(c["fmt"], q.view(torch.float8_e4m3fn), s, h, y)


def _own_route(st, fb):
    c = st["case"]
    if "work" not in st:
        st["work"] = fb.make_workspace(fb.moe_route_workspace_size(c["M"], c["E"]))
    ids, w = fb.moe_route_grouped(st["x"], st["wr"], c["k"], bias=st["bias"],
                                  scoring=fb.SCORE_SIGMOID if c["score"] == "sigmoid" else fb.SCORE_SOFTMAX,
                                  groups=c["G"], top_groups=c["tg"], group_best=c["best"], renormalize=c["renorm"],
                                  scale=c["scale"], workspace=st["work"])
    return dict(ids=ids, weights=w)


def _own_verify(st, fb):
    c = st["case"]
    if "work" not in st:
        st["work"] = fb.make_workspace(fb.speculative_verify_workspace_size(c["B"], c["L"], c["V"]))
    tokens, accepted, probs = fb.speculative_verify(st["x"], st["sample_u"], draft=st["draft"], accept_u=st["accept_u"],
                                                    draft_probs=st["q"], draft_len=st["draft_len"], temperature=st["temp"],
                                                    workspace=st["work"])
    return dict(tokens=tokens, accepted=accepted, probs=probs)


def run(st):
    if own:
        import fp8_block_scaled_token_gb300 as fb
        return {"norm": _own_norm, "route": _own_route, "verify": _own_verify}[st["case"]["op"]](st, fb)
    return _plain(st)


# ------------------------------------------------------------ 64-bit values
def _round_to(q, bits, emin, top):
    """float64 q to `bits` fraction bits, ties to even, least exponent emin, saturating at top."""
    a = q.abs()
    e = (torch.frexp(a)[1] - 1).clamp(min=emin)
    step = torch.exp2((e - bits).double())
    return torch.sign(q) * (torch.round(a / step) * step).clamp(max=top)


def _exact_norm(st):
    c = st["case"]
    M, K = c["M"], c["K"]
    h = st["x"].double()
    if c["res"]:  # the stored sum is bf16, and the norm is that of what is stored
        h = (h + st["res"].double()).float().to(torch.bfloat16).double()
    v = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / K + st["eps"]) * st["gamma"].double()
    per = 128 if c["fmt"] == "fp8" else 32
    b = v.view(M, K // per, per)
    am = b.abs().amax(dim=2)
    if c["fmt"] == "fp8":
        s = am / 448.0
        s[am == 0] = 1.0
        u = (h * st["gamma"].double()).view_as(b)  # what lies between two codes does so exactly
        b = u * 448.0
        d = u.abs().amax(dim=2)
        d[d == 0] = 1.0
        out = s if M <= 16 else s.t().contiguous()
    else:
        e = torch.floor(torch.log2(am)) - 8.0
        e[am == 0] = 0.0
        s = torch.exp2(e.clamp(min=-127.0))
        tt = -(-M // 128)
        out = torch.full((tt, K // 128, 32, 4, 4), 2.0 ** -127, dtype=torch.float64, device=v.device)
        row = torch.arange(M, device=v.device)
        out[row // 128, :, row % 32, row % 128 // 32, :] = s.view(M, K // 128, 4)
        out = out.view(tt * (K // 128), 512)
        d = s
    codes = _round_to((b / d[:, :, None]).view(M, K), 3, -6, 448.0)
    return _norm_out(c["fmt"], codes, out, h if c["res"] else None, v if c["y"] else None)


def _exact_route(st):
    c = st["case"]
    M, E, G, k = c["M"], c["E"], c["G"], c["k"]
    l = torch.einsum("mh,eh->me", st["x"].double(), st["wr"].double())
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
    t = s.clone() if st["bias"] is None else s + st["bias"].double()
    if c["tg"] < G:
        per = torch.topk(t.view(M, G, -1), c["best"], dim=2)[0].sum(dim=2)
        keep = torch.zeros((M, G), dtype=torch.bool, device=t.device)
        keep.scatter_(1, torch.topk(per, c["tg"], dim=1)[1], True)
        t.masked_fill_(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    w = s.gather(1, torch.topk(t, k, dim=1)[1])
    return dict(ids=None, weights=w * c["scale"] / (w.sum(dim=1, keepdim=True) if c["renorm"] else 1.0))


def _exact_verify(st):
    c = st["case"]
    B, L, V = c["B"], c["L"], c["V"]
    probs = torch.zeros((B, L + 1), dtype=torch.float64, device=st["x"].device)
    x = st["x"].reshape(B, L + 1, V)
    for b in range(B):
        t = 1.0 if st["temp"] is None else float(st["temp"][b])
        n = L if st["draft_len"] is None else int(st["draft_len"][b])
        for j in range(n + 1):
            row = x[b, j].double()
            if t > 0:
                p = torch.softmax(row / t, dim=0)
            else:
                p = torch.zeros_like(row)
                p[int(torch.nonzero(row == row.max())[0])] = 1.0
            w = p
            if j < n:
                tok = int(st["draft"][b, j])
                q = torch.zeros_like(p)
                if st["q"] is None:
                    q[tok] = 1.0
                else:
                    q = st["q"][b * L + j].double()
                if float(st["accept_u"][b, j]) * float(q[tok]) < float(p[tok]):
                    probs[b, j] = p[tok]
                    continue
                w = torch.relu(p - q)
                w = w if bool(w.any()) else p
            cum = torch.cumsum(w, dim=0)
            at = torch.searchsorted(cum, cum[-1:] * st["sample_u"][b].double(), right=True)
            probs[b, j] = p[min(int(at), int(torch.nonzero(w)[-1]))]
            break
    return dict(tokens=None, accepted=None, probs=probs)


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "verify": _exact_verify}[case["op"]](st)
