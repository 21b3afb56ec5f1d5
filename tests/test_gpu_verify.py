"""GPU parity of the verification of drafted tokens against its definition in
64 bits.

A weight is off by at most 2^-28 of itself (seven fp32 roundings of at most
2^-31 each, the first term left out of the power series below 2^-39), and so are
a cumulative sum and the total that the target is a part of; under max(p - q, 0)
the same holds in units of the total of p.  A decision has to agree where it is
further than 2^-26 from its border: the target from a step of the cumulative
sum, in those units, u q from p over the larger.
All inputs below are seeded, and their margins are asserted.  Probabilities: one
rounding to fp32 (2^-24), the weight's and the total's errors: below 2^-23.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_token_gb300 as fb
from tests.gpu_helpers import Ran
from tests.verify_reference import verify

pytestmark = pytest.mark.gpu

RUNS_ROWS, RUNS_RESIDUAL = 98, 99
MARGIN, P_TOL = 2.0 ** -26, 2.0 ** -23


class Batch:
    """Random logits with a few outstanding tokens a row, and drafts that are
    accepted about half of the time."""

    def __init__(self, B, L, V, dtype=torch.bfloat16, q=False, ragged=False, temps=None, seed=0, pad=0, masked=0.0,
                 std=2.0):
        rng = np.random.RandomState(seed)
        R = B * (L + 1)
        x = rng.standard_normal((R, V)) * std
        for r in range(R):
            x[r, rng.randint(0, V, 6)] += 4 + 6 * rng.rand(6)
        if masked:
            x[rng.rand(R, V) < masked] = -np.inf
            x[np.arange(R), rng.randint(0, V, R)] = 1.0
        full = torch.full((R, V + pad), 50.0, dtype=dtype)
        full[:, :V] = torch.from_numpy(x).to(dtype)
        self.full, self.x = full, full[:, :V]
        x = self.x.double().numpy()
        self.kw = dict(sample_u=rng.rand(B).astype(np.float32))
        if L:
            draft = np.zeros((B, L), np.int32)
            qs = np.zeros((B * L, V), np.float32)
            for b in range(B):
                for j in range(L):
                    z = x[b * (L + 1) + j]
                    z = np.where(np.isfinite(z), z + 0.7 * rng.standard_normal(V), -np.inf)
                    w = np.exp(z - z.max())
                    qs[b * L + j] = w / w.sum()
                    draft[b, j] = rng.choice(V, p=w / w.sum()) if q else int(np.argsort(z)[-1 - rng.randint(0, 2)])
            self.kw.update(draft=draft, accept_u=rng.rand(B, L).astype(np.float32))
            if q:
                self.kw["draft_probs"] = qs
            if ragged:
                self.kw["draft_len"] = rng.randint(0, L + 1, B).astype(np.int32)
        if temps is not None:
            self.kw["temperature"] = np.resize(np.array(temps, np.float32), B)

    def device(self):
        full = self.full.cuda()
        return full[:, :self.x.shape[1]], {k: torch.from_numpy(v).cuda() for k, v in self.kw.items()}

    def want(self):
        return verify(self.x.float().numpy().astype(np.float64), **self.kw)

    def run(self, **more):
        x, kw = self.device()
        return fb.speculative_verify(x, **kw, **more)


def _check(got, want):
    tokens, accepted, probs, m = want
    assert m > MARGIN, "the inputs have a decision at a border (%g): another seed" % m
    assert np.array_equal(got[1].cpu().numpy(), accepted)
    assert np.array_equal(got[0].cpu().numpy(), tokens)
    g = got[2].cpu().double().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(probs))
    ok = np.isnan(probs) | (np.abs(g - probs) <= P_TOL * probs)
    assert ok.all()


SHAPES = [(1, 0, 1), (1, 0, 5), (3, 0, 1000), (1, 4, 1000), (2, 1, 2), (5, 3, 257), (8, 7, 8192), (4, 2, 8193), (3, 5, 8191),
          (1, 31, 300), (2, 3, 50001), (1, 2, 248320), (17, 1, 3001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,L,V", SHAPES)
def test_matches_the_definition(B, L, V, dtype):
    for n, (q, ragged, temps) in enumerate([(True, False, None), (False, True, (0.7, 1.3)), (True, True, (1.0, 0.0, 0.25))]):
        t = Batch(B, L, V, dtype, q and L > 0, ragged, temps, seed=100 * B + 10 * L + n)
        with Ran() as r:
            got = t.run()
        assert r.launched() == ({RUNS_ROWS: 1, RUNS_RESIDUAL: 1} if "draft_probs" in t.kw else {RUNS_ROWS: 1})
        _check(got, t.want())


@pytest.mark.parametrize("pad", [1, 2, 7, 8, 13])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_address(dtype, pad):
    """Row strides that put every row at another offset from 16 bytes; what lies
    between the rows is larger than any logit and does not count."""
    t = Batch(3, 3, 9001, dtype, True, False, None, seed=pad, pad=pad)
    _check(t.run(), t.want())
    t = Batch(4, 0, 7, dtype, seed=pad, pad=pad)
    _check(t.run(), t.want())


@pytest.mark.parametrize("q", [True, False])
def test_masked_logits(q):
    t = Batch(6, 3, 12345, torch.float32, q, True, (0.9, 0.0), seed=3, masked=0.6)
    _check(t.run(), t.want())
    t = Batch(4, 2, 300, torch.bfloat16, q, False, None, seed=4, masked=1.1)  # one logit a row is left
    _check(t.run(), t.want())


def test_the_ends_of_the_range_of_logits():
    """The type's lowest value as a mask, rows far from zero on either side, and
    rows of equal logits."""
    V = 700
    rng = np.random.RandomState(0)
    rows = np.stack([np.where(rng.rand(V) < 0.5, -3.3895314e38, rng.standard_normal(V)), rng.standard_normal(V) - 3000.0,
                     rng.standard_normal(V) + 5000.0, np.full(V, -3.3895314e38), np.full(V, 3.3895314e38),
                     np.where(rng.rand(V) < 0.1, 1e30, -1e30), rng.standard_normal(V) * 1e-30, np.zeros(V)])
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.from_numpy(rows).to(dtype)
        u = np.linspace(0.0313, 0.9719, len(rows)).astype(np.float32)
        for T in (None, np.full(len(rows), 0.31, np.float32), np.full(len(rows), 300.0, np.float32)):
            want = verify(x.float().numpy().astype(np.float64), u, temperature=T)
            got = fb.speculative_verify(x.cuda(), torch.from_numpy(u).cuda(),
                                        temperature=None if T is None else torch.from_numpy(T).cuda())
            _check(got, want)


def test_rows_without_a_distribution():
    """NaN, +infinity, nothing but -infinity: token -1 and probability NaN there,
    the accepted tokens before it stand, other sequences do not notice."""
    for dtype in (torch.float32, torch.bfloat16):
        t = Batch(6, 3, 9000, dtype, True, False, None, seed=21)
        x = t.full
        x[1 * 4 + 0, 17] = float("nan")
        x[2 * 4 + 2, 8999] = float("inf")
        x[3 * 4 + 1] = -float("inf")
        x[4 * 4 + 3, 0] = float("nan")
        t.kw["accept_u"][1:5] = 0.0  # whatever has a probability is accepted
        want = t.want()
        assert list(want[1][1:5]) == [0, 2, 1, 3] and np.isnan(want[2]).sum() == 4
        _check(t.run(), want)
    for T in (-1.0, float("nan"), float("inf"), 1e-7, 2e6):
        t = Batch(2, 1, 100, temps=(T, 1.0), seed=2)
        want = t.want()
        assert want[0][0, 0] == -1
        _check(t.run(), want)


def test_equal_logits_take_the_lowest_index_at_temperature_zero():
    x = torch.zeros((3, 20000), dtype=torch.bfloat16)
    x[0, [9000, 12000, 15000]] = 3.0
    x[1, [19999, 4]] = 2.0
    x[2] = -1.0
    x[2, [8500, 8499]] = torch.tensor([0.0, -0.0], dtype=torch.bfloat16)
    got = fb.speculative_verify(x.cuda(), torch.rand(3, device="cuda"), temperature=torch.zeros(3, device="cuda"))
    assert got[0].cpu().flatten().tolist() == [9000, 4, 8499] and (got[2] == 1.0).all()


def test_the_same_probabilities_accept_and_draw_from_the_target():
    """q = p: u q < p for every u below 1 but for roundings of q; where a draft is
    rejected all the same nothing is left of p - q but them, or nothing at all."""
    V = 4
    x = torch.log2(torch.tensor([[0.5, 0.25, 0.125, 0.125]])) * np.log(2)
    x = x.repeat(2, 1).cuda()
    q = torch.tensor([[0.5, 0.25, 0.125, 0.125]], device="cuda")
    one = torch.ones((1, 1), device="cuda")
    for r, token in ((0.1, 0), (0.6, 1), (0.8, 2), (0.95, 3)):
        got = fb.speculative_verify(x, torch.full((1,), r, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                    one * 2, draft_probs=torch.cat([q * 4]))  # rejected; p - 4 q is negative everywhere
        assert got[1].tolist() == [0] and got[0].tolist() == [[token, -1]]
    got = fb.speculative_verify(x, torch.full((1,), 0.3, device="cuda"), torch.ones((1, 1), dtype=torch.int32, device="cuda"),
                                one * 0.99, draft_probs=q)
    assert got[1].tolist() == [1] and got[0].tolist() == [[1, 0]]


def test_a_rejected_draft_that_has_all_the_weight_but_traces():
    """p of the draft is 1 but for 2^-23, spread so thin that no other token has a
    unit (2^-41) of weight; rejected (by a number just below 1), another token has to
    come, with its probability; with a number above 1 and nothing left at all, the
    draft itself."""
    V = 600_000
    x = torch.full((2, V), -np.log(V * 2.0 ** 23), dtype=torch.float32)
    x[:, 77_777] = 0.0
    draft = torch.full((1, 1), 77_777, dtype=torch.int32)
    for u in (0.1, 0.7, float(np.nextafter(np.float32(1), np.float32(0)))):
        tok, acc, p = fb.speculative_verify(x.cuda(), torch.tensor([u]).cuda(), draft.cuda(), torch.tensor([[1 - 2.0 ** -24]]).cuda())
        assert acc.tolist() == [0] and 0 <= tok[0, 0] < V and tok[0, 0] != 77_777 and tok[0, 1] == -1
        assert abs(tok[0, 0].item() - u * V) < 1100  # in the right part of the row
        assert abs(p[0, 0].item() * V * 2.0 ** 23 - 1) < 1e-5
    x[:, :77_777] = x[:, 77_778:] = -float("inf")
    tok, acc, p = fb.speculative_verify(x.cuda(), torch.tensor([0.4]).cuda(), draft.cuda(), torch.tensor([[2.0]]).cuda())
    assert acc.tolist() == [0] and tok.tolist() == [[77_777, -1]] and p.tolist() == [[1.0, 0.0]]
    tok = fb.speculative_verify(x[:1].cuda(), torch.tensor([5.0]).cuda())[0]
    assert tok.tolist() == [[77_777]]


def test_drafted_tokens_outside_the_vocabulary_are_rejected():
    for q in (True, False):
        t = Batch(4, 2, 500, torch.bfloat16, q, seed=6)
        t.kw["draft"][:, 0] = [-1, 500, 2 ** 31 - 1, -2 ** 31]
        want = t.want()
        assert (want[1] == 0).all()
        _check(t.run(), want)


def test_draft_lengths_out_of_range_are_clamped():
    t = Batch(4, 3, 400, torch.bfloat16, True, seed=7)
    t.kw["draft_len"] = np.array([-5, 99, 2 ** 31 - 1, -2 ** 31], np.int32)
    _check(t.run(), t.want())


def test_random_numbers_at_and_past_their_ends():
    t = Batch(5, 0, 30000, torch.bfloat16, seed=8)
    x, _ = t.device()
    u = torch.tensor([0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, 2.0, float("nan")], device="cuda")
    tok, _, p = fb.speculative_verify(x, u)
    w = t.want()
    first = int(np.nonzero(np.exp(t.x[0].double().numpy() - t.x[0].double().max().item()) > 2.0 ** -42)[0][0])
    assert tok[0, 0] == first
    assert ((tok >= 0) & (tok < 30000)).all() and (p > 0).all()
    assert w[0].shape == tok.shape


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_random_numbers_at_their_ends_draw_the_first_and_last_tokens(dtype):
    """0, what is not positive and NaN: the first token whose weight is one unit (2^-41 of
    the largest) or more; the largest number below 1: the definition's token; 1 and more:
    the last one with a unit.  The weights here are 2^-33 and more."""
    V, ends = 30000, [0.0, -1.0, float("nan"), 1 - 2.0 ** -24, 1.0, 2.0, float("inf")]
    t = Batch(1, 0, V, dtype, seed=8)
    row = t.x[:1]
    assert (row.double().max() - row.double().min()) * np.log2(np.e) < 33
    x = row.repeat(len(ends), 1).cuda()
    tok, _, p = fb.speculative_verify(x, torch.tensor(ends, device="cuda"))
    near = verify(row.double().numpy(), np.array([1 - 2.0 ** -24]))
    assert near[3] > MARGIN
    want = [0, 0, 0, int(near[0][0, 0]), V - 1, V - 1, V - 1]
    assert tok.cpu()[:, 0].tolist() == want
    w = torch.softmax(row.double(), dim=1)[0, want]
    assert ((p.cpu().double()[:, 0] - w).abs() <= P_TOL * w).all()


@pytest.mark.parametrize("probs", [True, False])
def test_random_numbers_at_their_ends_behind_a_rejected_draft(probs):
    """The same over max(p - q, 0): its first and last tokens with a unit.  A drafted token
    that all of q lies on has none."""
    V, ends = 9000, [0.0, float("nan"), 1.0, 3.0]
    B = len(ends)
    t = Batch(1, 1, V, torch.float32, q=True, seed=12)
    p = torch.softmax(t.x[:1].double(), dim=1)[0]
    q = torch.zeros(V, dtype=torch.float64)
    if probs:
        q[:] = p * (1 + 2.0 ** -20)
        q[100:8001:7] *= 0.5          # p - q is positive there alone
        q = q.float().double()
        r = p - q
        assert torch.equal(torch.nonzero(r >= 0)[:, 0], torch.arange(100, 8001, 7)) and r[[100, 7996]].min() > 2.0 ** -36
        first, last, draft = 100, 7996, 5
    else:
        first, last, draft = 0, V - 2, V - 1
    d = torch.full((B, 1), draft, dtype=torch.int32, device="cuda")
    au = torch.full((B, 1), 1.5, device="cuda")                # rejected: u q is above p
    tok, acc, _ = fb.speculative_verify(t.x.repeat(B, 1).cuda(), torch.tensor(ends, device="cuda"), d, au,
                                        draft_probs=q.float()[None].repeat(B, 1).cuda() if probs else None)
    assert acc.tolist() == [0] * B and (tok[:, 1] == -1).all()
    assert tok.cpu()[:, 0].tolist() == [first, first, last, last]


def test_the_distribution_of_many_draws():
    """Draws at 4,096 evenly spaced numbers fall into each token's share."""
    V = 12
    p = torch.softmax(torch.linspace(-2, 2, V).double(), 0)
    x = torch.log(p).float()[None].repeat(4096, 1)
    u = (torch.arange(4096) + 0.5) / 4096
    tok = fb.speculative_verify(x.cuda(), u.float().cuda())[0].cpu().flatten()
    share = torch.bincount(tok.long(), minlength=V).double() / 4096
    assert ((share - p).abs() <= 1.0 / 4096 + 1e-6).all()


def test_outputs_of_the_caller_nothing_behind_them_and_clean_words():
    t = Batch(7, 4, 20000, torch.bfloat16, True, True, (1.0, 0.0, 0.5), seed=9)
    want = t.want()
    x, kw = t.device()
    n = fb.speculative_verify_workspace_size(7, 4, 20000)
    buf = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    buf[n:] = 77
    ints, floats = torch.full((64,), -9, dtype=torch.int32, device="cuda"), torch.full((48,), -9.0, device="cuda")
    out = dict(tokens=ints[1:36].view(7, 5), accepted=ints[40:47], probs=floats[3:38].view(7, 5))
    for _ in range(3):
        got = fb.speculative_verify(x, **kw, **out, workspace=buf[:n])
        assert got[0] is out["tokens"] and got[1] is out["accepted"] and got[2] is out["probs"]
        _check(got, want)
        assert (ints[:1] == -9).all() and (ints[36:40] == -9).all() and (ints[47:] == -9).all()
        assert (floats[:3] == -9).all() and (floats[38:] == -9).all() and (buf[n:] == 77).all()
        assert not buf[:1024 + 65536].any(), "status and counters back at zero"
        assert torch.equal(x, t.x.cuda())
    assert fb.workspace_status(buf) == 0


def test_bitwise_reproducible_captured_and_on_another_stream():
    t = Batch(16, 7, 40000, torch.bfloat16, True, False, None, seed=10)
    x, kw = t.device()
    work = fb.make_workspace(fb.speculative_verify_workspace_size(16, 7, 40000))
    first = fb.speculative_verify(x, **kw, workspace=work)
    _check(first, t.want())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            got = fb.speculative_verify(x, **kw, workspace=work, flags=fb.FLAG_OVERLAP_PREV)
            for a, b in zip(first, got):
                assert torch.equal(a, b)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = fb.speculative_verify(x, **kw, workspace=work)
    for _ in range(3):
        for k in kept:
            k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, kept):
            assert torch.equal(a, b)


def test_calls_of_different_sizes_share_a_workspace():
    calls = [Batch(1, 0, 100, seed=1), Batch(40, 3, 9000, q=True, seed=2), Batch(2, 9, 30000, seed=3), Batch(64, 0, 513, seed=4)]
    sizes = [fb.speculative_verify_workspace_size(len(c.kw["sample_u"]), c.kw["draft"].shape[1] if "draft" in c.kw else 0,
                                                  c.x.shape[1]) for c in calls]
    work = fb.make_workspace(max(sizes))
    for _ in range(2):
        for c in calls:
            _check(c.run(workspace=work), c.want())


@pytest.mark.parametrize("B,V,dtype", [(160, 60001, torch.bfloat16), (320, 60000, torch.bfloat16), (330, 59996, torch.float32)])
def test_a_batch_that_fills_the_gpu_several_times_gives_the_bits_of_its_sequences(B, V, dtype):
    """Several parts a warp, rows left out behind a stop: integer sums do not depend on it."""
    L = 3
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn((B * (L + 1), V), generator=g, device="cuda").mul_(2.0)
    x.scatter_add_(1, torch.randint(0, V, (B * (L + 1), 8), generator=g, device="cuda"),
                   torch.rand((B * (L + 1), 8), generator=g, device="cuda") * 6 + 6)
    x = x.to(dtype)
    z = x.view(B, L + 1, V)[:, :L].float()
    q = torch.softmax(z + 0.5 * torch.randn(z.shape, generator=g, device="cuda"), dim=2).view(B * L, V)
    draft = torch.multinomial(q, 1, generator=g).view(B, L).to(torch.int32)
    au, su = torch.rand((B, L), generator=g, device="cuda"), torch.rand((B,), generator=g, device="cuda")
    temp = torch.rand((B,), generator=g, device="cuda") + 0.5
    temp[::9] = 0.0
    n = torch.randint(0, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
    for probs in (q, None):
        all_of_them = fb.speculative_verify(x, su, draft, au, draft_probs=probs, draft_len=n, temperature=temp)
        if probs is not None:
            assert len(all_of_them[1].unique()) == L + 1, "the inputs have every number of accepted tokens"
        for b in range(0, B, 5):
            r = slice(b * (L + 1), (b + 5) * (L + 1))
            one = fb.speculative_verify(x[r], su[b:b + 5], draft[b:b + 5], au[b:b + 5], draft_len=n[b:b + 5],
                                        draft_probs=None if probs is None else probs[b * L:(b + 5) * L], temperature=temp[b:b + 5])
            for a, o in zip(all_of_them, one):
                assert torch.equal(a[b:b + 5], o)


def test_a_long_vocabulary_and_rows_past_32_bit_offsets():
    """The largest vocabulary, and logits of more than 2^32 bytes of which only a
    view's rows are read."""
    t = Batch(1, 1, 1048576, torch.float32, False, seed=5)
    _check(t.run(), t.want())
    big = torch.empty((4, 700_000_000), dtype=torch.bfloat16, device="cuda")
    view = big[:, 699_000_000:699_000_000 + 1001]
    t = Batch(4, 0, 1001, torch.bfloat16, seed=6)
    view.copy_(t.x)
    _check(fb.speculative_verify(view, torch.from_numpy(t.kw["sample_u"]).cuda()), t.want())


def test_refusals():
    t = Batch(2, 3, 64, torch.bfloat16, True, True, (1.0,), seed=1)
    x, kw = t.device()
    assert len(fb.speculative_verify(x, **kw)) == 3
    bad = [(dict(draft=kw["draft"].long()), TypeError), (dict(accept_u=kw["accept_u"][:1]), ValueError),
           (dict(accept_u=None), TypeError), (dict(draft=None), ValueError), (dict(draft_probs=kw["draft_probs"][:5]), ValueError),
           (dict(draft_probs=kw["draft_probs"].double()), TypeError), (dict(draft_len=kw["draft_len"][:1]), ValueError),
           (dict(temperature=torch.ones(3, device="cuda")), ValueError), (dict(sample_u=torch.rand(3, device="cuda")), ValueError),
           (dict(tokens=torch.empty((2, 3), dtype=torch.int32, device="cuda")), ValueError),
           (dict(probs=torch.empty((2, 4), device="cuda").half()), TypeError), (dict(flags=2), fb.Fp8bsError),
           (dict(workspace=fb.make_workspace(1024)), fb.Fp8bsError), (dict(sample_u=[0.5, 0.5]), TypeError)]
    for change, err in bad:
        with pytest.raises(err):
            fb.speculative_verify(x, **{**kw, **change})
    for logits, err in ((x.half(), TypeError), (x[:7], ValueError), (x.t().contiguous().t(), ValueError), (x.cpu(), ValueError),
                        (x[0], ValueError)):
        with pytest.raises(err):
            fb.speculative_verify(logits, **kw)
    for B, L, V in ((1, 32, 10), (129, 31, 10), (1, 0, 1048577)):
        with pytest.raises(fb.Fp8bsError):
            fb.speculative_verify_workspace_size(B, L, V)
