"""Token log-probabilities, rank, entropy and alternatives on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import head_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTS = [torch.bfloat16, torch.float32]
INF = float("inf")


def logits(rows, V, seed, dtype, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, V, generator=g) * std).to(dtype)


def tokens_for(rows, V, seed):
    return torch.randint(V, (rows,), generator=torch.Generator().manual_seed(seed),
                         dtype=torch.int32)


def check(x, tok, T, top, r, rows=None):
    """Outputs r against the definition; `rows` limits the comparison."""
    rows = torch.arange(x.shape[0]) if rows is None else torch.as_tensor(rows)
    V = x.shape[1]
    x64 = x[rows].double()
    want = ref.token_logprobs(x64, None if tok is None else tok[rows], T, top)
    z = x64 / T
    zmax = torch.where(torch.isfinite(z), (z - z.amax(1, keepdim=True)).abs(),
                       torch.zeros_like(z)).amax(1)
    tol = torch.tensor([ref.logp_tol(V, float(v)) for v in zmax], dtype=torch.float64)
    if tok is not None:
        assert ((r.logp.cpu()[rows].double() - want["logp"]).abs() <= tol).logical_or(
            r.logp.cpu()[rows].double() == want["logp"]).all()
        assert torch.equal(r.rank.cpu()[rows].long(), want["rank"])
    # the entropy's sum adds each term p |z| with the relative error of p
    assert ((r.entropy.cpu()[rows].double() - want["entropy"]).abs()
            <= 2 * tol * (1 + want["spread"])).all()
    if top:
        assert torch.equal(r.top_ids.cpu()[rows].long(), want["top_ids"])
        a, b = r.top_logp.cpu()[rows].double(), want["top_logp"]
        assert torch.equal(torch.isinf(a), torch.isinf(b))
        f = torch.isfinite(b)
        assert ((a - b).abs()[f] <= tol[:, None].expand_as(a)[f]).all()


def run(x, tok, T=1.0, top=0, **kw):
    ws = S.Workspace(device=DEV)
    r = S.spec_token_logprobs(x.to(DEV), None if tok is None else tok.to(DEV), T, top=top,
                              workspace=ws, **kw)
    torch.cuda.synchronize()
    return r, ws.status()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (2, 7), (4, 31), (5, 33), (1, 1000), (2, 1024),
                                    (3, 4099), (2, 50257), (1, 129280), (7, 32000), (400, 515),
                                    (320, 8191)])
@pytest.mark.parametrize("T,top", [(1.0, 20), (0.7, 1)])
def test_shapes(rows, V, dt, T, top):
    x, tok = logits(rows, V, rows + V, dt), tokens_for(rows, V, V)
    r, st = run(x, tok, T, top)
    assert st == 0
    check(x, tok, T, top, r)


@pytest.mark.parametrize("top", [0, 2, 5, 31, 32])
@pytest.mark.parametrize("V", [20, 3000, 40000])
def test_alternatives(top, V):
    x, tok = logits(6, V, top + V, torch.bfloat16), tokens_for(6, V, 1)
    r, _ = run(x, tok, 1.3, top)
    check(x, tok, 1.3, top, r)


def order_cases(V):
    up = torch.linspace(-5, 5, V)
    const = torch.zeros(V)
    blocks = (torch.arange(V) // 700).float() * 0.5
    tail = torch.zeros(V)
    tail[-40:] = 1.0
    one = torch.full((V,), -INF)
    one[V // 2] = 3.0
    few = torch.full((V,), -INF)
    few[[1, V // 3, V - 1]] = torch.tensor([1.0, 2.0, 2.0])
    low = torch.full((V,), torch.finfo(torch.bfloat16).min)
    low[5] = 0.0
    alllow = torch.full((V,), torch.finfo(torch.bfloat16).min)
    saw = (torch.arange(V) % 97).float() * 0.1
    zeros = torch.zeros(V)
    zeros[::2] = -0.0
    return torch.stack([up, up.flip(0), const, blocks, tail, one, few, low, alllow, saw, zeros])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V,repeat", [(60, 1), (4096, 1), (20001, 1), (70000, 1), (70000, 40)])
def test_orders_ties_and_masks(V, dt, repeat):
    """Sorted rows either way, equal logits, rows masked down to one or a few tokens with -inf or
    with the type's lowest value, a row of nothing but the lowest value, zeros of both signs."""
    x = order_cases(V).to(dt).repeat(repeat, 1)
    tok = tokens_for(x.shape[0], V, 3)
    r, st = run(x, tok, 1.0, 32)
    assert st == 0
    check(x, tok, 1.0, 32, r)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V", [100, 30000])
def test_masked_token_and_large_scores(V, dt):
    x = logits(4, V, 5, dt)
    tok = tokens_for(4, V, 6)
    x[0, tok[0]] = -INF
    x[1] *= 1e4
    x[2] = x[2] * 1e30
    x[3, : V // 2] = -INF
    tok[3] = V - 1
    r, st = run(x, tok, 1.0, 8)
    assert st == 0
    assert r.logp[0].item() == -INF
    x64 = x.double()
    assert r.rank[0].item() == int((x64[0] > -INF).sum()) + 1
    check(x, tok, 1.0, 8, r, rows=[1, 2, 3])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V", [50, 33000])
def test_rows_without_a_normaliser(V, dt):
    """NaN, +inf and empty rows are reported and have NaN outputs; their neighbours are right."""
    x, tok = logits(6, V, 8, dt), tokens_for(6, V, 9)
    x[1, 7] = float("nan")
    x[2, 9] = INF
    x[4] = -INF
    r, st = run(x, tok, 1.0, 4)
    assert st == S.SPEC_DEV_NONFINITE
    for row in (1, 2, 4):
        assert torch.isnan(r.logp[row]) and torch.isnan(r.entropy[row])
    assert r.top_ids[2, 0].item() == 9 and torch.isnan(r.top_logp[2]).all()
    assert 7 not in r.top_ids[1].tolist()
    assert r.top_ids[4].tolist() == [-1] * 4 and r.top_logp[4].tolist() == [-INF] * 4
    check(x, tok, 1.0, 4, r, rows=[0, 3, 5])


@pytest.mark.parametrize("V", [50, 33000])
def test_skipped_rows_and_bad_tokens(V):
    x, tok = logits(6, V, 8, torch.bfloat16), tokens_for(6, V, 9)
    tok[1], tok[2], tok[4] = -1, V, -7
    out = S.TokenLogprobs(*(torch.full((6,), 77, dtype=d, device=DEV)
                            for d in (torch.float32, torch.int32, torch.float32)),
                          torch.full((6, 3), 77, dtype=torch.int32, device=DEV),
                          torch.full((6, 3), 77.0, device=DEV))
    r, st = run(x, tok, 1.0, 3, out=out)
    assert st == S.SPEC_DEV_BAD_TOKEN
    for t in (r.logp, r.rank, r.entropy, r.top_ids, r.top_logp):
        assert (t[1] == 77).all()
    for row in (2, 4):
        assert torch.isnan(r.logp[row]) and r.rank[row].item() == 0
    good = tok.clone()
    good[[2, 4]] = 0
    full, _ = run(x, good, 1.0, 3)
    for name in ("entropy", "top_ids", "top_logp"):
        assert torch.equal(getattr(r, name)[[0, 2, 3, 4, 5]],
                           getattr(full, name)[[0, 2, 3, 4, 5]])
    check(x, tok, 1.0, 3, r, rows=[0, 3, 5])


def test_outputs_left_out_and_no_tokens():
    x = logits(5, 3000, 1, torch.float32)
    r, st = run(x, None, 1.0, 3)
    assert st == 0 and r.logp is None and r.rank is None
    check(x, None, 1.0, 3, r)
    only = S.TokenLogprobs(top_ids=torch.zeros(5, 3, dtype=torch.int32, device=DEV))
    run(x, None, 1.0, 3, out=only)
    assert torch.equal(only.top_ids, r.top_ids)
    zero, _ = run(x, None, 0.0, 3)                 # temperature 0: the unscaled softmax
    assert torch.equal(zero.top_logp, r.top_logp)
    empty, st = run(torch.zeros(0, 100), torch.zeros(0, dtype=torch.int32), 1.0, 2)
    assert st == 0 and empty.logp.shape == (0,)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cut", [0, 1, 8])
def test_strided_and_misaligned_rows(dt, cut):
    wide = logits(9, 3000, 4, dt).to(DEV)
    x = wide[:, cut:2500 + cut]
    tok = tokens_for(9, 2500, 2)
    ws = S.Workspace(device=DEV)
    a = S.spec_token_logprobs(x, tok.to(DEV), 1.0, top=7, workspace=ws)
    check(x.cpu(), tok, 1.0, 7, a)


def test_same_answer_every_time_on_a_stream_and_in_a_graph():
    x, tok = logits(33, 20000, 4, torch.bfloat16).to(DEV), tokens_for(33, 20000, 2).to(DEV)
    ws = S.Workspace(256, device=DEV)
    names = ("logp", "rank", "entropy", "top_ids", "top_logp")
    want = S.spec_token_logprobs(x, tok, 0.9, top=10, workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = [S.spec_token_logprobs(x, tok, 0.9, top=10, workspace=ws) for _ in range(3)]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again.append(S.spec_token_logprobs(x, tok, 0.9, top=10, workspace=ws))
    graph.replay()
    torch.cuda.synchronize()
    for r in again:
        assert all(torch.equal(getattr(r, n), getattr(want, n)) for n in names)


def test_agrees_with_the_verify_normalisers():
    """logp of a window's tokens from the normalisers of spec_target_stats."""
    x, tok = logits(16, 4096, 4, torch.bfloat16), tokens_for(16, 4096, 2)
    r, _ = run(x, tok, 0.8, 0)
    st = S.spec_target_stats(x.to(DEV), 0.8).cpu()
    at = x.gather(1, tok.long()[:, None])[:, 0].float()
    lp = at / 0.8 - st[:, 0] - st[:, 1]
    assert ((lp - r.logp.cpu()).abs() <= 1e-5 * lp.abs().clamp(min=1)).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T", [1.0, 0.7, 1.3])
def test_point_masses_are_exact(dt, T):
    """One token above -inf, or so far above the rest that they vanish in fp32."""
    x = torch.full((6, 9000), -INF)
    x[:, 4321] = torch.tensor([0.0, 3.7, -11.3, 250.0, -1e5, 1e20])
    x[1, 77], x[3, 5] = -400.0, 0.0
    tok = torch.full((6,), 4321, dtype=torch.int32)
    r, st = run(x.to(dt), tok, T, 2)
    assert st == 0
    assert (r.logp == 0).all() and (r.entropy == 0).all() and (r.top_logp[:, 0] == 0).all()
    one, _ = run(torch.full((3, 1), 5.5).to(dt), torch.zeros(3, dtype=torch.int32), T, 1)
    assert (one.logp == 0).all() and (one.entropy == 0).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("top", [1, 20, 32])
def test_rows_that_renew_their_bound(dt, top):
    """Long rows that are not split, with a few or hundreds of logits equal to the last one that
    has a place, and maxima that come late."""
    V, g = 150001, torch.Generator().manual_seed(top)
    x = torch.stack([torch.randn(V, generator=g) * 2, torch.rand(V, generator=g),
                     torch.round(torch.randn(V, generator=g) * 4),
                     torch.randn(V, generator=g) + torch.linspace(0, 4, V),
                     torch.randn(V, generator=g) * torch.linspace(3, 0.1, V)]).to(dt)
    tok = tokens_for(5, V, top)
    r, st = run(x.repeat(32, 1), tok.repeat(32), 0.9, top)
    assert st == 0
    # the copies begin at other addresses, so their sums may add in another order
    for c in (0, 5, 155):
        check(x, tok, 0.9, top, S.TokenLogprobs(*(getattr(r, f)[c:c + 5]
                                                  for f in S.TokenLogprobs.__slots__)))
    assert torch.equal(r.rank, r.rank[:5].repeat(32))
    assert torch.equal(r.top_ids, r.top_ids[:5].repeat(32, 1))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("first", [1, 1300])
def test_alternatives_behind_a_run_of_nans(first, dt):
    """A row that begins with more NaN logits than the first bound is made from still has its
    alternatives, whatever rows were before it."""
    V, n, k = 129280, 17000, 20
    x = logits(4, V, 5, dt)
    x[0] += 50
    x[1:, :n] = float("nan")
    x[2, :n:700] = x[2, n:n + 25]
    rows = torch.tensor([0] * first + [1, 2, 3] * 40)
    r = S.spec_token_logprobs(x.to(DEV)[rows.to(DEV)], None, 1.0, top=k,
                              workspace=S.Workspace(device=DEV))
    want = torch.where(x.isnan(), -INF, x.double())
    order = want.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.top_ids.cpu().long(), order[rows])
    assert r.top_logp[first:].isnan().all() and r.top_logp[:first].isfinite().all()
