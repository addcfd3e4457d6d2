"""Truncated sampling and truncation on the GPU against 64 bits."""
import math

import numpy as np
import pytest
import torch

import sample_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTS = [torch.bfloat16, torch.float32]
INF = float("inf")


def uniforms(rows, seed):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed))


def check(x, u, rule, drawn=None, cut=None, rows=None):
    """Outputs of both calls against the definition; rule: (T, k, p, mp) or one for each row."""
    for r in range(x.shape[0]) if rows is None else rows:
        T, k, p, mp = (float(np.float32(v)) for v in (rule[r] if isinstance(rule, list) else rule))
        xr = x[r].double().numpy()
        tok, logp, kept, mask, (m, lz), near, near_u = ref.row_draw(xr, T, int(k), p, mp,
                                                                    float(u[r]))
        if near < ref.SHARE:
            continue
        if drawn is not None:
            assert int(drawn.kept[r]) == kept, r
            if near_u >= ref.SHARE:
                assert int(drawn.tokens[r]) == tok, r
                assert ref.log_close(float(drawn.logp[r]), logp), (r, float(drawn.logp[r]), logp)
        if cut is not None:
            assert int(cut.kept[r]) == kept, r
            want = torch.where(torch.from_numpy(mask), x[r], torch.full_like(x[r], -INF))
            assert torch.equal(cut.logits[r].cpu(), want), r
            assert ref.log_close(float(cut.stats[r, 0]), m)
            assert ref.log_close(float(cut.stats[r, 1]), lz), (float(cut.stats[r, 1]), lz)


def both(x, u, T, k, p, mp, **kw):
    """Both calls on x, outputs on the host, and the status word."""
    ws = S.Workspace(device=DEV)
    xd, ud = x.to(DEV), u.to(DEV)
    kw = dict(top_k=k, top_p=p, min_p=mp, workspace=ws, **kw)
    d = S.spec_sample(xd, ud, T, **kw)
    c = S.spec_truncate(xd, T, **kw)
    torch.cuda.synchronize()
    assert torch.equal(xd.cpu().view(torch.uint8), x.view(torch.uint8))
    d = S.SampledTokens(d.tokens.cpu(), d.logp.cpu(), d.kept.cpu())
    c = S.TruncatedRows(c.logits.cpu(), c.kept.cpu(), c.stats.cpu())
    return d, c, ws.status()


RULES = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 20, 0.8, 0.05),
         (1.0, 0, 1.0, 0.1), (0.7, 1000, 0.95, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0),
         (1.0, 0, 0.99, 0.02)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (2, 7), (4, 31), (5, 33), (1, 1000), (3, 4099),
                                    (2, 50257), (1, 129280), (7, 32000), (500, 515), (90, 8191)])
def test_shapes(rows, V, dt, rule):
    x, u = ref.logits(rows, V, rows + V, dt), uniforms(rows, V)
    d, c, st = both(x, u, *rule)
    assert st == 0
    some = range(rows) if rows < 10 else range(0, rows, 7)
    check(x, u, rule, d, c, some)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", ["const", "up", "down", "two", "ties", "zeros", "masked", "single",
                                  "lowest", "huge", "steps"])
@pytest.mark.parametrize("rule", [(1.0, 100, 0.9, 0.0), (1.0, 0, 0.7, 0.0), (0.8, 3000, 0.9, 0.0),
                                  (1.0, 5000, 1.0, 0.0), (1.0, 0, 1.0, 0.3)])
def test_orders(kind, dt, rule):
    """Rows that defeat the list, or have borders between equal logits."""
    V = 9001
    i = torch.arange(V)
    x = {"const": torch.zeros(V), "up": i / V * 4, "down": -i / V * 4,
         "two": (i % 2).float(), "ties": (i * 7919 % 13).float(),
         "zeros": torch.where(i % 3 == 0, 0.0, -0.0),
         "masked": torch.where(i % 5 == 0, (i * 7919 % 997).float() / 200, -INF),
         "single": torch.where(i == 4321, 1.5, -INF),
         "lowest": torch.where(i % 4 == 0, torch.finfo(dt).min, (i % 29).float() / 8),
         "huge": (i * 7919 % 1009).float() * 1e30,
         "steps": torch.floor(i / 100.0) / 16}[kind].to(dt)
    x = x.repeat(2, 1).contiguous()
    u = torch.tensor([0.03125, 0.8125])
    d, c, st = both(x, u, *rule)
    assert st == 0
    check(x, u, rule, d, c)


def test_borders_exact():
    """Equal masses: p and u on the border itself, in whole numbers."""
    x = torch.zeros(8, 64)
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 2.0 ** -24, 1 / 64, 3 / 64])
    d, c, _ = both(x, u, 1.0, 0, 0.5, 0.0)
    assert d.kept.tolist() == [32] * 8 and c.kept.tolist() == [32] * 8
    assert d.tokens.tolist() == [0, 8, 16, 24, 31, 0, 0, 1]
    d, _, _ = both(x, u, 1.0, 0, 1.0, 0.0)
    assert d.tokens.tolist() == [0, 16, 32, 48, 63, 0, 1, 3]
    d, _, _ = both(x, u, 1.0, 48, 1.0, 1.0)
    assert d.tokens.tolist() == [0, 12, 24, 36, 47, 0, 0, 2]


def test_draws_reach_the_tail():
    """Borders of unlikely tokens: every token of a flat row is where 64 bits have it."""
    V, rows = 129280, 64
    x = (torch.randn(1, V, generator=torch.Generator().manual_seed(3)) * 2).expand(rows, V)
    x = x.to(torch.bfloat16).contiguous()
    u = (torch.arange(rows) + 0.37) / rows
    d, _, _ = both(x, u, 1.0, 0, 1.0, 0.0)
    check(x, u, (1.0, 0, 1.0, 0.0), d)
    d, _, _ = both(x.float(), u, 1.0, 0, 0.97, 0.0)
    check(x.float(), u, (1.0, 0, 0.97, 0.0), d, rows=[0, 31, 63])


@pytest.mark.parametrize("T", [1e-30, 1e-3, 50.0, 1e30, 3e38])
@pytest.mark.parametrize("dt", DTS)
def test_temperatures(T, dt):
    x, u = ref.logits(4, 3001, 5, dt), uniforms(4, 6)
    for k, p, mp in ((0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.6, 0.2)):
        d, c, st = both(x, u, T, k, p, mp)
        assert st == 0
        check(x, u, (T, k, p, mp), d, c)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [2, 5, 40, 400])
def test_nuclei_that_end_next_to_a_heavy_token(heads, dt):
    """A few tokens hold most of the mass, alone in their places; p is a hundredth or less of the mass
    away from where one of them ends, so that a border guessed from counts is often a token off."""
    V, rows = 40000, 180
    g = torch.Generator().manual_seed(heads)
    x = torch.randn(rows, V, generator=g) * 2
    at = torch.stack([torch.randperm(V, generator=g)[:heads] for _ in range(rows)])
    x = x.scatter(1, at, 12 + 6 * torch.rand(rows, heads, generator=g)).to(dt)
    w = torch.softmax(x.double(), 1).sort(1, descending=True).values.cumsum(1)
    j = torch.randint(0, heads, (rows,), generator=g)
    off = (torch.rand(rows, generator=g).double() - 0.5) * 0.02
    p = (w.gather(1, j[:, None])[:, 0] * (1 + off)).clamp(0.01, 0.9999).float()
    u = uniforms(rows, heads)
    for n in (rows, 9):
        d, c, st = both(x[:n], u[:n], 1.0, 0, p[:n].contiguous().to(DEV), 0.0)
        assert st == 0
        check(x[:n], u[:n], [(1.0, 0, float(p[r]), 0.0) for r in range(n)], d, c,
              range(0, n, 1 if n < 20 else 6))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows", [6, 170])
@pytest.mark.parametrize("flat", [False, True])
def test_large_top_k_with_the_other_rules(flat, rows, dt):
    """More tokens than a list holds, by each rule and by two or three of them, ending before and
    behind one another."""
    V = 40000
    x = ref.logits(rows, V, 21, dt) if not flat else \
        (torch.randn(rows, V, generator=torch.Generator().manual_seed(22)) * 0.3).to(dt)
    u = uniforms(rows, 23)
    for k in (2000, 9000, 39999):
        for p in (0.3, 0.9, 0.999, 1.0):
            for mp in (0.0, 1e-4, 0.02, 0.3):
                d, c, st = both(x, u, 1.1, k, p, mp)
                assert st == 0
                check(x, u, (1.1, k, p, mp), d, c, (0, rows - 1))
    for p, mp in ((0.3, 1e-4), (0.9, 0.02), (0.99, 0.3), (1.0, 0.05)):
        d, c, st = both(x, u, 1.1, 0, p, mp)
        assert st == 0
        check(x, u, (1.1, 0, p, mp), d, c, (0, 1, rows - 1))


@pytest.mark.parametrize("rows", [1, 5, 170])
def test_thousands_of_equal_logits(rows):
    """bf16 logits far from zero lie on a coarse grid: a border is within thousands of equal ones, and
    ids decide."""
    V = 60000
    g = torch.Generator().manual_seed(31)
    x = torch.randn(rows, V, generator=g)
    x = torch.cat([x[:1] + 70, x[1:2] - 70, x[2:3] * 0.01 - 3, x[3:] * 2 + 40]).to(torch.bfloat16)
    x[:, ::7] = -INF
    u = uniforms(rows, 32)
    for k, p, mp in ((0, 0.3, 0.0), (0, 0.95, 0.0), (0, 0.9999, 0.0), (7000, 1.0, 0.0),
                     (30001, 1.0, 0.0), (30001, 0.77, 0.0), (20000, 0.9, 0.1), (0, 0.8, 0.2)):
        d, c, st = both(x, u, 1.0, k, p, mp)
        assert st == 0
        check(x, u, (1.0, k, p, mp), d, c, sorted({0, 1 % rows, 2 % rows, 3 % rows, rows - 1}))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows", [24, 600])
def test_parameters_per_request(rows, dt):
    V, per = 3001, 3
    x, u = ref.logits(rows, V, 11, dt), uniforms(rows, 12)
    n = rows // per
    g = torch.Generator().manual_seed(13)

    def pick(v, dtype):
        return torch.tensor(v, dtype=dtype)[torch.randint(len(v), (n,), generator=g)]
    T, k = pick([0.0, 0.7, 1.0, 1.3], torch.float32), pick([0, 1, 20, 200, 4000], torch.int32)
    p, mp = pick([1.0, 0.0, 0.8, 0.95], torch.float32), pick([0.0, 0.05, 1.0], torch.float32)
    rule = [(float(T[r // per]), int(k[r // per]), float(p[r // per]), float(mp[r // per]))
            for r in range(rows)]
    d, c, st = both(x, u, T.to(DEV), k.to(DEV), p.to(DEV), mp.to(DEV))
    assert st == 0
    check(x, u, rule, d, c, range(0, rows, max(1, rows // 40)))


def test_parameters_without_meaning():
    x, u = ref.logits(4, 500, 1, torch.float32), uniforms(4, 2)
    nan = float("nan")
    T = torch.tensor([nan, -1.0, INF, 1.0], device=DEV)
    p = torch.tensor([0.9, 0.9, nan, 2.0], device=DEV)
    mp = torch.tensor([0.0, nan, 0.1, -1.0], device=DEV)
    d, c, st = both(x, u, T, torch.tensor([5, -3, 7, 4], dtype=torch.int32, device=DEV), p, mp)
    assert st == S.SPEC_DEV_BAD_PARAM
    check(x, u, [(1.0, 5, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 7, 1.0, 0.1), (1.0, 4, 1.0, 0.0)],
          d, c)
    bad = torch.tensor([nan, -0.5, 1.0, INF])
    ws = S.Workspace(device=DEV)
    r = S.spec_sample(x.to(DEV), bad.to(DEV), 1.0, top_k=3, workspace=ws)
    top = x.topk(3, 1).indices
    assert ws.status() == S.SPEC_DEV_BAD_PARAM
    assert r.tokens.tolist() == [int(top[0].min()), int(top[1].min()), int(top[2].max()),
                                 int(top[3].max())]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rule", [(1.0, 0, 1.0, 0.0), (1.0, 5, 0.9, 0.0), (0.0, 0, 1.0, 0.0)])
@pytest.mark.parametrize("rows", [5, 400])
def test_rows_without_a_distribution(dt, rule, rows):
    x, u = ref.logits(rows, 2500, 21, dt), uniforms(rows, 22)
    x[0, 7] = float("nan")
    x[1, 1234] = INF
    x[2] = -INF
    x[3] = float("nan")
    d, c, st = both(x, u, *rule)
    assert st == S.SPEC_DEV_NONFINITE
    first = x[0].clone()
    first[7] = -INF
    assert d.tokens[:4].tolist() == [int(first.argmax()), 1234, 0, 0]
    assert torch.isnan(d.logp[:4]).all() and (d.kept[:4] == 0).all() and (c.kept[:4] == 0).all()
    assert torch.isnan(c.stats[:4]).all()
    bits = torch.int16 if dt == torch.bfloat16 else torch.int32
    assert torch.equal(c.logits[:4].view(bits), x[:4].view(bits))
    check(x, u, rule, d, c, [4, rows - 1])


@pytest.mark.parametrize("dt", DTS)
def test_strides_alignment_in_place(dt):
    """Row strides, odd offsets, inputs of more dimensions, an output of another alignment, and the
    output in place of the input."""
    rows, V = 9, 1003
    rule = (0.9, 0, 0.85, 0.0)
    wide = ref.logits(rows, V + 21, 31, dt)
    u = uniforms(rows, 32)
    x = wide[:, 5:5 + V]
    for T in (rule,):
        ws = S.Workspace(device=DEV)
        wd = wide.to(DEV)
        kw = dict(top_k=T[1], top_p=T[2], min_p=T[3], workspace=ws)
        d = S.spec_sample(wd[:, 5:5 + V], u.to(DEV), T[0], **kw)
        for shift in (0, 1, 5):
            to = torch.full((rows, V + 40), 7.0, dtype=dt, device=DEV)
            out = S.TruncatedRows.empty(x.to(DEV), rows)
            out.logits = to[:, shift:shift + V]
            S.spec_truncate(wd[:, 5:5 + V], T[0], out=out, **kw)
            check(x, u, rule, d, out)
            rest = to.cpu()
            rest[:, shift:shift + V] = 7.0
            assert (rest == 7.0).all()
        same = S.TruncatedRows(wd[:, 5:5 + V])
        S.spec_truncate(wd[:, 5:5 + V], T[0], out=same, **kw)
        check_in = same.logits.cpu()
        assert torch.equal(check_in, out.logits.cpu())
        after = wd.cpu()
        assert torch.equal(after[:, :5], wide[:, :5]) and torch.equal(after[:, 5 + V:],
                                                                      wide[:, 5 + V:])
    three = ref.logits(12, V, 33, dt).view(3, 4, V)
    d = S.spec_sample(three.to(DEV)[:, 1], u[:3].to(DEV), 1.0, top_k=9)
    check(three[:, 1], u, (1.0, 9, 1.0, 0.0), d)
    c = S.spec_truncate(three.to(DEV), 1.0, top_k=9)
    assert c.logits.shape == three.shape
    c.logits = c.logits.view(12, V)
    check(three.view(12, V), torch.zeros(12), (1.0, 9, 1.0, 0.0), None, c)


@pytest.mark.parametrize("rows", [10, 700])
def test_row_count(rows):
    V = 2100
    x, u = ref.logits(rows, V, 41, torch.bfloat16), uniforms(rows, 42)
    x[rows // 2:] = float("nan")
    ws = S.Workspace(device=DEV)
    for n, first in ((rows // 2, rows // 2), (0, 0), (-3, 0)):
        count = torch.tensor([n], dtype=torch.int32, device=DEV)
        d = S.SampledTokens.empty(rows, DEV)
        c = S.TruncatedRows.empty(x.to(DEV), rows)
        for t in (d.tokens, d.logp, d.kept, c.logits, c.kept, c.stats):
            t.fill_(-7)
        kw = dict(top_p=0.9, row_count=count, workspace=ws)
        S.spec_sample(x.to(DEV), u.to(DEV), 1.0, out=d, **kw)
        S.spec_truncate(x.to(DEV), 1.0, out=c, **kw)
        assert ws.status() == 0
        check(x, u, (1.0, 0, 0.9, 0.0), d, c, range(0, first, 5))
        for t in (d.tokens, d.logp, d.kept, c.logits, c.kept, c.stats):
            assert (t[first:] == -7).all()


def test_optional_outputs():
    x, u = ref.logits(3, 400, 51, torch.float32).to(DEV), uniforms(3, 52).to(DEV)
    full = S.spec_sample(x, u, 1.0, top_p=0.8)
    some = S.SampledTokens(torch.empty(3, dtype=torch.int32, device=DEV))
    S.spec_sample(x, u, 1.0, top_p=0.8, out=some)
    assert torch.equal(some.tokens, full.tokens)
    cut = S.TruncatedRows(torch.empty_like(x))
    S.spec_truncate(x, 1.0, top_p=0.8, out=cut)
    assert torch.equal(cut.logits, S.spec_truncate(x, 1.0, top_p=0.8).logits)


def test_same_however_split():
    """A row alone, split over a cluster, and among many that are not split: the same numbers."""
    V = 60000
    x, u = ref.logits(1000, V, 61, torch.bfloat16), uniforms(1000, 62)
    xd, ud = x.to(DEV), u.to(DEV)
    for rule in (dict(top_p=0.97), dict(), dict(top_k=300), dict(top_k=5000, top_p=0.9)):
        many = S.spec_sample(xd, ud, 0.9, **rule)
        for at in (0, 17, 999):
            one = S.spec_sample(xd[at:at + 1], ud[at:at + 1], 0.9, **rule)
            assert one.tokens[0] == many.tokens[at] and one.logp[0] == many.logp[at]
            assert one.kept[0] == many.kept[at]


def test_graph_streams_and_two_workspaces():
    x, u = ref.logits(40, 5000, 71, torch.bfloat16).to(DEV), uniforms(40, 72).to(DEV)
    want = S.spec_sample(x, u, 0.8, top_p=0.9)
    side, ws = torch.cuda.Stream(device=DEV), S.Workspace(256, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = S.spec_sample(x, u, 0.8, top_p=0.9, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.tokens, want.tokens) and torch.equal(got.logp, want.logp)
    out, cut = S.SampledTokens.empty(40, DEV), S.TruncatedRows.empty(x, 40)
    static = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.spec_truncate(static, 0.8, top_p=0.9, out=cut, workspace=ws)
        S.spec_sample(cut.logits, u, 0.8, out=out, workspace=ws)
    for seed in (73, 74):
        static.copy_(ref.logits(40, 5000, seed, torch.bfloat16))
        g.replay()
        again = S.spec_sample(static, u, 0.8, top_p=0.9)
        assert torch.equal(out.tokens, again.tokens) and torch.equal(out.kept, again.kept)
        assert torch.equal(out.logp, again.logp)


def test_large_vocabulary_and_far_rows():
    V = S.SPEC_SAMPLE_MAX_VOCAB
    x, u = ref.logits(2, V, 81, torch.float32), uniforms(2, 82)
    for rule in ((1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.5, 64, 0.9, 0.0)):
        d, c, st = both(x, u, *rule)
        assert st == 0
        check(x, u, rule, d, c)
    # rows more than 2^32 elements apart
    free = torch.cuda.mem_get_info()[0]
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    ld = (1 << 32) + 24
    buf = torch.empty(ld + 4096, dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((2, 4001), (ld, 1))
    src = ref.logits(2, 4001, 83, torch.bfloat16)
    far.copy_(src)
    d = S.spec_sample(far, u[:2].to(DEV), 1.0, top_p=0.9)
    check(src, u, (1.0, 0, 0.9, 0.0), d)


def test_another_device_is_refused_and_nothing_else_current():
    x = torch.zeros(2, 8, device=DEV)
    with pytest.raises(ValueError):
        S.spec_sample(x, torch.zeros(2), 1.0)
    with pytest.raises(ValueError):
        S.spec_sample(x, torch.zeros(2, device=DEV), torch.ones(2))
    assert math.isfinite(float(S.spec_sample(x, torch.zeros(2, device=DEV)).logp[0]))
