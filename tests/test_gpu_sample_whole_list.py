"""Top-k tokens that are exactly the ones a call lists, with a gap below them: the row is cut there."""
import pytest
import torch

from draft_sampling_verification_markov_gb300 import spec as S
from test_gpu_sample import DEV, DTS, both, check, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mp", [0.0, 1e-4])
@pytest.mark.parametrize("rows", [1, 6, 200])
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("k", [200, 300, 1000])
def test_k_tokens_above_a_gap(k, dt, rows, mp):
    """One of the k tokens in every batch of 64 bytes that a thread reads (pieces of 16 bytes, 32
    apart), so that the bound found from the batches' largest lies in the gap."""
    N = 8 if dt == torch.bfloat16 else 4
    V = 40000
    i = torch.arange(k)
    at = i // 32 * 128 * N + i % 32 * N
    g = torch.Generator().manual_seed(k)
    x = torch.randn(rows, V, generator=g)
    x[:, at] = 20 + torch.rand(rows, k, generator=g)
    x = x.to(dt)
    u = uniforms(rows, k)
    d, c, st = both(x, u, 2.0, k, 1.0, mp)
    assert st == 0
    check(x, u, (2.0, k, 1.0, mp), d, c, range(0, rows, 9))
    # however few rows a call has
    assert ((c.logits > -float("inf")).sum(1) == c.kept).all()


@pytest.mark.parametrize("mp", [0.0, 1e-30])
@pytest.mark.parametrize("rows", [1, 6, 200])
@pytest.mark.parametrize("dt", DTS)
def test_a_window_above_a_gap(dt, rows, mp):
    """5000 tokens, of which the last 1000 are one step of ten leading bits, and nothing else is in it."""
    V, k = 40000, 5000
    g = torch.Generator().manual_seed(3)
    x = torch.rand(rows, V, generator=g)
    ids = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(rows)])
    high = torch.cat([16 + torch.rand(rows, 4000, generator=g), 12 + torch.rand(rows, 1000, generator=g)], 1)
    x = x.scatter(1, ids, high).to(dt)
    x = torch.where((x >= 13) & (x < 16), torch.full_like(x, 12.5), x)
    u = uniforms(rows, 4)
    u[0] = 0.9999
    d, c, st = both(x, u, 3.0, k, 1.0, mp)
    assert st == 0
    check(x, u, (3.0, k, 1.0, mp), d, c, range(0, rows, 9))
    assert ((c.logits > -float("inf")).sum(1) == c.kept).all()


@pytest.mark.parametrize("dt", DTS)
def test_lists_of_many_rows(dt):
    """Random rows: what is left of a row is as many tokens as are said to be."""
    rows, V = 600, 3001
    x = torch.randn(rows, V, generator=torch.Generator().manual_seed(5)).to(dt).to(DEV)
    for k in range(257, 420, 3):
        for mp in (0.0, 0.01):
            c = S.spec_truncate(x, 2.0, top_k=k, min_p=mp)
            assert ((c.logits > -float("inf")).sum(1) == c.kept).all(), k
            if mp == 0.0:
                assert (c.kept == k).all()
