"""Truncated sampling where logits are far apart beside the temperature, or beside fp32's range."""
import math

import pytest
import torch

import sample_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S
from test_gpu_sample import DEV, both, check, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,step,most,T", [(100.0, 2.0 ** -17, 43, 1e-5), (2048.0, 2.0 ** -13, 27, 1e-4),
                                           (30.0, 2.0 ** -19, 1, 4e-8), (-100.0, 2.0 ** -17, 43, 1e-5)])
@pytest.mark.parametrize("rows", [1, 3, 160])
def test_rows_on_the_grid_below_their_largest(rows, m, step, most, T):
    """Every logit within a few steps of fp32 of the largest, the last of them next to where masses
    end (2^-47 of the largest's). The rows differ only in which tokens those are."""
    V = 40000
    g = torch.Generator().manual_seed(7)
    j = torch.randint(0, most + 1, (rows, V), generator=g)
    j[0, 1:] = most                    # one token far above the others, which weigh nothing
    j[0, 0] = 0
    x = (m - j.double() * step).float()
    assert (x.double() == m - j.double() * step).all()
    u = uniforms(rows, 8)
    for k, p, mp in ((0, 1.0, 0.0), (0, 0.9, 0.0), (0, 0.999, 0.0), (9000, 0.97, 0.0), (0, 1.0, 0.01)):
        d, c, st = both(x, u, T, k, p, mp)
        assert st == 0
        check(x, u, (T, k, p, mp), d, c, sorted({0, min(1, rows - 1), rows - 1}))


@pytest.mark.parametrize("T", [1.0, 1e38, 3e38])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_logits_farther_apart_than_the_largest_number(dt, T):
    """What is more than 3.4e38 below the largest weighs nothing; the rest as ever."""
    V, rows = 6000, 4
    g = torch.Generator().manual_seed(9)
    x = torch.full((rows, V), -3e38)
    x[:, ::3] = 3e38 * torch.rand(rows, V // 3, generator=g)
    x[:, 30] = 3e38
    x = x.to(dt)
    near = x.double() >= x.double().amax(1, keepdim=True) - 3.4e38
    u = uniforms(rows, 10)
    for p in (1.0, 0.8):
        d, c, st = both(x, u, T, 0, p, 0.0)
        assert st == 0
        z = torch.where(near, (x.double() - x.double().amax(1, keepdim=True)) / T, -math.inf)
        if p == 1.0:
            assert (d.kept == V).all() and (c.kept == V).all()
            lz = torch.logsumexp(z, 1)
            assert torch.allclose(c.stats[:, 1].double(), lz, rtol=1e-5, atol=1e-6)
            lp = z.gather(1, d.tokens.long()[:, None])[:, 0] - lz
            assert torch.allclose(d.logp.double(), lp, rtol=1e-5, atol=1e-6)
        assert near.gather(1, d.tokens.long()[:, None]).all()


@pytest.mark.parametrize("rows", [2, 170])
def test_bf16_logits_far_below_the_largest_in_magnitude(rows):
    """Tails of logits near zero beside a largest of 4 to 5: their differences from it take more than 24
    bits, so that a mass may be off by 2^-24 (max - x) / T, 2^-21 here. Borders farther off than that
    are where 64 bits have them."""
    V = 30000
    g = torch.Generator().manual_seed(11)
    x = 1e-5 + 3e-5 * torch.rand(rows, V, generator=g)
    x[:, 77] = 4 + torch.rand(rows, generator=g)
    x = x.to(torch.bfloat16)
    u = uniforms(rows, 12)
    for p in (0.3, 0.9):
        d, c, st = both(x, u, 1.0, 0, p, 0.0)
        assert st == 0
        for r in (0, 1, rows - 1):
            tok, logp, kept, _, (m, lz), near, near_u = ref.row_draw(
                x[r].double().numpy(), 1.0, 0, float(torch.tensor(p)), 0.0, float(u[r]))
            if near >= 2.0 ** -21:
                assert int(d.kept[r]) == kept == int(c.kept[r])
                if near_u >= 2.0 ** -21:
                    assert int(d.tokens[r]) == tok
            assert ref.log_close(float(c.stats[r, 1]), lz) or int(d.kept[r]) != kept
