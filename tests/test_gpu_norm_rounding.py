"""Codes and scales of the residual RMS norm, element by element, against exact arithmetic: products
that are exact, and products next to the formats' midpoints."""
from fractions import Fraction
from math import isqrt

import numpy as np
import pytest
import torch

import head_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMTS = [S.SPEC_MX_E2M1, S.SPEC_MX_E4M3]
BF16, F32 = torch.bfloat16, torch.float32


def magnitudes(fmt):
    return ref.code_values(fmt)[:(8 if fmt == ref.E2M1 else 127)]


def block_codes(y, fmt):
    """Scale byte and codes of one block of Fractions: the least scale that fits, each element the
    nearest value, a tie the even code."""
    vals = [Fraction(float(v)) for v in magnitudes(fmt)]
    mids = [(a + b) / 2 for a, b in zip(vals, vals[1:])]
    amax, e = max(map(abs, y)), -127
    while amax > vals[-1] * Fraction(2) ** e:
        e += 1
    codes = []
    for v in y:
        a = abs(v) / Fraction(2) ** e
        lo, hi = 0, len(mids)       # number of midpoints that a passes
        while lo < hi:
            m = (lo + hi) // 2
            if a > mids[m] or (a == mids[m] and m % 2 == 1):
                lo = m + 1
            else:
                hi = m
        codes.append(lo + (len(vals) + (fmt == ref.E4M3) if v < 0 else 0))
    return e + 127, codes


def exact(h, w, root, fmt):
    """Bytes [rows, K / 32] and codes [rows, K] of h * root[row] * w, for K a multiple of 32."""
    rows, K = h.shape
    byte, code = np.zeros((rows, K // 32), int), np.zeros((rows, K), int)
    hw = [[Fraction(float(a)) * Fraction(float(b)) for a, b in zip(r, w)] for r in h]
    for r in range(rows):
        for b in range(K // 32):
            at = slice(32 * b, 32 * b + 32)
            byte[r, b], code[r, at] = block_codes([v * root[r] for v in hw[r][at]], fmt)
    return byte, code


def stored(q, K):
    """The same of an MXTensor; codes of zeros without their sign."""
    c, s = q.codes.cpu().numpy().astype(int), q.scales.cpu().numpy().astype(int)
    if q.fmt == ref.E2M1:
        c = np.stack([c & 15, c >> 4], 2).reshape(q.rows, -1)
    c = np.where(c == (8 if q.fmt == ref.E2M1 else 128), 0, c)[:, :K]
    r, k = np.arange(q.rows)[:, None], np.arange(K // 32)[None, :]
    return s[r // 128, k // 4, r % 32, r % 128 // 32, k % 4], c


def assert_same(q, byte, code):
    sign = 8 if q.fmt == ref.E2M1 else 128
    got_byte, got = stored(q, code.shape[1])
    np.testing.assert_array_equal(got_byte, byte)
    np.testing.assert_array_equal(got, np.where(code == sign, 0, code))


def border_weights(fmt, K, scale):
    """Blocks of the format's largest value, its midpoints and its values, times `scale`; a last
    block whose largest is one step of bf16 above the largest value (so that its scale is twice)."""
    v = magnitudes(fmt)
    pts = np.concatenate([(v[1:] + v[:-1]) / 2, v])
    w = np.zeros((K // 32, 32))
    at = 0
    for b in range(K // 32):
        w[b, 0] = v[-1]
        for i in range(1, 32):
            w[b, i] = pts[at % len(pts)] * (1 if at % 3 else -1)
            at += 1
    w[-1, 0] = v[-1] + 2.0 ** (np.floor(np.log2(v[-1])) - 7)
    return w.reshape(-1) * scale


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt,wdt", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("K", [32, 512, 992, 9216])
def test_exact_products(K, dt, wdt, fmt):
    """eps = 0 and rows of one power of two: 1 / rms is one too, and every product is a number of
    eight bits. Blocks whose largest product is the format's largest value keep the least scale,
    ties go to the even code."""
    n = [0, 2, -7, 30, -30]
    rng = np.random.default_rng(K)
    sign = rng.choice([-1.0, 1.0], (len(n), K))
    h = sign * 2.0 ** np.array(n)[:, None]
    w = border_weights(fmt, K, 2.0 ** -2)
    x = torch.from_numpy(h).to(dt)
    half = x / 2                                     # x + residual = h, exactly
    wt = torch.from_numpy(w).to(wdt)
    assert (wt.double().numpy() == w).all()
    byte, code = exact(h, w, [Fraction(2) ** -e for e in n], fmt)
    for args in (dict(x=x, res=None), dict(x=half, res=half)):
        res = None if args["res"] is None else args["res"].to(DEV)
        _, q = S.spec_rmsnorm_mx(args["x"].to(DEV), wt.to(DEV), 0.0, residual=res, fmt=fmt)
        assert_same(q, byte, code)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt,wdt", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("root,K", [(3, 288), (5, 800), (15, 7200), (21, 14112)])
def test_exact_odd_roots(root, K, dt, wdt, fmt):
    """K / root^2 ones in a row of zeros: 1 / rms = root, an odd number."""
    ones = K // root ** 2
    h = np.zeros((2, K))
    h[0, :ones] = 1.0
    h[1, K - ones:] = -4.0
    v = magnitudes(fmt)
    pts = np.concatenate([(v[1:] + v[:-1]) / 2, v])
    pts = pts[(pts / root * 2 ** 9) % 1 == 0]        # w = pts / root has a few bits
    w = np.resize(pts / root, K)
    w[::7] = 2.0 * v[1]
    wt = torch.from_numpy(w).to(wdt)
    assert (wt.double().numpy() == w).all()
    byte, code = exact(h, w, [Fraction(root), Fraction(root, 4)], fmt)
    _, q = S.spec_rmsnorm_mx(torch.from_numpy(h).to(dt).to(DEV), wt.to(DEV), 0.0, fmt=fmt)
    assert_same(q, byte, code)


@pytest.mark.parametrize("fmt", FMTS)
def test_exact_root_of_other_elements(fmt):
    """Rows with rms 2 whose elements are not powers of two, fp32 weights of 24 bits that bring
    them to within 2^-24 of a midpoint, or onto it."""
    h = np.array([5, 5, 2, 2, 1, 1, 1, 1, 1, 1, 0, 0, 0, 0, 0, 0] * 2, float)  # sum of squares 128
    h = np.tile(h, 8)
    v = magnitudes(fmt)
    mid = (v[1:] + v[:-1]) / 2
    w = np.zeros(h.size)
    for i in range(h.size):
        if h[i]:
            w[i] = np.float32(mid[(7 * i) % len(mid)] * 2 / h[i])
    w[::32] = np.float32(v[-1] * 2 / 5)
    root = [Fraction(1, 2)]
    byte, code = exact(h[None], w, root, fmt)
    for dt in (F32, BF16):
        _, q = S.spec_rmsnorm_mx(torch.from_numpy(h[None]).to(dt).to(DEV),
                                 torch.from_numpy(w).float().to(DEV), 0.0, fmt=fmt)
        assert_same(q, byte, code)


# ------------------------------------------------------------------------------ rounded once

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", [96, 992, 4096, 9216])
def test_products_next_to_midpoints(K, dt, fmt):
    """Rows of small whole numbers, whose sum of squares is exact in fp32, with an irrational root:
    1 / rms is known to 2^-44 (the pair's Newton step and its sums). The weights are the fp32
    numbers that bring every product to within 2^-24 of a midpoint of the format, where a product
    rounded to fp32 first lands on the midpoint and the tie may go the wrong way."""
    rng = np.random.default_rng(K + fmt)
    h = rng.integers(1, 4, K).astype(float)
    total = int((h * h).sum())
    assert total < 2 ** 24 and isqrt(total * K) ** 2 != total * K
    root = Fraction(isqrt(2 ** 240 * K * total), 2 ** 120 * total)  # sqrt(K / total) to 2^-110
    v = magnitudes(fmt)
    mid = (v[1:] + v[:-1]) / 2
    sign = rng.choice([-1.0, 1.0], K)
    w = np.zeros(K)
    for i in range(K):
        at = v[-1] * 0.97 if i % 32 == 0 else mid[rng.integers(len(mid))] * sign[i]
        w[i] = np.float32(at / (h[i] * float(root)))
    byte, code = exact(h[None], w, [root], fmt)
    # none within the root's error of a midpoint, so every code is decided
    a = h * np.abs(w) * float(root) / 2.0 ** (np.repeat(byte[0], 32) - 127.0)
    close = mid[np.abs(a[:, None] / mid - 1).argmin(1)]
    near = min(abs(Fraction(x) * Fraction(abs(y)) * root / Fraction(2) ** int(e - 127) /
                   Fraction(m) - 1)
               for x, y, e, m in zip(h, w, np.repeat(byte[0], 32), close))
    assert near > Fraction(1, 2 ** 42)
    _, q = S.spec_rmsnorm_mx(torch.from_numpy(h[None]).to(dt).to(DEV),
                             torch.from_numpy(w).float().to(DEV), 0.0, fmt=fmt)
    assert_same(q, byte, code)


# 1 / rms from a sum in fp32 within a thread and a warp. A square passes at most 4 roundings in its
# thread's chain, 1 that joins two chains, 5 in its warp and, in rows above 8192, 1 of the thread's
# pair; across warps the sum is exact to 2^-42. The root halves the relative error of the sum.
NORM_REL = (0.5 * 11 + 0.01) * ref.U32


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt,wdt", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("rows,K", [(300, 96), (200, 992), (130, 4096), (64, 8192), (9, 16384)])
def test_codes_of_random_rows(rows, K, dt, wdt, fmt):
    """Codes and scales are those of the exact product, but for products that lie within the
    root's own error of a midpoint or, for the scale, of the format's largest value."""
    g = torch.Generator().manual_seed(rows + K)
    x, r = torch.randn(rows, K, generator=g).to(dt), (3 * torch.randn(rows, K, generator=g)).to(dt)
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(wdt)
    eps = float(np.float32(1e-5))
    h, q = S.spec_rmsnorm_mx(x.to(DEV), w.to(DEV), eps, residual=r.to(DEV), fmt=fmt)
    h = h.cpu().double().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w.double().numpy()
    byte, code = stored(q, K)
    # scales: the least that fits, at both ends of the error
    amax = np.abs(y).reshape(rows, -1, 32).max(2) / ref.TOP[fmt]
    lo = 127 + np.ceil(np.log2(amax * (1 - NORM_REL))).astype(int)
    hi = 127 + np.ceil(np.log2(amax * (1 + NORM_REL))).astype(int)
    assert ((lo <= byte) & (byte <= hi)).all() and (lo != hi).sum() <= 2
    # codes: the number of midpoints below, at both ends of the error
    v = magnitudes(fmt)
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(y) / 2.0 ** (np.repeat(byte, 32, 1) - 127.0)
    least, most = (np.searchsorted(mid, a * (1 + s * NORM_REL)) for s in (-1, 1))
    got = code & (7 if fmt == ref.E2M1 else 127)
    assert ((least <= got) & (got <= most)).all()
    assert (least != most).mean() < 1e-4                # and nearly all have no choice
    sign = code >= (8 if fmt == ref.E2M1 else 128)
    assert (sign == ((y < 0) & (got > 0))).all()


# ------------------------------------------------------------------------------ range of the rows

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", [40, 1000, 8192, 9000])
def test_rows_whose_squares_leave_fp32(K, dt, fmt):
    """Rows of 1e-38 to 1e38, one large element among small ones, and an eps of their size."""
    g = torch.Generator().manual_seed(K)
    base = torch.randn(12, K, generator=g)
    base = base.clamp(-3, 3) + 0.01
    size = torch.tensor([1e38, 1e30, 3e19, 1.5e19, 1e-12, 1e-16, 1e-20, 1e-25, 1e-30, 1e-36, 1.0,
                         1e-37])[:, None]
    x = (base * size).to(dt)
    x[8, 1:] *= 1e-6                                 # one element of 1e-30, the others far below
    x[3, K // 2] = 2e38
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(dt)
    assert torch.isfinite(x).all()
    for eps in (0.0, float(np.float32(1e-34)), float(np.float32(1e-6)), 1e30):
        # further rows would have products below fp32's normal range
        rows = x if eps == 0 else x[:6] if eps > 1 else x[:8]
        ws = S.Workspace(256, device=DEV)
        _, q = S.spec_rmsnorm_mx(rows.to(DEV), w.to(DEV), eps, fmt=fmt, workspace=ws)
        h = rows.double().numpy()
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + float(np.float32(eps)))
        y = y * w.double().numpy()
        got = ref.dequantize(q.codes.cpu(), q.scales.cpu(), fmt, K)
        assert np.isfinite(got).all() and ws.status() == 0
        ref.check_rounded(got, q.scales.cpu(), fmt, y, NORM_REL)


@pytest.mark.parametrize("K", [256, 9216])
def test_exact_products_of_extreme_rows(K):
    """One power of two a row, subnormals and the largest among them: the codes of its weights."""
    n = [127, 70, -55, -110, -126, -133, -149]
    h = 2.0 ** np.array(n, float)[:, None] * np.random.default_rng(1).choice([-1.0, 1.0],
                                                                             (len(n), K))
    w = border_weights(ref.E4M3, K, 0.25)
    byte, code = exact(h, w, [Fraction(2) ** -e for e in n], ref.E4M3)
    _, q = S.spec_rmsnorm_mx(torch.from_numpy(h).float().to(DEV),
                             torch.from_numpy(w).float().to(DEV), 0.0)
    assert_same(q, byte, code)


@pytest.mark.parametrize("K", [256, 9216])
def test_rows_without_a_scale(K):
    """A row of zeros is 0 with any eps above 0 and NaN without; rows beside it are not touched by
    its second sum, nor by that of rows with a NaN or an infinity."""
    x = torch.randn(6, K, generator=torch.Generator().manual_seed(3))
    x[1] = 0.0
    x[2, 5], x[3, 7], x[4, 9] = float("nan"), float("inf"), -float("inf")
    x[5] *= 1e30
    for eps, zero in ((0.0, False), (1e-45, True), (1e-33, True)):
        ws = S.Workspace(256, device=DEV)
        _, q = S.spec_rmsnorm_mx(x.to(DEV), torch.ones(K, device=DEV), eps, workspace=ws)
        y = S.spec_mx_dequantize(q, dtype=torch.float32, workspace=ws).cpu()
        assert torch.isnan(y[2:5]).all() and torch.isfinite(y[[0, 5]]).all()
        assert (y[1] == 0).all() if zero else torch.isnan(y[1]).all()
        assert ws.status() == S.SPEC_DEV_NONFINITE


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [288, 9216])
@pytest.mark.parametrize("wdt", [F32, BF16])
def test_products_beyond_fp32(K, wdt, fmt):
    """Finite rows and weights whose product passes fp32's largest number: that block is NaN, those
    beside it are not."""
    x = torch.zeros(2, K)
    x[0, :32 * (K // 288)] = 1.0                     # 1 / rms = 3
    x[1] = torch.randn(K, generator=torch.Generator().manual_seed(1)).clamp(-2, 2)
    x[1, 40] = 2.0
    w = torch.ones(K)
    w[[5, 40]] = torch.tensor([1.2e38, 2.5e38])
    ws = S.Workspace(256, device=DEV)
    _, q = S.spec_rmsnorm_mx(x.to(DEV), w.to(wdt).to(DEV), 0.0, fmt=fmt, workspace=ws)
    h, w64 = x.double().numpy(), w.to(wdt).double().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True)) * w64
    bad = (np.abs(y) >= 2.0 ** 128).reshape(2, -1, 32).any(2)
    assert bad[0, 0] and bad[1, 1] and bad.sum() <= 3
    np.testing.assert_array_equal(stored(q, K)[0] == 255, bad)
    assert ws.status() == S.SPEC_DEV_NONFINITE
