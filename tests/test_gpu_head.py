"""Block-scaled quantisation, the residual RMS norm and the vocabulary product on the GPU
against their 64-bit definitions."""
import numpy as np
import pytest
import torch

import head_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMTS = [S.SPEC_MX_E2M1, S.SPEC_MX_E4M3]
DTS = [torch.bfloat16, torch.float32]


def randn(*shape, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def status(ws):
    torch.cuda.synchronize()
    return ws.status()


def random_mx(rows, K, fmt, seed):
    """A quantised matrix of rows of very different sizes."""
    x = randn(rows, K, seed=seed).double().numpy()
    x *= 2.0 ** np.random.default_rng(seed).integers(-6, 7, (rows, 1))
    codes, s = ref.quantize(x, fmt)
    return (S.MXTensor(torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), fmt, K),
            ref.dequantize(codes, s, fmt, K))


# ------------------------------------------------------------------------------ quantise

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (127, 33), (128, 128), (129, 129),
                                    (257, 1000), (5, 8192), (300, 520)])
def test_quantize_and_read_back(rows, K, dt, fmt):
    x = randn(rows, K, seed=rows * K, dtype=dt) * torch.exp2(
        randn(rows, 1, seed=7, std=6.0)).to(dt)
    x[0, 0] = 0.0
    x[rows - 1, : min(K, 32)] = 0.0
    codes, s = ref.quantize(f64(x), fmt)
    ws = S.Workspace(device=DEV)
    q = S.spec_mx_quantize(x.to(DEV), fmt, workspace=ws)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)
    for odt in DTS:
        y = S.spec_mx_dequantize(q, dtype=odt, workspace=ws)
        np.testing.assert_array_equal(f64(y), ref.dequantize(codes, s, fmt, K))
    assert status(ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rounding_borders(fmt):
    """Every midpoint between neighbouring values, and its fp32 neighbours, at scales from the
    smallest to the largest."""
    v = ref.code_values(fmt)[:(8 if fmt == ref.E2M1 else 127)]
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    pts = np.concatenate([mid, np.nextafter(mid, np.float32(0)),
                          np.nextafter(mid, np.float32(1e9)), v.astype(np.float32)])
    pts = np.concatenate([pts, -pts])
    pts = np.pad(pts, (0, -len(pts) % 31)).reshape(-1, 31)
    rows = []
    for e in (-126, -100, -3, 0, 5, 100, 118 if fmt == ref.E4M3 else 124):
        blk = np.concatenate([np.full((len(pts), 1), ref.TOP[fmt]), pts], 1)
        rows.append(blk * 2.0 ** e)
    x = np.concatenate(rows).astype(np.float32)
    codes, s = ref.quantize(x.astype(np.float64), fmt)
    q = S.spec_mx_quantize(torch.from_numpy(x).to(DEV), fmt)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_scale_borders(fmt):
    """Largest magnitudes just at, below and above the format's largest value times a power of
    two, subnormals and the type's extremes."""
    top = np.float32(ref.TOP[fmt])
    near = [top, np.nextafter(top, np.float32(0)), np.nextafter(top, np.float32(1e9))]
    big = [np.float32(a) * np.float32(2.0) ** e for a in near for e in (-120, -1, 0, 1, 60)]
    big += [np.float32(1e-45), np.float32(1.1e-38), np.float32(1e-38), np.float32(0.0)]
    x = np.zeros((len(big), 64), np.float32)
    x[:, 3] = big
    x[:, 40] = -np.array(big)
    codes, s = ref.quantize(x.astype(np.float64), fmt)
    q = S.spec_mx_quantize(torch.from_numpy(x).to(DEV), fmt)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_non_finite_block(fmt, bad):
    x = randn(3, 200, seed=1)
    x[1, 37] = bad
    ws = S.Workspace(device=DEV)
    q = S.spec_mx_quantize(x.to(DEV), fmt, workspace=ws)
    y = S.spec_mx_dequantize(q, dtype=torch.float32, workspace=ws).cpu()
    assert torch.isnan(y[1, 32:64]).all()
    y[1, 32:64] = 0
    assert torch.isfinite(y).all()
    assert status(ws) == S.SPEC_DEV_NONFINITE


def test_quantize_strided_rows_and_leading_dimensions():
    big = randn(6, 5, 300, seed=3, dtype=torch.bfloat16).to(DEV)
    for view in (big[:, 2, :200], big[:, :, 17:217], big[1:4].transpose(0, 1)[2, :, 3:],
                 big[0, 0:1]):
        x = view.reshape(-1, view.shape[-1]).contiguous()
        a, b = S.spec_mx_quantize(view, S.SPEC_MX_E4M3), S.spec_mx_quantize(x, S.SPEC_MX_E4M3)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    out = torch.zeros(30, 400, dtype=torch.bfloat16, device=DEV)
    q = S.spec_mx_quantize(big, S.SPEC_MX_E4M3)
    S.spec_mx_dequantize(q, out=out[:, 50:350])
    assert torch.equal(out[:, 50:350], S.spec_mx_dequantize(q))
    assert (out[:, :50] == 0).all() and (out[:, 350:] == 0).all()
    with pytest.raises(ValueError, match="contiguous"):
        S.spec_mx_quantize(big[0].t())
    with pytest.raises(ValueError, match="evenly"):
        S.spec_mx_quantize(big[:, :4])


def test_workspaces_named_without_an_index():
    x = randn(3, 64, seed=1).to(DEV)
    want = S.spec_mx_quantize(x)
    got = S.spec_mx_quantize(x, workspace=S.Workspace(device="cuda"))
    assert torch.equal(got.codes, want.codes)


def test_no_rows():
    q = S.spec_mx_quantize(torch.zeros(0, 64, device=DEV), S.SPEC_MX_E4M3)
    assert q.shape == (0, 64) and S.spec_mx_dequantize(q).shape == (0, 64)
    w, _ = random_mx(10, 64, S.SPEC_MX_E2M1, 1)
    assert S.spec_mx_logits(q, w).shape == (0, 10)
    h, y = S.spec_rmsnorm_mx(torch.zeros(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert h.shape == (0, 64) and y.shape == (0, 64)


# ------------------------------------------------------------------------------ norm

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt,wdt", [(torch.bfloat16, torch.bfloat16),
                                    (torch.float32, torch.float32),
                                    (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("rows,K,res", [(1, 1, True), (1, 4096, True), (3, 127, False),
                                        (130, 1000, True), (2, 33, True), (5, 2056, False),
                                        (4, 9000, True), (257, 512, True), (2, 33000, True)])
def test_norm(rows, K, res, dt, wdt, fmt):
    x, r = randn(rows, K, seed=rows + K, dtype=dt), randn(rows, K, seed=K, dtype=dt, std=3.0)
    w = 1 + randn(K, seed=2, std=0.2)
    w = w.to(wdt)
    eps = 1e-5
    ws = S.Workspace(device=DEV)
    h, q = S.spec_rmsnorm_mx(x.to(DEV), w.to(DEV), eps, residual=r.to(DEV) if res else None,
                             fmt=fmt, workspace=ws)
    want = (x.float() + r.float()).to(dt) if res else x
    assert torch.equal(h.cpu(), want)
    h64, w64 = f64(want), f64(w)
    y = h64 / np.sqrt((h64 * h64).mean(1, keepdims=True) + eps) * w64
    got = ref.dequantize(q.codes.cpu(), q.scales.cpu(), fmt, K)
    ref.check_rounded(got, q.scales.cpu(), fmt, y, ref.norm_rel(K))
    s = q.scales.cpu().numpy()
    pad = np.arange(rows, -(-rows // 128) * 128)
    assert (s[pad // 128, :, pad % 32, pad % 128 // 32] == 0).all()
    assert status(ws) == 0


@pytest.mark.parametrize("where", ["x", "residual", "strided"])
@pytest.mark.parametrize("K", [512, 300, 9000])
def test_norm_in_place_and_strided(where, K):
    both = randn(9, 2, K + 8, seed=5, dtype=torch.bfloat16).to(DEV)
    x, r = both[:, 0, :K], both[:, 1, :K]
    w = randn(K, seed=6).to(DEV)
    h0, q0 = S.spec_rmsnorm_mx(x.contiguous(), w, residual=r.contiguous())
    out = {"x": x, "residual": r,
           "strided": torch.zeros(9, K + 24, dtype=torch.bfloat16, device=DEV)[:, 8:8 + K]}[where]
    before = both.clone()
    h, q = S.spec_rmsnorm_mx(x, w, residual=r, residual_out=out)
    assert h is out and torch.equal(out, h0)
    assert torch.equal(q.codes, q0.codes) and torch.equal(q.scales, q0.scales)
    assert torch.equal(both[:, :, K:], before[:, :, K:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_non_finite_row(bad):
    x = randn(4, 300, seed=8)
    x[2, 299] = bad
    ws = S.Workspace(device=DEV)
    _, q = S.spec_rmsnorm_mx(x.to(DEV), torch.ones(300, device=DEV), workspace=ws)
    y = S.spec_mx_dequantize(q, workspace=ws).cpu()
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()
    assert status(ws) == S.SPEC_DEV_NONFINITE


def test_norm_between_rows_of_one_buffer():
    """x, residual and the stored sum as column ranges of one wide buffer."""
    wide = randn(7, 3, 264, seed=12, dtype=torch.bfloat16).to(DEV)
    x, r, o = wide[:, 0], wide[:, 1], wide[:, 2]
    w = randn(264, seed=6).to(DEV)
    h0, q0 = S.spec_rmsnorm_mx(x.clone(), w, residual=r.clone())
    _, q = S.spec_rmsnorm_mx(x, w, residual=r, residual_out=o)
    assert torch.equal(o, h0) and torch.equal(q.codes, q0.codes)
    shifted = wide.as_strided((6, 264), (792, 1), 8)  # eight elements into x's columns
    with pytest.raises(S.SpecError):
        S.spec_rmsnorm_mx(x[:6], w, residual=r[:6], residual_out=shifted)


def test_norm_zero_row():
    x = torch.zeros(2, 256, device=DEV)
    _, q = S.spec_rmsnorm_mx(x, torch.ones(256, device=DEV), 1e-6)
    assert (S.spec_mx_dequantize(q) == 0).all()


# ------------------------------------------------------------------------------ product

def check_logits(out, a64, w64, K, dt):
    """Products of codes are exact; the sum of K of them takes at most one unit of fp32
    (2 * U32, whichever way an addition rounds) of the running magnitude an addition, then the
    output's own rounding."""
    want = a64 @ w64.T
    mag = np.abs(a64) @ np.abs(w64).T
    tol = (K + 4) * 2 * ref.U32 * mag
    if dt == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    else:
        tol = tol + np.abs(want) * ref.U32
    assert (np.abs(f64(out) - want) <= tol + 1e-300).all(), np.max(np.abs(f64(out) - want) - tol)


@pytest.mark.parametrize("M,V,K", [(1, 1, 1), (1, 128, 128), (3, 127, 31), (16, 129, 129),
                                   (17, 1000, 256), (33, 300, 1000), (100, 255, 384),
                                   (128, 640, 520), (129, 257, 128), (240, 130, 256),
                                   (257, 1111, 640), (500, 384, 2048), (1, 20000, 512),
                                   (64, 5000, 1024), (1000, 2500, 256)])
@pytest.mark.parametrize("dt", DTS)
def test_logits(M, V, K, dt):
    a, a64 = random_mx(M, K, S.SPEC_MX_E4M3, M + K)
    w, w64 = random_mx(V, K, S.SPEC_MX_E2M1, V + K)
    ws = S.Workspace(device=DEV)
    out = S.spec_mx_logits(a, w, dtype=dt, workspace=ws)
    assert status(ws) == 0
    check_logits(out, a64, w64, K, dt)


@pytest.mark.parametrize("af", FMTS)
@pytest.mark.parametrize("wf", FMTS)
@pytest.mark.parametrize("M,V,K", [(5, 300, 300), (300, 520, 256)])
def test_logits_formats(M, V, K, af, wf):
    a, a64 = random_mx(M, K, af, 1)
    w, w64 = random_mx(V, K, wf, 2)
    check_logits(S.spec_mx_logits(a, w, dtype=torch.float32), a64, w64, K, torch.float32)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V", [256, 301])
@pytest.mark.parametrize("M", [6, 300])
def test_logits_into_a_position_and_odd_strides(M, V, dt):
    a, _ = random_mx(M, 256, S.SPEC_MX_E4M3, 3)
    w, _ = random_mx(V, 256, S.SPEC_MX_E2M1, 4)
    want = S.spec_mx_logits(a, w, dtype=dt)
    U = torch.full((M, 3, V), 7.0, dtype=dt, device=DEV)
    S.spec_mx_logits(a, w, out=U[:, 1])
    assert torch.equal(U[:, 1], want) and (U[:, 0] == 7).all() and (U[:, 2] == 7).all()
    wide = torch.full((M, V + 5), 7.0, dtype=dt, device=DEV)
    S.spec_mx_logits(a, w, out=wide[:, 1:V + 1])
    assert torch.equal(wide[:, 1:V + 1], want)
    assert (wide[:, 0] == 7).all() and (wide[:, V + 1:] == 7).all()


@pytest.mark.parametrize("M", [5, 300])
def test_logits_nan_scales_and_zero_blocks(M):
    a, _ = random_mx(M, 256, S.SPEC_MX_E4M3, 5)
    w, _ = random_mx(300, 256, S.SPEC_MX_E2M1, 6)
    x = randn(M, 256, seed=9)
    x[3, 40] = float("nan")
    a = S.spec_mx_quantize(x.to(DEV), S.SPEC_MX_E4M3)
    y = randn(300, 256, seed=10)
    y[200, 7] = float("inf")
    y[77] = 0.0
    w = S.spec_mx_quantize(y.to(DEV), S.SPEC_MX_E2M1)
    out = S.spec_mx_logits(a, w, dtype=torch.float32).cpu()
    nan = torch.zeros(M, 300, dtype=torch.bool)
    nan[3] = True
    nan[:, 200] = True
    assert torch.equal(torch.isnan(out), nan)
    assert (out[:3, 77] == 0).all()


def test_logits_extreme_scales():
    """Scales at both ends of their range meet scales that bring the product back."""
    a, w = np.ones((4, 64)), np.ones((130, 64))
    a[0], a[1], w[3], w[129] = 2.0 ** -120, 2.0 ** 110, 2.0 ** 118, 2.0 ** -115
    qa, qw = ref.quantize(a, ref.E4M3), ref.quantize(w, ref.E2M1)
    ta = S.MXTensor(*(torch.from_numpy(t).to(DEV) for t in qa), ref.E4M3, 64)
    tw = S.MXTensor(*(torch.from_numpy(t).to(DEV) for t in qw), ref.E2M1, 64)
    out = f64(S.spec_mx_logits(ta, tw, dtype=torch.float32))
    with np.errstate(over="ignore"):
        want = (a @ w.T).astype(np.float32).astype(np.float64)
    np.testing.assert_array_equal(out, want)


def test_logits_refuses_mismatched_operands():
    a, _ = random_mx(4, 256, S.SPEC_MX_E4M3, 5)
    w, _ = random_mx(8, 128, S.SPEC_MX_E2M1, 6)
    with pytest.raises(ValueError, match="elements"):
        S.spec_mx_logits(a, w)
    w, _ = random_mx(8, 256, S.SPEC_MX_E2M1, 6)
    with pytest.raises(ValueError, match="rows"):
        S.spec_mx_logits(a, w, out=torch.zeros(4, 9, device=DEV))
    with pytest.raises(TypeError):
        S.spec_mx_logits(a, w, dtype=torch.float16)


def test_arrays_beyond_two_to_the_31_elements():
    """Logits of 17000 rows over 129280 tokens, quantised and read back: last rows against the
    definitions."""
    M, V, K = 17000, 129280, 128
    a, a64 = random_mx(M, K, S.SPEC_MX_E4M3, 1)
    w, w64 = random_mx(V, K, S.SPEC_MX_E2M1, 2)
    ws = S.Workspace(device=DEV)
    out = S.spec_mx_logits(a, w, workspace=ws)
    rows = [0, 8191, M - 130, M - 1]
    check_logits(out[rows], a64[rows], w64, K, torch.bfloat16)
    q = S.spec_mx_quantize(out, S.SPEC_MX_E4M3, workspace=ws)
    del a, w
    x = f64(out[M - 3:])
    codes, s = ref.quantize(np.concatenate([np.zeros((M % 128 - 3, V)), x]), S.SPEC_MX_E4M3)
    np.testing.assert_array_equal(q.codes[M - 3:].cpu().numpy(), codes[-3:])
    y = S.spec_mx_dequantize(q, workspace=ws)
    np.testing.assert_array_equal(f64(y[M - 3:]),
                                  ref.dequantize(codes, s, S.SPEC_MX_E4M3, V)[-3:])
    tok = torch.full((M,), -1, dtype=torch.int32)
    tok[[5, M - 1]] = torch.tensor([7, V - 1], dtype=torch.int32)
    r = S.spec_token_logprobs(out, tok.to(DEV), 1.0, top=3, workspace=ws)
    for row in (5, M - 1):
        want = ref.token_logprobs(out[row:row + 1].cpu().double(), tok[row:row + 1], 1.0, 3)
        assert torch.equal(r.top_ids[row].cpu().long(), want["top_ids"][0])
        assert r.rank[row].item() == want["rank"].item()
        z = out[row].float()
        tol = ref.logp_tol(V, float(z.max() - z.min()))
        assert abs(r.logp[row].item() - want["logp"].item()) <= tol
    h, n = S.spec_rmsnorm_mx(out, torch.ones(V, device=DEV), residual=y, workspace=ws)
    last = h[M - 1:].double().cpu().numpy()
    want = last / np.sqrt((last ** 2).mean() + 1e-6)
    tile = n.scales[-1:].cpu()
    keep = (M - 1) % 128
    s1 = np.zeros((1,) + tuple(tile.shape[1:]), np.uint8)
    s1[0, :, 0, 0] = tile[0, :, keep % 32, keep // 32]
    got = ref.dequantize(n.codes[M - 1:].cpu(), s1, S.SPEC_MX_E4M3, V)
    ref.check_rounded(got, s1, S.SPEC_MX_E4M3, want, ref.norm_rel(V))
    assert status(ws) == 0


def test_head_chain_on_a_stream_and_in_a_graph():
    """norm -> product on a side stream and replayed from a graph with new inputs equals the
    eager run; the same calls twice in a row do not disturb each other."""
    M, V, K = 40, 700, 384
    x, r = randn(M, K, seed=1).to(DEV), randn(M, K, seed=2).to(DEV)
    x2 = randn(M, K, seed=3).to(DEV)
    w, _ = random_mx(V, K, S.SPEC_MX_E2M1, 4)
    g = torch.ones(K, device=DEV)
    ws = S.Workspace(256, device=DEV)

    def step(x):
        h, q = S.spec_rmsnorm_mx(x, g, residual=r, workspace=ws)
        return h, S.spec_mx_logits(q, w, workspace=ws)

    want, want2 = step(x), step(x2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(buf)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    buf.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want2))
    assert status(ws) == 0
