"""Grouped 4-bit weights on the GPU against 64 bits: packing, reading back, products."""
import threading
import time

import pytest
import torch

import w4_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, dtype, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def packed(N, K, group, sdt, seed, zeros=False):
    """(W4Tensor on the device, its values in 64 bits)."""
    codes, scales = ref.pack(randn((N, K), seed, F32, K ** -0.5), group, sdt)
    z = None
    if zeros:
        z = torch.randint(0, 128, scales.shape, dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(seed + 1))
    w = S.W4Tensor(codes.to(DEV), scales.to(DEV), group, K, zeros=None if z is None else z.to(DEV))
    return w, ref.values(codes, scales, group, K, z)


def check(x, w, values, dtype=None, norm=None, eps=1e-6, residual=None):
    ws = S.Workspace(device=DEV)

    def dev(t):
        return None if t is None else t.to(DEV)
    r = S.spec_w4_logits(x.to(DEV), w, norm_weight=dev(norm), eps=eps, residual=dev(residual),
                         dtype=dtype, workspace=ws)
    assert ws.status() == 0
    h, y, mag = ref.product(x, values, w.K, norm, eps, residual)
    if residual is not None:
        assert torch.equal(r[0].cpu(), h)
        r = r[1]
    assert r.dtype == (dtype or x.dtype)
    off = (r.cpu().double() - y).abs()
    tol = ref.tolerance(w.K, w.group, mag, y, r.dtype, x.dtype == BF and norm is None)
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("sdt", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,K,group", [(1, 1, 128), (3, 31, 32), (5, 129, 64), (2, 1000, 32),
                                          (130, 384, 128), (7, 4096, 64), (1001, 257, 128)])
def test_pack(rows, K, group, dt, sdt):
    x = randn((rows, K), rows + K, dt) * torch.exp2(randn((rows, 1), 3, F32, 8.0)).to(dt)
    x[0, 0] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2, :] = x[2, 0]
    codes, scales = ref.pack(x, group, sdt)
    ws = S.Workspace(device=DEV)
    q = S.spec_w4_quantize(x.to(DEV), group, scale_dtype=sdt, workspace=ws)
    assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes.cpu(), codes)
    v = ref.values(codes, scales, group, K)
    for out in (BF, F32):
        assert torch.equal(S.spec_w4_dequantize(q, dtype=out).cpu(),
                           v.float().to(out) if sdt == BF else v.to(out))
    assert ws.status() == 0


def test_pack_ties_and_extremes():
    """Quotients on the middle between two codes, subnormal groups, the largest numbers."""
    half = torch.arange(-13, 14).float() / 2                       # of a scale of 1
    x = torch.zeros(6, 32)
    x[0, :27], x[0, 27] = half, 7.0
    x[1, :27], x[1, 27] = half * 3, 21.0
    x[2, :4] = torch.tensor([1e-45, -4e-45, 3e-45, 0.0])
    x[3, :3] = torch.tensor([3.4e38, -1.7e38, 1e38])
    x[4, :3] = torch.tensor([1.17549435e-38, 5e-39, -8e-39])
    x[5, 0] = -0.0
    for sdt in (BF, F32):
        codes, scales = ref.pack(x, 32, sdt)
        q = S.spec_w4_quantize(x.to(DEV), 32, scale_dtype=sdt)
        assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes.cpu(), codes)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("power", [-130, -100, -99, 0, 60, 124])
def test_pack_quotients_in_the_middle(power, dt):
    """Multiples of a quarter or a 32nd: many quotients are halves, at sizes where the reciprocal is
    taken, where it is not, and at the largest."""
    g = torch.Generator().manual_seed(power + 200)
    x = torch.cat([torch.randint(-28, 29, (64, 512), generator=g) / 4.0,
                   torch.randint(-112, 113, (64, 512), generator=g) / 32.0,
                   torch.randn(64, 512, generator=g)]).clamp_(-7, 7)
    x = torch.ldexp(x.double(), torch.tensor(power)).to(dt)
    for sdt in (BF, F32):
        codes, scales = ref.pack(x, 32, sdt)
        q = S.spec_w4_quantize(x.to(DEV), 32, scale_dtype=sdt)
        assert torch.equal(q.scales.cpu(), scales)
        assert torch.equal(q.codes.cpu(), codes)
        for odt in (BF, F32):
            y = S.spec_w4_dequantize(q, dtype=odt)
            assert torch.equal(y.cpu(), ref.values(codes, scales, 32, 512).to(odt))


def test_read_back_rounds_once():
    """fp32 scales: a bf16 value is the product's own rounding, not that of its fp32 form."""
    g = torch.Generator().manual_seed(4)
    scales = torch.randint(1 << 23, 1 << 24, (1 << 16, 4), generator=g).float()
    codes = torch.randint(0, 256, (1 << 16, 64), generator=g).to(torch.uint8)
    zeros = torch.randint(0, 128, scales.shape, generator=g).to(torch.uint8)
    q = S.W4Tensor(codes.to(DEV), scales.to(DEV), 32, 128, zeros=zeros.to(DEV))
    v = ref.values(codes, scales, 32, 128, zeros).long()  # whole numbers of up to 31 bits
    mag = v.abs()
    step = torch.ones_like(mag)
    for _ in range(23):                                   # a bf16 number has 8 bits
        step = torch.where(mag >= 256 * step, 2 * step, step)
    n, rest = mag // step, mag % step
    n = n + ((2 * rest > step) | ((2 * rest == step) & (n % 2 == 1))).long()
    want = (n * step * v.sign()).double()
    assert torch.equal(S.spec_w4_dequantize(q).cpu().double(), want)


def test_pack_without_meaning_and_strides():
    x = randn((4, 300), 5, F32)
    x[1, 40], x[2, 299] = float("inf"), float("nan")
    wide = torch.zeros(4, 331)
    wide[:, 7:307] = x
    ws = S.Workspace(device=DEV)
    q = S.spec_w4_quantize(wide.to(DEV)[:, 7:307], 32, workspace=ws)
    assert ws.status() == S.SPEC_DEV_NONFINITE
    nan = torch.isnan(q.scales.cpu().float())
    assert nan.nonzero().tolist() == [[1, 1], [2, 9]]
    out = torch.full((4, 340), 5.0, device=DEV)
    S.spec_w4_dequantize(q, out=out[:, 3:303])
    ok = torch.isfinite(x)
    ok[1, 32:64] = ok[2, 288:300] = False
    codes, scales = ref.pack(torch.where(ok, x, 0.0), 32, BF)
    v = ref.values(codes, scales, 32, 300).float()
    assert torch.equal(out.cpu()[:, 3:303][ok], v[ok])
    assert torch.isnan(out.cpu()[:, 3:303][~ok]).all()
    assert (out[:, :3] == 5.0).all() and (out[:, 303:] == 5.0).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 17, 128), (2, 40, 100), (3, 515, 1000),
                                   (8, 1000, 384), (9, 300, 4096), (17, 700, 640), (33, 129, 257),
                                   (1, 20000, 512), (5, 9001, 256)])
def test_shapes(M, N, K, group, norm, dt):
    w, v = packed(N, K, group, BF if group == 128 else F32, M + N + K, zeros=group == 64)
    x = randn((M, K), 1, dt)
    if norm:
        check(x, w, v, norm=(1 + randn((K,), 2, F32, 0.1)).to(dt), residual=randn((M, K), 3, dt, 4.0))
    else:
        check(x, w, v)


@pytest.mark.parametrize("M", [1, 2, 4, 8, 10, 11, 16, 24, 32, 40])
@pytest.mark.parametrize("form", ["plain", "norm", "wide"])
def test_rows(M, form):
    """Every number of column tiles and chunks."""
    w, v = packed(1234, 512, 128, BF, M)
    x = randn((M, 512), 4, F32 if form == "wide" else BF)
    check(x, w, v, norm=None if form == "plain" else (1 + randn((512,), 5, F32, 0.1)).to(x.dtype))


@pytest.mark.parametrize("K,dt", [(8192, F32), (16384, BF), (36864, F32)])
def test_wide_rows(K, dt):
    w, v = packed(48, K, 64, F32, K, zeros=True)
    check(randn((7, K), 6, dt), w, v, norm=randn((K,), 7, F32), dtype=F32)
    with pytest.raises(S.SpecError) as e:
        big = S.W4Tensor.empty(4, 36865, 64, F32, DEV)
        S.spec_w4_logits(torch.zeros(1, 36865, device=DEV), big)  # a fp32 product
    assert e.value.status == S.SPEC_ERR_TOO_LARGE


def test_mixed_types():
    w, v = packed(300, 640, 32, F32, 9)
    x = randn((3, 640), 10, BF)
    check(x, w, v, dtype=F32, norm=1 + randn((640,), 11, F32, 0.1))
    check(x, w, v, dtype=F32)
    check(x.float(), w, v, dtype=BF, norm=(1 + randn((640,), 11, F32, 0.1)).to(BF))
    check(x, w, v, dtype=F32, residual=randn((3, 640), 12, BF))


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_any_size_are_normalised(dt):
    """Squares beyond fp32's range on both sides, and eps where it matters."""
    w, v = packed(64, 256, 128, F32, 13)
    x = randn((6, 256), 14, F32)
    x = (x * torch.tensor([1e37, 1e-36, 1e19, 1e-25, 1.0, 3e-4])[:, None]).to(dt)
    g = (1 + randn((256,), 15, F32, 0.1)).to(dt)
    check(x, w, v, norm=g, eps=0.0, dtype=F32)
    check(x, w, v, norm=g, eps=1e-6, dtype=F32)


def test_rows_without_meaning():
    w, v = packed(40, 256, 128, BF, 16)
    x = randn((4, 256), 17, BF)
    x[1, 5], x[3, 200] = float("nan"), float("inf")
    for kw in ({}, dict(norm_weight=torch.ones(256, dtype=BF, device=DEV))):
        ws = S.Workspace(device=DEV)
        y = S.spec_w4_logits(x.to(DEV), w, workspace=ws, **kw).cpu()
        assert ws.status() == S.SPEC_DEV_NONFINITE
        assert torch.isfinite(y[[0, 2]]).all() and not torch.isfinite(y[[1, 3]]).any()
    y = S.spec_w4_logits(torch.zeros(2, 256, dtype=BF, device=DEV), w, eps=0.0,
                         norm_weight=torch.ones(256, dtype=BF, device=DEV))
    assert torch.isnan(y).all()


def test_scales_of_the_padding_do_not_matter():
    codes, scales = ref.pack(randn((50, 130), 18, F32), 32, F32)
    v = ref.values(codes, scales, 32, 130)
    codes[:, 65:] = 0xff
    scales[:, 5:] = float("nan")
    w = S.W4Tensor(codes.to(DEV), scales.to(DEV), 32, 130)
    check(randn((2, 130), 19, F32), w, v)


def test_strides_and_outputs():
    w, v = packed(333, 200, 64, BF, 20)
    wide, res = randn((5, 260), 21, BF), randn((5, 300), 22, BF)
    x, r = wide.to(DEV)[:, 3:203], res.to(DEV)[:, 9:209]
    out = torch.full((5, 400), 3.0, dtype=F32, device=DEV)
    hid = torch.full((5, 220), 3.0, dtype=BF, device=DEV)
    h, y = S.spec_w4_logits(x, w, residual=r, residual_out=hid[:, 1:201], out=out[:, 7:340])
    want_h, want, mag = ref.product(wide[:, 3:203], v, 200, residual=res[:, 9:209])
    assert torch.equal(h.cpu(), want_h)
    assert ((y.cpu().double() - want).abs() <= ref.tolerance(200, 64, mag, want, F32)).all()
    assert (out[:, :7] == 3.0).all() and (out[:, 340:] == 3.0).all()
    assert (hid[:, :1] == 3.0).all() and (hid[:, 201:] == 3.0).all()
    three = randn((2, 3, 200), 23, BF)
    y = S.spec_w4_logits(three.to(DEV), w)
    assert y.shape == (2, 3, 333)
    assert torch.equal(y.view(6, 333), S.spec_w4_logits(three.view(6, 200).to(DEV), w))
    assert S.spec_w4_logits(three.to(DEV)[:0], w).shape == (0, 3, 333)


def test_overlaps_are_refused():
    w, _ = packed(64, 128, 128, BF, 24)
    x = torch.zeros(2, 128, dtype=BF, device=DEV)
    for kw in (dict(residual=torch.zeros_like(x), residual_out=x), dict(out=x[:, :64])):
        with pytest.raises(S.SpecError):
            S.spec_w4_logits(x, w, **kw)


def test_graph_and_streams():
    w, _ = packed(2000, 512, 128, BF, 25)
    x = randn((4, 512), 26, BF).to(DEV)
    want = S.spec_w4_logits(x, w)
    side, ws = torch.cuda.Stream(device=DEV), S.Workspace(256, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = S.spec_w4_logits(x, w, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out, static = torch.empty_like(want), x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.spec_w4_logits(static, w, out=out, workspace=ws)
    for seed in (27, 28):
        static.copy_(randn((4, 512), seed, BF))
        g.replay()
        assert torch.equal(out, S.spec_w4_logits(static, w))


def test_product_right_after_packing():
    """The copies see what the kernel before them wrote, call after call into the same matrix."""
    x = randn((2, 256), 41, BF).to(DEV)
    ms = [randn((3000, 256), 42 + i, BF, 0.1).to(DEV) for i in range(6)]
    want = [S.spec_w4_logits(x, S.spec_w4_quantize(m, 64)) for m in ms]
    w = S.spec_w4_quantize(ms[0], 64)
    got = []
    for m in ms * 3:
        S.spec_w4_quantize(m, 64, out=w)
        got.append(S.spec_w4_logits(x, w))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 6]), i


def test_calls_of_several_threads():
    """Forms with different shared memory, at once from several host threads on streams of their own."""
    sizes = [(1, 256), (5, 2048), (17, 4096), (40, 1024)]
    w = [packed(600, K, 128, BF, K)[0] for _, K in sizes]
    x = [randn((M, K), M, BF).to(DEV) for M, K in sizes]
    want = [S.spec_w4_logits(a, b) for a, b in zip(x, w)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        side, ws = torch.cuda.Stream(device=DEV), S.Workspace(256, device=DEV)
        out = torch.empty_like(want[i])
        side.wait_stream(torch.cuda.default_stream(torch.device(DEV)))
        for _ in range(100):
            S.spec_w4_logits(x[i], w[i], out=out, workspace=ws, stream=side)
        side.synchronize()
        if ws.status() or not torch.equal(out, want[i]):
            wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_expired_wait_reports_timeout():
    w, _ = packed(3000, 1024, 128, BF, 31)
    x = randn((3, 1024), 32, BF).to(DEV)
    ws = S.Workspace(256, device=DEV)
    want = S.spec_w4_logits(x, w, workspace=ws).clone()
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert S.lib().spec_test_stall_next_markov() == 0
    t0 = time.time()
    S.spec_w4_logits(x, w, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() & S.SPEC_DEV_TIMEOUT
    assert 0.5 < time.time() - t0 < 30.0
    assert torch.equal(S.spec_w4_logits(x, w, workspace=ws), want)
    torch.cuda.synchronize()
    assert ws.status() == 0


def test_matrix_beyond_2_31_elements():
    """Rows of the matrix whose element indexes pass 31 and 32 bits."""
    N, K = 1100000, 4096
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    w = S.W4Tensor.empty(N, K, 128, BF, DEV)
    w.codes.fill_(0x88)
    w.scales.fill_(1.0)
    rows = torch.tensor([0, 1, 524287, 524289, 1048577, N - 1], device=DEV)
    w.codes[rows] = torch.randint(0, 256, (6, K // 2), dtype=torch.uint8, device=DEV)
    x = randn((2, K), 29, BF)
    y = S.spec_w4_logits(x.to(DEV), w, dtype=F32)
    v = ref.values(w.codes[rows].cpu(), w.scales[rows].cpu(), 128, K)
    _, want, mag = ref.product(x, v, K)
    got = y[:, rows].cpu().double()
    assert ((got - want).abs() <= ref.tolerance(K, 128, mag, want, F32)).all()
    y[:, rows] = 0.0
    assert not y.any()
