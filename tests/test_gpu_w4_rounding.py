"""What is rounded to bf16 is the product of the rows as they are, not of rows of fewer bits."""
import pytest
import torch

import w4_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S
from test_gpu_w4 import BF, DEV, F32, packed, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["norm", "wide", "wide norm"])
@pytest.mark.parametrize("M,N,K,group", [(1, 4001, 512, 128), (8, 3000, 640, 64), (17, 999, 257, 32)])
def test_bf16_products_are_rounded_once(M, N, K, group, form):
    """Every number is the rounding of one within the fp32 sums' tolerance of the 64-bit product. Rows
    held in 11 bits move an output by some 2^-13 of it, and pass a border between two bf16 numbers in
    one output of ten."""
    w, v = packed(N, K, group, BF if group == 128 else F32, K, zeros=group == 64)
    x = randn((M, K), 1, BF if form == "norm" else F32)
    norm = (1 + randn((K,), 2, F32, 0.1)).to(BF) if "norm" in form else None
    got = S.spec_w4_logits(x.to(DEV), w, dtype=BF, eps=1e-6,
                           norm_weight=None if norm is None else norm.to(DEV)).cpu()
    _, y, mag = ref.product(x, v, K, norm, 1e-6)
    tol = ref.tolerance(K, group, mag, y, F32)
    lo, hi = ((y + s * tol).float().to(BF) for s in (-1, 1))
    assert ((got >= lo) & (got <= hi)).all(), int(((got < lo) | (got > hi)).sum())


def one_by_one(K):
    """A matrix whose row n is element n of the product's rows: code 9 there, 8 elsewhere, scale 1."""
    codes = torch.full((K, ref.padded(K)), 8, dtype=torch.uint8)
    codes[torch.arange(K), torch.arange(K)] = 9
    codes = (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()
    return S.W4Tensor(codes.to(DEV), torch.ones(K, ref.padded(K) // 128, device=DEV), 128, K)


# of a row: what is served at once, its ends, and what is scaled by its own power
LARGEST = [0.125, 0.13, 1.0, 100.0, 2047.0, 0.11, 3000.0, 1e20, 1e-30]


@pytest.mark.parametrize("K", [128, 600])
def test_small_elements_beside_a_large_one(K):
    """Each element of a 32-bit row by itself, from the largest to 2^-40 of it: two fp16 numbers, the
    second of what the first leaves times 2^12, hold it to 2^-23 of itself or 2^-38 of the largest."""
    x = 1 + torch.rand(len(LARGEST), K, generator=torch.Generator().manual_seed(K), dtype=torch.float64)
    x *= torch.exp2(-1 - 39.0 * torch.arange(K) / K)
    x[:, 0] = 1.0
    x = (x * torch.tensor(LARGEST, dtype=torch.float64)[:, None]).float()
    y = S.spec_w4_logits(x.to(DEV), one_by_one(K)).cpu().double()
    off, most = (y - x.double()).abs(), x.double()[:, :1]
    assert (off <= torch.maximum(2.0 ** -23 * x.double(), 2.0 ** -38 * most)).all()
    # normalised: a square root, a division and a product with the weight, each off by a rounding or two
    norm = torch.exp2(torch.randint(-2, 3, (K,), generator=torch.Generator().manual_seed(1)).float())
    norm[0] = 4.0
    y = S.spec_w4_logits(x.to(DEV), one_by_one(K), norm_weight=norm.to(DEV), eps=0.0).cpu().double()
    a = x.double() * norm.double()
    a /= x.double().square().mean(1, keepdim=True).sqrt()
    assert ((y - a).abs() <= torch.maximum(2.0 ** -23 * a, 2.0 ** -38 * a[:, :1])
            + 8 * 2.0 ** -24 * a).all()


def test_small_elements_of_bf16_rows():
    """One fp16 number each: exact from 2^-18 of the largest on, within 2^-26 of it below."""
    K = 384
    x = 1 + torch.rand(len(LARGEST), K, generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    x *= torch.exp2(-1 - 29.0 * torch.arange(K) / K)
    x[:, 0] = 1.0
    x = (x * torch.tensor(LARGEST, dtype=torch.float64)[:, None]).to(BF)
    for dt in (F32, BF):
        y = S.spec_w4_logits(x.to(DEV), one_by_one(K), dtype=dt).cpu().double()
        off, most = (y - x.double()).abs(), x.double()[:, :1]
        exact = x.double() >= 2.0 ** -18 * most
        assert (off[exact] == 0).all()
        rounded = 2.0 ** -8 * y if dt == BF else 0.0
        assert (off <= 2.0 ** -26 * most + rounded).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size", [3.3e38, 2e38, 1.7e38, 8e37, 1e-36, 1e-38, 1e-40, 9.2e-41])
def test_rows_of_any_size_without_a_norm(size, dt):
    """Finite rows up to the largest number and down to subnormals, against scales that bring the
    product back, with a row of the matrix whose product is 0."""
    K, group = 256, 128
    x = torch.rand(3, K, generator=torch.Generator().manual_seed(1)) * 2 - 1
    x[:, 0] = 1.0
    x[1] = 0.0
    x[2, 200] = -1.0
    x = (x.double() * size).to(dt)
    codes, scales = ref.pack(randn((40, K), 2, F32), group, F32)
    codes[7], scales = 0x88, scales * (2.0 ** -100 if size > 1 else 2.0 ** 80)
    w = S.W4Tensor(codes.to(DEV), scales.to(DEV), group, K)
    v = ref.values(codes, scales, group, K)
    ws = S.Workspace(device=DEV)
    for out in (F32, BF):
        y = S.spec_w4_logits(x.to(DEV), w, dtype=out, workspace=ws).cpu().double()
        _, want, mag = ref.product(x, v, K)
        assert ws.status() == 0 and (y[:, 7] == 0).all() and (y[1] == 0).all()
        # without the floor of 1e-37 that ref.tolerance adds: it is far above some of these
        tol = ref.tolerance(K, group, mag, want, out, dt == BF) - 1e-37
        assert ((y - want).abs() <= tol).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_normalised_rows_of_any_size_and_weights(eps, dt):
    """Rows to both ends of their type, weights whose products with them are small or large."""
    K, group = 256, 64
    x = torch.rand(6, K, generator=torch.Generator().manual_seed(3)) * 2 - 1
    x[:, 5] = 1.0
    sizes = torch.tensor([3.3e38, 1.7e38, 1.0, 1e-30, 1e-38, 1e-40], dtype=torch.float64)
    x = (x.double() * sizes[:, None]).to(dt)
    codes, scales = ref.pack(randn((40, K), 4, F32), group, F32)
    for wp in (-99, -60, 0, 60, 99):
        norm = ((1 + randn((K,), 5, F32, 0.1)) * 2.0 ** wp).to(dt)
        a = x.double().square().mean(1, keepdim=True)
        a = x.double() / (a + eps).sqrt() * norm.double()
        # products of about 1, or as near as 2^80 brings them
        s = (scales.double() * 2.0 ** min(80, -wp)).float()
        w = S.W4Tensor(codes.to(DEV), s.to(DEV), group, K)
        v = ref.values(codes, s, group, K)
        ws = S.Workspace(device=DEV)
        y = S.spec_w4_logits(x.to(DEV), w, norm_weight=norm.to(DEV), eps=eps, dtype=F32,
                             workspace=ws).cpu().double()
        want, mag = a @ v.t(), a.abs() @ v.abs().t()
        # without the floor, but for a rounding or two of subnormal numbers
        tol = ref.tolerance(K, group, mag, want, F32) - 1e-37 + 2.0 ** -148
        assert ws.status() == 0
        assert ((y - want).abs() <= tol).all(), wp
