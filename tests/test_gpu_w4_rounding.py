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
