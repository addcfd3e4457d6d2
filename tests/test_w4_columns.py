"""Operands and outputs of the 4-bit product that are columns of one wide buffer: apart they are taken, as
the other calls take them, and refused where they meet."""
import ctypes

import pytest
import torch

import w4_ref as ref
from test_w4_abi import MUL, S, changed  # noqa: F401  (S is a fixture)

vp = ctypes.c_void_p


@pytest.mark.parametrize("at", [
    # x in columns 0 .. 63 of 0x10000, residual_out in columns that reach into them, or into the next row
    dict(res=vp(0x40000), ldx=128, ldh=128, ro=vp(0x10000 + 2 * 63)),
    dict(res=vp(0x40000), ldx=128, ldh=128, ro=vp(0x10000 + 2 * 65)),
    dict(res=vp(0x40000), ldx=127, ldh=127, ro=vp(0x10000 + 2 * 64)),
    dict(res=vp(0x40000), ldx=128, ldh=128, ro=vp(0x10000 - 2 * 63)),
    dict(res=vp(0x40000), ldx=128, ldh=256, ro=vp(0x10000 + 2 * 64)),
    # a fp32 out of 32 columns, in the bytes of 64
    dict(ldx=128, odt=0, ldo=64, out=vp(0x10000 + 2 * 62)),
    dict(ldx=128, odt=0, ldo=64, out=vp(0x10000 + 2 * 66)),
    dict(M=1, ldx=128, ldo=128, out=vp(0x10000 + 2 * 40)),
    dict(ldx=96, ldo=128, out=vp(0x10000 + 2 * 64))])
def test_columns_that_meet_are_refused(S, at):  # noqa: F811
    assert S.lib().spec_w4_logits(*changed(MUL, at)) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("order", [(0, 1, 2, 3), (3, 1, 0, 2), (2, 3, 1, 0)])
@pytest.mark.parametrize("M", [1, 2, 25])
def test_columns_of_one_buffer(M, order):
    from draft_sampling_verification_markov_gb300 import spec
    K, N, dev = 200, 120, "cuda:0"
    g = torch.Generator().manual_seed(M)
    codes, scales = ref.pack(torch.randn(N, K, generator=g), 128, torch.bfloat16)
    w = spec.W4Tensor(codes.to(dev), scales.to(dev), 128, K)
    wide = torch.randn(M, 4 * K + 6, generator=g).to(torch.bfloat16).to(dev)
    x, res, hid, out = (wide[:, 3 + K * i:3 + K * (i + 1)] for i in order)
    out = out[:, 40:40 + N]
    x0, r0, before = x.clone(), res.clone(), wide.clone()
    want = spec.spec_w4_logits(x0, w, residual=r0)
    h, y = spec.spec_w4_logits(x, w, residual=res, residual_out=hid, out=out)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    hid.copy_(before[:, 3 + K * order[2]:3 + K * (order[2] + 1)])
    out.copy_(before[:, 3 + K * order[3] + 40:3 + K * order[3] + 40 + N])
    assert torch.equal(wide, before)
