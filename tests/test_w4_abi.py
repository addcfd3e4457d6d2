"""Refusals of the grouped 4-bit weights on the host: every bad argument returns its status before
any launch."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
P, ODD, MIS = vp(0x10000), vp(0x10001), vp(0x10008)


@pytest.fixture(scope="module")
def S():
    from draft_sampling_verification_markov_gb300 import build
    build.build()
    from draft_sampling_verification_markov_gb300 import spec
    spec.lib()
    return spec


def changed(base, at):
    assert set(at) <= set(base)
    return tuple({**base, **at}.values())


PACK = dict(x=P, dt=1, ldx=64, rows=4, K=64, group=32, codes=P, scales=P, sdt=1, ws=P, wn=256,
            st=None)
BACK = dict(codes=P, scales=P, sdt=1, zeros=None, rows=4, K=64, group=64, out=P, odt=1, ldo=64,
            ws=P, wn=256, st=None)
MUL = dict(x=P, ldx=64, res=None, ldr=64, dt=1, nw=None, nwdt=1, eps=1e-6, M=4, K=64, codes=P,
           scales=P, sdt=1, zeros=None, group=128, N=32, ro=vp(0x20000), ldh=64, out=vp(0x30000),
           odt=1, ldo=32, ws=P, wn=256, st=None)


def test_sizes(S):
    assert S.lib().spec_w4_code_bytes(5, 1000) == 5 * 512
    assert S.lib().spec_w4_code_bytes(5, 0) == 0


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(ldx=63), -1), (dict(group=16), -1),
    (dict(group=96), -1), (dict(dt=2), -2), (dict(sdt=3), -2), (dict(ws=None), -1),
    (dict(wn=255), -3), (dict(x=None), -1), (dict(x=ODD), -1), (dict(codes=MIS), -1),
    (dict(scales=MIS), -1), (dict(codes=None), -1), (dict(rows=0, x=None), 0)])
def test_quantize_refusals(S, at, rc):
    assert S.lib().spec_w4_quantize(*changed(PACK, at)) == rc


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(ldo=63), -1), (dict(group=0), -1),
    (dict(odt=2), -2), (dict(sdt=3), -2), (dict(ws=vp(0x1010)), -1), (dict(wn=0), -3),
    (dict(out=None), -1), (dict(out=ODD), -1), (dict(codes=MIS), -1), (dict(scales=None), -1),
    (dict(rows=0, out=None), 0)])
def test_dequantize_refusals(S, at, rc):
    assert S.lib().spec_w4_dequantize(*changed(BACK, at)) == rc


@pytest.mark.parametrize("at,rc", [
    (dict(M=-1), -1), (dict(K=0), -1), (dict(N=0), -1), (dict(ldx=63), -1), (dict(ldo=31), -1),
    (dict(group=256), -1), (dict(res=vp(0x40000), ldr=63), -1), (dict(res=vp(0x40000), ldh=63), -1),
    (dict(dt=2), -2), (dict(sdt=2), -2), (dict(odt=2), -2), (dict(nw=P, nwdt=2), -2),
    (dict(nw=P, eps=-1.0), -1), (dict(nw=P, eps=float("nan")), -1), (dict(ws=None), -1),
    (dict(wn=8), -3), (dict(dt=0, odt=0, K=36865, ldx=36865), -7), (dict(K=73729, ldx=73729), -7),
    (dict(x=None), -1), (dict(x=ODD), -1), (dict(out=None), -1), (dict(out=ODD), -1),
    (dict(codes=MIS), -1), (dict(scales=None), -1), (dict(nw=ODD), -1),
    (dict(res=vp(0x40000), ro=None), -1), (dict(res=ODD), -1),
    (dict(res=vp(0x40000), ro=P), -1), (dict(res=vp(0x40000), ro=vp(0x40000)), -1),
    (dict(res=vp(0x40000), ro=vp(0x40000 + 2 * (3 * 64 + 60))), -1),
    (dict(out=P), -1), (dict(res=vp(0x40000), out=vp(0x20000)), -1), (dict(M=0, x=None), 0)])
def test_product_refusals(S, at, rc):
    assert S.lib().spec_w4_logits(*changed(MUL, at)) == rc


def test_binding_checks(S):
    codes, scales = torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 1)
    for args in ((codes, scales, 128, 128), (codes, scales, 96, 128), (codes, scales, 128, 129),
                 (codes.float(), scales, 128, 128), (codes, scales[:2], 128, 128),
                 (codes, scales, 128, 0)):
        with pytest.raises(ValueError):
            S.W4Tensor(*args)
    with pytest.raises(TypeError):
        S.W4Tensor(codes, scales.half(), 128, 128)
