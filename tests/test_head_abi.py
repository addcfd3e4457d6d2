"""Refusals of the block-scaled head and the token log-probabilities, on the host: every bad
argument returns its status before any launch, and the binding's checks raise."""
import ctypes

import numpy as np
import pytest
import torch

import head_ref as ref

vp, ci, cll, cf, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float,
                       ctypes.c_size_t)
OK_PTR, ODD = vp(0x1000), vp(0x1001)


@pytest.fixture(scope="module")
def L():
    from draft_sampling_verification_markov_gb300 import build
    build.build()
    from draft_sampling_verification_markov_gb300 import spec
    return spec.lib()


def changed(base, **at):
    """base (an ordered dict) with some arguments replaced, as a tuple."""
    assert set(at) <= set(base)
    return tuple({**base, **at}.values())


def test_sizes(L):
    assert L.spec_mx_code_bytes(0, 5, 1000) == 5 * 512
    assert L.spec_mx_code_bytes(1, 5, 1000) == 5 * 1024
    assert L.spec_mx_code_bytes(1, 0, 1000) == 0
    assert L.spec_mx_scale_bytes(129, 129) == 2 * 2 * 512
    assert L.spec_mx_code_bytes(2, 5, 8) == 0 and L.spec_mx_code_bytes(0, -1, 8) == 0
    assert L.spec_mx_scale_bytes(5, 0) == 0


QUANT = dict(x=OK_PTR, dt=1, ldx=64, rows=4, K=64, fmt=0, codes=OK_PTR, scales=OK_PTR, ws=OK_PTR,
             wn=256, st=None)


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(ldx=63), -1), (dict(fmt=2), -1),
    (dict(dt=2), -2), (dict(ws=None), -1), (dict(ws=vp(0x1010)), -1), (dict(wn=255), -3),
    (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(codes=vp(0x1010)), -1), (dict(scales=vp(0x1008)), -1), (dict(x=ODD), -1),
    (dict(K=(1 << 24) + 1, ldx=1 << 25), -1), (dict(rows=0, x=None, codes=None), 0)])
def test_quantize_refusals(L, at, rc):
    assert L.spec_mx_quantize(*changed(QUANT, **at)) == rc


DEQUANT = dict(codes=OK_PTR, scales=OK_PTR, fmt=0, rows=4, K=64, out=OK_PTR, dt=1, ldo=64,
               ws=OK_PTR, wn=256, st=None)


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(ldo=63), -1), (dict(fmt=-1), -1),
    (dict(dt=5), -2), (dict(out=None), -1), (dict(out=ODD), -1), (dict(codes=vp(0x1010)), -1),
    (dict(wn=8), -3), (dict(rows=0, out=None), 0)])
def test_dequantize_refusals(L, at, rc):
    assert L.spec_mx_dequantize(*changed(DEQUANT, **at)) == rc


NORM = dict(x=OK_PTR, ldx=64, r=OK_PTR, ldr=64, dt=1, w=OK_PTR, wdt=1, eps=1e-6, rows=4, K=64,
            ro=vp(0x9000), ldo=64, fmt=1, codes=OK_PTR, scales=OK_PTR, ws=OK_PTR, wn=256, st=None)


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(ldx=63), -1), (dict(ldr=63), -1),
    (dict(ldo=63), -1), (dict(fmt=7), -1), (dict(dt=3), -2), (dict(wdt=3), -2),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(x=None), -1), (dict(w=None), -1), (dict(ro=None), -1), (dict(ro=ODD), -1),
    (dict(codes=vp(0x1010)), -1), (dict(wn=0), -3), (dict(ws=None), -1),
    (dict(ro=OK_PTR, ldo=128), -1), (dict(ro=vp(0x1010)), -1), (dict(ro=vp(0x1000 + 2 * 64)), -1),
    (dict(ro=vp(0x1000 + 2 * 32), ldx=128, ldr=128, ldo=128), -1),
    (dict(ro=vp(0x1000 + 2 * 4 * 64 - 2)), -1),
    (dict(r=vp(0x8000), ro=vp(0x8000 + 2 * 100), ldr=128, ldo=128), -1),
    (dict(rows=0, x=None, ro=None), 0)])
def test_norm_refusals(L, at, rc):
    assert L.spec_rmsnorm_mx(*changed(NORM, **at)) == rc


LOGITS = dict(ac=OK_PTR, a=OK_PTR, af=1, wc=OK_PTR, w=OK_PTR, wf=0, M=4, V=100, K=64, out=OK_PTR,
              dt=1, ldo=100, ws=OK_PTR, wn=256, st=None)


@pytest.mark.parametrize("at,rc", [
    (dict(M=-1), -1), (dict(V=0), -1), (dict(K=0), -1), (dict(ldo=99), -1), (dict(af=2), -1),
    (dict(wf=-1), -1), (dict(dt=4), -2), (dict(ac=None), -1), (dict(w=None), -1),
    (dict(out=None), -1), (dict(out=ODD), -1), (dict(wc=vp(0x1010)), -1),
    (dict(a=vp(0x1008)), -1), (dict(ws=vp(0x1004)), -1), (dict(wn=100), -3),
    (dict(M=0, ac=None, out=None), 0)])
def test_logits_refusals(L, at, rc):
    assert L.spec_mx_logits(*changed(LOGITS, **at)) == rc


LOGPROBS = dict(x=OK_PTR, dt=1, ld=100, tok=OK_PTR, T=1.0, rows=4, V=100, top=5, lp=OK_PTR,
                rank=OK_PTR, ent=OK_PTR, ti=OK_PTR, tl=OK_PTR, ws=OK_PTR, wn=256, st=None)


@pytest.mark.parametrize("at,rc", [
    (dict(rows=-1), -1), (dict(V=0), -1), (dict(ld=99), -1), (dict(dt=9), -2),
    (dict(T=-1.0), -1), (dict(T=float("nan")), -1), (dict(T=float("inf")), -1),
    (dict(T=1e-44), -1), (dict(top=-1), -1), (dict(top=33), -7), (dict(x=None), -1),
    (dict(x=ODD), -1), (dict(tok=None), -1), (dict(tok=None, lp=None), -1), (dict(ws=None), -1),
    (dict(wn=255), -3), (dict(rows=0, x=None), 0)])
def test_logprobs_refusals(L, at, rc):
    assert L.spec_token_logprobs(*changed(LOGPROBS, **at)) == rc


def test_binding_refuses_host_tensors_and_bad_shapes():
    from draft_sampling_verification_markov_gb300 import spec
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device"):
        spec.spec_mx_quantize(x)
    with pytest.raises(ValueError, match="device"):
        spec.spec_token_logprobs(x, None)
    with pytest.raises(ValueError, match="codes"):
        spec.MXTensor(torch.zeros(4, 63, dtype=torch.uint8),
                      torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 0, 64)
    with pytest.raises(ValueError, match="scales"):
        spec.MXTensor(torch.zeros(4, 64, dtype=torch.uint8),
                      torch.zeros(1, 2, 32, 4, 4, dtype=torch.uint8), 0, 64)
    with pytest.raises(ValueError, match="fmt"):
        spec.MXTensor(torch.zeros(4, 64, dtype=torch.uint8),
                      torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 3, 64)
    with pytest.raises(ValueError, match="device tensors"):
        spec.MXTensor.empty(4, 64, 0, "cpu")
    with pytest.raises(ValueError, match="column"):
        spec.MXTensor.empty(4, 0, 0, "cpu")
    with pytest.raises(ValueError, match="CUDA device"):
        spec.MXTensor(torch.zeros(4, 64, dtype=torch.uint8),
                      torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 0, 64)


# --------------------------------------------------------------------- the 64-bit definitions

@pytest.mark.parametrize("fmt", [ref.E2M1, ref.E4M3])
def test_reference_keeps_format_values(fmt):
    """Every value of the format, under a block that holds its largest, is kept; layout indexes
    agree between writing and reading."""
    vals = ref.code_values(fmt)
    vals = vals[np.isfinite(vals)]
    rng = np.random.default_rng(0)
    x = rng.choice(vals, (130, 200)) * 2.0 ** rng.integers(-20, 20, (130, 1))
    x[:, ::32] = ref.TOP[fmt] * 2.0 ** rng.integers(-20, 20, (130, 1))
    codes, s = ref.quantize(x, fmt)
    y = ref.dequantize(codes, s, fmt, 200)
    big = np.repeat(np.abs(x.reshape(130, 200)).reshape(130, -1), 1, 1)
    same = y == x
    # a value may only change where its block's scale is larger than the one it was drawn with
    step = np.abs(y - x)
    assert same.mean() > 0.2 and (step <= big.max(1, keepdims=True)).all()
    ref.check_rounded(y, s, fmt, x, 0.0)


def test_reference_ties_go_to_the_even_code():
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]])
    codes, s = ref.quantize(x, ref.E2M1)
    y = ref.dequantize(codes, s, ref.E2M1, 8)
    np.testing.assert_array_equal(y, [[6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]])
