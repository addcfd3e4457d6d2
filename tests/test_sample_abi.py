"""Refusals of truncated sampling on the host: every bad argument returns its status before any
launch, and the binding's checks raise."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
OK_PTR, ODD = vp(0x1000), vp(0x1001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def S():
    from draft_sampling_verification_markov_gb300 import build
    build.build()
    from draft_sampling_verification_markov_gb300 import spec
    spec.lib()
    return spec


def rule(S, **at):
    r = S._Truncation(1.0, 0, 1.0, 0.0, None, None, None, None, 1)
    for k, v in at.items():
        setattr(r, k, v)
    return r


SAMPLE = dict(x=OK_PTR, dt=1, ld=64, rows=4, V=64, rule=None, u=OK_PTR, count=None, tokens=OK_PTR,
              logp=None, kept=None, ws=OK_PTR, wn=256, st=None)
CUT = dict(x=OK_PTR, dt=1, ld=64, rows=4, V=64, rule=None, count=None, out=vp(0x9000), ldo=64,
           kept=None, stats=None, ws=OK_PTR, wn=256, st=None)
SHARED = [(dict(rows=-1), -1), (dict(V=0), -1), (dict(ld=63), -1), (dict(dt=2), -2),
          (dict(V=(1 << 20) + 1, ld=1 << 21), -7), (dict(x=None), -1), (dict(x=ODD), -1),
          (dict(ws=None), -1), (dict(ws=vp(0x1010)), -1), (dict(wn=255), -3), (dict(rows=0), 0),
          (dict(rows=(1 << 26) + 1), -1), (dict(rule=0), -1)]


def call(S, name, base, at, r):
    args = {**base, "rule": ctypes.byref(r), **at}
    if args["rule"] == 0:
        args["rule"] = None
    return getattr(S.lib(), name)(*args.values())


@pytest.mark.parametrize("at,rc", SHARED + [(dict(u=None), -1), (dict(tokens=None), -1)])
def test_sample_refusals(S, at, rc):
    assert call(S, "spec_sample", SAMPLE, at, rule(S)) == rc


@pytest.mark.parametrize("at,rc", SHARED + [
    (dict(out=None), -1), (dict(out=vp(0x9001)), -1), (dict(ldo=63), -1),
    (dict(out=vp(0x1010)), -1), (dict(out=OK_PTR, ldo=128), -1), (dict(out=vp(0x1000 + 2 * 250)), -1)])
def test_truncate_refusals(S, at, rc):
    assert call(S, "spec_truncate", CUT, at, rule(S)) == rc


@pytest.mark.parametrize("at", [
    dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=INF), dict(temperature=1e-40),
    dict(top_k=-1), dict(top_p=-0.1), dict(top_p=1.5), dict(top_p=NAN), dict(min_p=-0.1),
    dict(min_p=1.5), dict(min_p=NAN), dict(rows_per_param=0)])
def test_rule_refusals(S, at):
    assert call(S, "spec_sample", SAMPLE, {}, rule(S, **at)) == -1
    assert call(S, "spec_truncate", CUT, {}, rule(S, **at)) == -1


def test_binding_checks(S):
    x, u = torch.zeros(2, 8), torch.zeros(2)
    with pytest.raises(ValueError):
        S.spec_sample(x, u)                       # not on a device
    with pytest.raises(ValueError):
        S.spec_truncate(x)
    dev = torch.device("cpu")
    with pytest.raises(ValueError):
        S._truncation(torch.ones(3), 0, 1.0, 0.0, 4, dev)
    with pytest.raises(ValueError):
        S._truncation(torch.ones(2), torch.ones(4, dtype=torch.int32), 1.0, 0.0, 4, dev)
    with pytest.raises(ValueError):
        S._truncation(torch.ones(2, dtype=torch.float64), 0, 1.0, 0.0, 4, dev)
    with pytest.raises(ValueError):
        S._row_count(torch.zeros(2, dtype=torch.int32), dev)
    r = S._truncation(torch.ones(2), 0, 1.0, 0.0, 6, dev)
    assert r.rows_per_param == 3
