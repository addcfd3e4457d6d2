"""A W4Tensor is what its tensors hold at the time of a call."""
import pytest
import torch

import w4_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S
from test_gpu_w4 import BF, DEV, F32, packed, randn

pytestmark = pytest.mark.gpu


def test_parts_are_not_exchanged():
    """Another tensor in the place of one that was checked would not be checked, or not be used."""
    w, _ = packed(40, 256, 64, BF, 1)
    for name in ("codes", "scales", "zeros", "group", "K"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name))


def test_storage_that_moves():
    w, v = packed(40, 256, 64, F32, 2, zeros=True)
    x = randn((3, 256), 3, BF)
    w.scales.data = w.scales * 2
    w.codes.data = w.codes.flip(0).contiguous()
    w.zeros.data = w.zeros.clone().fill_(9)
    v = ref.values(w.codes.cpu(), w.scales.cpu(), 64, 256, w.zeros.cpu())
    _, y, mag = ref.product(x, v, 256)
    got = S.spec_w4_logits(x.to(DEV), w, dtype=F32).cpu().double()
    assert ((got - y).abs() <= ref.tolerance(256, 64, mag, y, F32, True)).all()
    assert torch.equal(S.spec_w4_dequantize(w, dtype=F32).cpu(), v.float())
