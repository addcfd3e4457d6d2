"""The draft's vocabulary head: final norm and projection onto the vocabulary, in block-scaled
floating point.

"Module deepseek_v4_mtp", Forward, ends in logits = lm_head(rms_norm(h)). Over a large vocabulary
the projection is the draft's largest read (129280 x 4096 in bf16: 1.06 GB a position), and a draft
may round it freely: verification emits the target's distribution whatever the draft proposes.
The weights are quantised once, to 4 bits with a power-of-two scale per 32; the hidden rows to 8
bits as the norm writes them.
"""
from __future__ import annotations

import torch

from . import spec as S


class VocabHead:
    """weight [V, K] and norm_weight [K] (bf16 or fp32) on the device. `fmt` is the format of the
    vocabulary matrix: SPEC_MX_E2M1 (4 bits) or SPEC_MX_E4M3 (8 bits). The given weight is not
    kept."""

    def __init__(self, weight, norm_weight, eps=1e-6, *, fmt=S.SPEC_MX_E2M1, workspace=None):
        if weight.dim() != 2 or norm_weight.shape != (weight.shape[1],):
            raise ValueError("weight must be [V, K] and norm_weight [K]")
        if norm_weight.device != weight.device:
            raise ValueError("weight and norm_weight must be on one device")
        self.w = S.spec_mx_quantize(weight, fmt, workspace=workspace)
        self.norm_weight, self.eps = norm_weight.contiguous(), float(eps)

    @property
    def V(self):
        return self.w.rows

    @property
    def K(self):
        return self.w.K

    def logits(self, hidden, residual=None, *, dtype=torch.bfloat16, out=None, residual_out=None,
               workspace=None, stream=None):
        """Logits [..., V] of hidden rows [..., K] (plus residual, added first). Returns
        (h, logits) with h = hidden + residual, or hidden itself without a residual."""
        if out is None:
            out = S._on_stream(stream, torch.empty, *hidden.shape[:-1], self.V, dtype=dtype,
                               device=hidden.device)
        h, rows = S.spec_rmsnorm_mx(hidden, self.norm_weight, self.eps, residual=residual,
                                    residual_out=residual_out, workspace=workspace, stream=stream)
        S.spec_mx_logits(rows, self.w, out=out, workspace=workspace, stream=stream)
        return h, out
