"""Numbers as parameters of truncated sampling that their C types do not hold."""
import pytest
import torch

from draft_sampling_verification_markov_gb300 import spec


@pytest.mark.parametrize("k,want", [(5, 5), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                    (2 ** 32 + 1, 2 ** 31 - 1), (2 ** 70, 2 ** 31 - 1), (-1, -1),
                                    (-2 ** 31, -1), (-2 ** 32 + 5, -1)])
def test_top_k_is_not_cut_to_32_bits(k, want):
    """Past the vocabulary is all tokens, negative is refused by the call."""
    assert spec._truncation(1.0, k, 1.0, 0.0, 4, torch.device("cpu")).top_k == want
