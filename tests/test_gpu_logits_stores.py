"""The vocabulary product's two ways of storing bf16 output against each other: pieces of 16 rows
through shared memory and the copy engine (rows at multiples of 16 bytes), and plain stores (other
row strides). Same products, same rounding, so every element is equal."""
import pytest
import torch

import head_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def random_codes(rows, K, fmt, seed):
    """A block-scaled matrix of any codes but NaN, scales of 2^-3 .. 2^3."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = ref.groups(K) * (64 if fmt == ref.E2M1 else 128)
    codes = torch.randint(0, 256, (rows, width), generator=g, device=DEV, dtype=torch.uint8)
    if fmt == ref.E4M3:
        codes[(codes & 127) == 127] = 0
    scales = torch.randint(124, 131, (-(-rows // 128), ref.groups(K), 32, 4, 4), generator=g,
                           device=DEV, dtype=torch.uint8)
    return S.MXTensor(codes, scales, fmt, K)


@pytest.mark.parametrize("K,V", [(128, 129280), (512, 50000)])
@pytest.mark.parametrize("M", [1, 8, 16, 17, 33, 40, 48, 72, 300, 1000])
def test_staged_pieces_of_consecutive_tiles(M, K, V):
    """Tiles whose rows leave an odd number of 16-row pieces to half of the storing warps (1 .. 16
    or 33 .. 48 beyond a multiple of 64; a last tile of 300 or 1000 rows too) use one staging
    buffer twice in a row, across tiles. Few groups of K leave little time between them. Also 17
    rows, an even number."""
    a, w = random_codes(M, K, ref.E4M3, M), random_codes(V, K, ref.E2M1, V)
    ws = S.Workspace(256, device=DEV)
    plain = torch.empty(M, V + 1, dtype=torch.bfloat16, device=DEV)[:, :V]  # odd row stride
    S.spec_mx_logits(a, w, out=plain, workspace=ws)
    out = torch.empty(M, V, dtype=torch.bfloat16, device=DEV)
    assert out.data_ptr() % 16 == 0 and out.stride(0) % 8 == 0
    same = []
    for i in range(60):
        out.fill_(float(i))
        S.spec_mx_logits(a, w, out=out, workspace=ws)
        same.append((out == plain).all())
    assert torch.stack(same).all() and ws.status() == 0


@pytest.mark.parametrize("M", [1, 40, 108])
def test_staged_pieces_against_the_definition(M):
    """Every row and token of a product of many tiles of one group of K."""
    V, K = 40000, 100
    a, w = random_codes(M, K, ref.E4M3, 1), random_codes(V, K, ref.E2M1, 2)
    out = S.spec_mx_logits(a, w).cpu().double()
    a64, w64 = (torch.from_numpy(ref.dequantize(q.codes.cpu(), q.scales.cpu(), q.fmt, 128))
                for q in (a, w))
    want, mag = a64 @ w64.T, a64.abs() @ w64.abs().T
    # exact products; 128 additions of at most a unit of fp32 each, then half a step of bf16
    tol = 132 * 2 * ref.U32 * mag
    tol += (want.abs() + tol) * 2.0 ** -8
    assert ((out - want).abs() <= tol + 1e-300).all()
