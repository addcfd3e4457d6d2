"""The truncated-sampling and 4-bit operators where they are used: a head of grouped weights, drafts
drawn from truncated rows, truncated targets in verification, and the decoding loop with all of it."""
import numpy as np
import pytest
import torch

import oracle
import sample_ref as sref
import w4_ref as wref
from draft_sampling_verification_markov_gb300 import spec as S
from draft_sampling_verification_markov_gb300 import workloads as W
from gpu_util import compare_verify

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FIELDS = ("anchors", "draft_tokens", "accept_len", "out_tokens")


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def rn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def test_a_step_with_grouped_head_and_truncated_rows(built):
    """Hidden states -> logits -> drafts drawn from truncated rows -> verification against truncated
    target rows: the tokens are the oracle's on the same truncated logits."""
    from draft_sampling_verification_markov_gb300.head import GroupedHead
    R, gamma, V, K, T = 60, 3, 1500, 256, 0.8
    head = GroupedHead((rn((V, K), 1) * 0.3).to(DEV), (1 + 0.1 * rn((K,), 2)).to(DEV), group=64)
    hidden, residual = rn((R, gamma, K), 3).to(DEV), rn((R, gamma, K), 4).to(DEV)
    h, U = head.logits(hidden, residual)
    assert torch.equal(h, (hidden.float() + residual.float()).to(torch.bfloat16))
    v = wref.values(head.w.codes.cpu(), head.w.scales.cpu(), 64, K)
    _, want, mag = wref.product(h.cpu().view(-1, K), v, K, head.norm_weight.cpu(), head.eps)
    got = U.cpu().view(-1, V).double()
    assert ((got - want).abs() <= wref.tolerance(K, 64, mag, want, torch.bfloat16)).all()

    g = torch.Generator().manual_seed(5)
    target = (torch.cat([U.cpu(), rn((R, 1, V), 6)], 1).float()
              + 0.7 * torch.randn(R, gamma + 1, V, generator=g)).to(torch.bfloat16)
    u = torch.rand(R, gamma, generator=g)
    ua, ur = torch.rand(R, gamma, generator=g), torch.rand(R, generator=g)
    k = torch.randint(1, 60, (R,), generator=g, dtype=torch.int32).to(DEV)
    p = (0.6 + 0.4 * torch.rand(R, generator=g)).to(DEV)
    ws = S.Workspace(device=DEV)
    draft = S.spec_sample(U, u.to(DEV).view(-1), T, top_k=k, top_p=p, workspace=ws)
    cut = S.spec_truncate(U, T, top_k=k, top_p=p, workspace=ws)
    tcut = S.spec_truncate(target.to(DEV), T, top_k=k, top_p=p, workspace=ws)
    n, out, nxt = S.spec_verify_rejection(
        tcut.logits, cut.logits, None, None, torch.zeros(R, dtype=torch.int32, device=DEV),
        draft.tokens.view(R, gamma), draft.logp.view(R, gamma), cut.stats.view(R, gamma, 2),
        ua.to(DEV), ur.to(DEV), T, target_stats=tcut.stats, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    # every draft is a token that its row leaves, at the log-probability that verification uses
    row = cut.logits.view(-1, V).gather(1, draft.tokens.long()[:, None])[:, 0].float()
    assert torch.isfinite(row).all()
    again = row / T - cut.stats[:, 0] - cut.stats[:, 1]
    assert ((again - draft.logp).abs() <= 2e-6 * (1 + again.abs())).all()
    rv = oracle.verify_rejection(tcut.logits.cpu(), cut.logits.cpu(), None, None,
                                 torch.zeros(R, dtype=torch.int32),
                                 draft.tokens.cpu().view(R, gamma), ua, ur, T)
    compare_verify(n.cpu().numpy(), out.cpu().numpy(), nxt.cpu().numpy(), rv)
    # what is emitted lies in the target's nucleus
    nn, oo = n.cpu().numpy(), out.cpu().numpy()
    fin = torch.isfinite(tcut.logits).cpu().numpy()
    for r in range(R):
        assert all(fin[r, i, oo[r, i]] for i in range(nn[r] + 1))


def make(wl, iters, target=None, **kw):
    from draft_sampling_verification_markov_gb300.loop import SpecLoop
    g = {k: v.cuda() for k, v in wl.tensors().items()}
    return SpecLoop(g["U"], g["target"] if target is None else target, g["W1"], g["W2"],
                    g["anchors"], g["u_draft"], g["u_accept"], g["u_resid"], wl.temperature,
                    g.get("sps"), iterations=iters, **kw)


def truncated(target, T, rule, rows):
    """Target rows truncated by the definition, on the host."""
    R, g1, V = target.shape
    out = target.clone()
    for r in range(R):
        for i in range(g1):
            k, p, mp = rule(r)
            x = target[r, i].double().numpy()
            order, n, _, margin = sref.row_truncation(x, T, k, p, mp)
            assert margin > sref.SHARE
            out[r, i, torch.from_numpy(order[n:].copy())] = -float("inf")
    return out


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("async_schedule", [False, True])
def test_loop_with_a_truncated_target(built, flat, async_schedule):
    """The loop equals one over a target that was truncated beforehand."""
    iters = 3
    wl = W.full_loop("cpu", R=20, gamma=3, V=900, rank=64, iterations=iters, seed=7)
    T = float(np.float32(wl.temperature))
    lp = make(wl, iters, top_k=40, top_p=0.9, min_p=0.01, flat=flat,
              async_schedule=async_schedule)
    lp.run()
    torch.cuda.synchronize()
    assert lp.ws.status() == 0
    want = truncated(wl.target, T, lambda r: (40, float(np.float32(0.9)), float(np.float32(0.01))),
                     20)
    assert torch.equal(lp.truncated_target.cpu(), want)
    assert torch.equal(lp.kept.cpu(), torch.isfinite(want).sum(2).to(torch.int32))
    one = make(wl, iters, target=want.cuda(), flat=flat, async_schedule=async_schedule)
    one.run()
    torch.cuda.synchronize()
    for name in FIELDS:
        assert torch.equal(getattr(one, name), getattr(lp, name)), name


def test_loop_with_a_rule_for_each_request_head_and_graph(built):
    from draft_sampling_verification_markov_gb300.head import GroupedHead
    iters, R, gamma, V, K = 3, 16, 2, 800, 128
    wl = W.full_loop("cpu", R=R, gamma=gamma, V=V, rank=64, iterations=iters, seed=9)
    head = GroupedHead((rn((V, K), 12) * 0.3).to(DEV), torch.ones(K, dtype=torch.bfloat16,
                                                                    device=DEV))
    hidden, res = rn((iters, R, gamma, K), 13).to(DEV), rn((iters, R, gamma, K), 14).to(DEV)
    k = torch.arange(R, dtype=torch.int32, device=DEV) % 5 * 10
    p = torch.linspace(0.5, 1.0, R, device=DEV)
    kw = dict(top_k=k, top_p=p, head=head, hidden=hidden, residual=res, logprobs=2)
    lp, cap = make(wl, iters, **kw), make(wl, iters, **kw)
    lp.run()
    cap.run()
    torch.cuda.synchronize()
    cap.out_tokens.zero_()
    cap.replay()
    torch.cuda.synchronize()
    assert lp.ws.status() == 0 and cap.ws.status() == 0
    for name in FIELDS + ("token_logp", "kept"):
        a, b = getattr(lp, name), getattr(cap, name)
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())), name
    T = float(np.float32(wl.temperature))
    pc = p.cpu().numpy().astype(np.float64)
    want = truncated(wl.target, T, lambda r: (r % 5 * 10, pc[r], 0.0), R)
    assert torch.equal(lp.truncated_target.cpu(), want)


def test_loop_without_a_truncation_is_unchanged(built):
    wl = W.full_loop("cpu", R=6, gamma=2, V=300, rank=64, iterations=2, seed=3)
    lp = make(wl, 2)
    assert lp.truncation is None
    lp.run()
    one = make(wl, 2, top_p=torch.ones(6, device=DEV))
    one.run()
    torch.cuda.synchronize()
    for name in FIELDS:
        assert torch.equal(getattr(one, name), getattr(lp, name)), name
    assert torch.equal(one.truncated_target.cpu(), wl.target.view(6, 3, 300))


def test_head_from_a_checkpoint(built):
    """Packed weights with zero points as they come."""
    from draft_sampling_verification_markov_gb300.head import GroupedHead
    codes, scales = wref.pack(torch.randn(70, 200, generator=torch.Generator().manual_seed(1)), 32,
                              torch.float32)
    zeros = torch.randint(0, 16, scales.shape, dtype=torch.uint8)
    w = S.W4Tensor(codes.to(DEV), scales.to(DEV), 32, 200, zeros=zeros.to(DEV))
    head = GroupedHead(w, torch.ones(200, device=DEV))
    assert (head.V, head.K) == (70, 200)
    x = rn((2, 200), 2)
    same, y = head.logits(x.to(DEV), dtype=torch.float32)
    assert same.shape == x.shape
    _, want, mag = wref.product(x, wref.values(codes, scales, 32, 200, zeros), 200, torch.ones(200),
                                head.eps)
    assert ((y.cpu().double() - want).abs()
            <= wref.tolerance(200, 32, mag, want, torch.float32)).all()
    with pytest.raises(ValueError):
        GroupedHead(w, torch.ones(201, device=DEV))
