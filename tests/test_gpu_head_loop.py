"""The decoding loop with a vocabulary head and with log-probabilities of its emitted tokens, and
the bounded waits of the vocabulary product."""
import time

import pytest
import torch

import head_ref as ref
from draft_sampling_verification_markov_gb300 import spec as S
from draft_sampling_verification_markov_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FIELDS = ("anchors", "draft_tokens", "accept_len", "out_tokens")


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(wl, iters, **kw):
    from draft_sampling_verification_markov_gb300.loop import SpecLoop
    g = {k: v.cuda() for k, v in wl.tensors().items()}
    U = kw.pop("U", g["U"])
    return SpecLoop(U, g["target"], g["W1"], g["W2"], g["anchors"], g["u_draft"], g["u_accept"],
                    g["u_resid"], wl.temperature, g.get("sps"), iterations=iters, **kw)


def workload(iters=3):
    return W.full_loop("cpu", R=24, gamma=3, V=1000, rank=64, iterations=iters, seed=5)


def head_inputs(wl, iters, K=192, residual=True):
    from draft_sampling_verification_markov_gb300.head import VocabHead
    g = torch.Generator().manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    head = VocabHead(rn(wl.V, K) * 0.2, 1 + 0.1 * rn(K))
    hidden = rn(iters, wl.R, wl.gamma, K)
    return head, hidden, rn(iters, wl.R, wl.gamma, K) if residual else None


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("flat", [False, True])
def test_head_feeds_the_proposal(built, residual, flat):
    """Each iteration equals a loop over the logits that the head gives for its hidden states."""
    iters = 3
    wl = workload(iters)
    head, hidden, res = head_inputs(wl, iters, residual=residual)
    lp = make(wl, iters, U=None, head=head, hidden=hidden, residual=res, flat=flat)
    lp.run()
    torch.cuda.synchronize()
    assert lp.ws.status() == 0
    for t in range(iters):
        _, U = head.logits(hidden[t], None if res is None else res[t])
        one = make(wl, iters, U=U, flat=flat)
        one.anchors[t].copy_(lp.anchors[t])
        one.run(t, t + 1)
        torch.cuda.synchronize()
        for name in FIELDS:
            rows = slice(t, t + 2) if name == "anchors" else slice(t, t + 1)
            assert torch.equal(getattr(one, name)[rows], getattr(lp, name)[rows]), (name, t)
    if residual:
        want = (hidden[-1].float() + res[-1].float()).to(torch.bfloat16)
        assert torch.equal(lp.draft_hidden, want)


def test_head_logits_against_the_definition(built):
    """norm, quantisation and product of the class, from its quantised weights, in 64 bits."""
    wl = workload(1)
    head, hidden, res = head_inputs(wl, 1)
    h, out = head.logits(hidden[0], res[0], dtype=torch.float32)
    assert out.shape == (wl.R, wl.gamma, wl.V)
    x = h.double().cpu().reshape(-1, head.K).numpy()
    y = x / ((x ** 2).mean(1, keepdims=True) + head.eps) ** 0.5
    y = y * head.norm_weight.double().cpu().numpy()
    w = ref.dequantize(head.w.codes.cpu(), head.w.scales.cpu(), head.w.fmt, head.K)
    want = y @ w.T
    _, q = S.spec_rmsnorm_mx(hidden[0], head.norm_weight, head.eps, residual=res[0])
    rows = ref.dequantize(q.codes.cpu(), q.scales.cpu(), q.fmt, head.K)
    ref.check_rounded(rows, q.scales.cpu(), q.fmt, y, ref.norm_rel(head.K))
    mag = abs(rows) @ abs(w).T
    tol = (head.K + 4) * 2 * ref.U32 * mag
    assert (abs(out.reshape(-1, wl.V).double().cpu().numpy() - rows @ w.T) <= tol).all()
    # and the whole of it: an E4M3 element is off by at most 2^-4 of itself, or 2^-10 of its block's
    # scale where it is subnormal (below 2^-6 of it; the scale is at most 2^-7 of the maximum)
    big = abs(y).max(1, keepdims=True)
    off = (abs(y) * 2.0 ** -4 + big * 2.0 ** -17) @ abs(w).T
    assert (abs(rows @ w.T - want) <= off * 1.001).all()


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("k", [0, 5])
def test_logprobs_of_the_emitted_tokens(built, flat, k):
    iters = 3
    wl = workload(iters)
    lp = make(wl, iters, flat=flat, logprobs=k)
    plain = make(wl, iters, flat=flat)
    lp.run()
    plain.run()
    torch.cuda.synchronize()
    assert lp.ws.status() == 0
    for name in FIELDS:
        assert torch.equal(getattr(lp, name), getattr(plain, name))
    x = wl.target.reshape(-1, wl.V).double()
    for t in range(iters):
        tok = lp.out_tokens[t].cpu().reshape(-1)
        want = ref.token_logprobs(x, tok, wl.temperature, k)
        said = tok >= 0
        assert said.sum() == (lp.accept_len[t] + 1).sum()
        zmax = float((x.amax(1) - x.amin(1)).max() / wl.temperature)
        tol = ref.logp_tol(wl.V, zmax)
        got = lp.token_logp[t].cpu().reshape(-1).double()
        assert ((got - want["logp"]).abs()[said] <= tol).all() and torch.isnan(got[~said]).all()
        rank = lp.token_rank[t].cpu().reshape(-1).long()
        assert torch.equal(rank[said], want["rank"][said]) and (rank[~said] == 0).all()
        ent = lp.token_entropy[t].cpu().reshape(-1).double()
        assert ((ent - want["entropy"]).abs()[said]
                <= (2 * tol * (1 + want["spread"]))[said]).all()
        if k:
            ids = lp.top_ids[t].cpu().reshape(-1, k).long()
            assert torch.equal(ids[said], want["top_ids"][said]) and (ids[~said] == -1).all()


def test_captured_loop_with_head_and_logprobs(built):
    iters = 3
    wl = workload(iters)
    head, hidden, res = head_inputs(wl, iters)
    kw = dict(U=None, head=head, hidden=hidden, residual=res, logprobs=4, async_schedule=True)
    eager, graph = make(wl, iters, **kw), make(wl, iters, **kw)
    eager.run()
    graph.capture()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for name in FIELDS + ("token_rank", "top_ids", "top_logp"):
        assert torch.equal(getattr(eager, name), getattr(graph, name)), name
    a, b = eager.token_logp, graph.token_logp
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])
    assert graph.ws.status() == 0


def test_loop_refusals(built):
    wl = workload(2)
    head, hidden, res = head_inputs(wl, 2)
    with pytest.raises(ValueError, match="together"):
        make(wl, 2, head=head)
    with pytest.raises(ValueError, match="hidden must be"):
        make(wl, 2, head=head, hidden=hidden[..., :100])
    with pytest.raises(ValueError, match="slice"):
        make(wl, 2, head=head, hidden=hidden[:1])
    with pytest.raises(ValueError, match="shape"):
        make(wl, 2, head=head, hidden=hidden, residual=res[:1])


def test_expired_wait_of_the_product_reports_timeout(built):
    a = S.spec_mx_quantize(torch.randn(100, 512, device=DEV), S.SPEC_MX_E4M3)
    w = S.spec_mx_quantize(torch.randn(3000, 512, device=DEV), S.SPEC_MX_E2M1)
    ws = S.Workspace(256, device=DEV)
    want = S.spec_mx_logits(a, w, workspace=ws).clone()
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert S.lib().spec_test_stall_next_markov() == 0
    t0 = time.time()
    S.spec_mx_logits(a, w, workspace=ws)
    torch.cuda.synchronize()
    waited = time.time() - t0
    assert ws.status() & S.SPEC_DEV_TIMEOUT
    assert 0.5 < waited < 30.0
    again = S.spec_mx_logits(a, w, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0 and torch.equal(again, want)


def test_tensors_of_a_call_belong_to_its_stream(built, monkeypatch):
    """What a call allocates comes from the stream it was given, not from the current one, where
    the memory may still be read or be given away again: the intermediate rows of the head too."""
    from draft_sampling_verification_markov_gb300.head import VocabHead
    side, seen = torch.cuda.Stream(), []
    g = torch.Generator().manual_seed(3)
    w, x = (torch.randn(n, 256, generator=g).to(DEV) for n in (640, 5))
    head = VocabHead(w, torch.ones(256, device=DEV))
    tok = torch.zeros(5, dtype=torch.int32, device=DEV)

    def calls(**kw):
        h, z = head.logits(x, x, dtype=torch.float32, **kw)
        q = S.spec_mx_quantize(x, **kw)
        y = S.spec_mx_dequantize(q, dtype=torch.float32, **kw)
        z2 = S.spec_mx_logits(q, head.w, dtype=torch.float32, **kw)
        r = S.spec_token_logprobs(z, tok, 1.0, top=3, **kw)
        return [h, z, y, z2, r.logp, r.rank, r.entropy, r.top_ids, r.top_logp]

    want = calls()
    torch.cuda.synchronize()
    empty = torch.empty

    def recorded(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", recorded)
    got = calls(stream=side)
    side.synchronize()
    assert seen and set(seen) == {side.cuda_stream}
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_in_a_row_wait_for_what_they_read(built):
    """Each call may be scheduled while the kernel before it ends. Chains that hand buffers over
    and write them again, over two streams that meet, after copies and fills, eager and replayed
    from a graph, give what the same calls give one at a time."""
    from draft_sampling_verification_markov_gb300.head import VocabHead
    g = torch.Generator().manual_seed(9)
    K, V, M, n = 512, 5000, 40, 12
    head = VocabHead(torch.randn(V, K, generator=g).to(DEV) * 0.1, torch.ones(K, device=DEV))
    xs = torch.randn(n, M, K, generator=g).to(DEV)
    tok = torch.randint(V, (n, M), generator=g, dtype=torch.int32).to(DEV)
    side = torch.cuda.Stream()
    ws, ws2 = S.Workspace(device=DEV), S.Workspace(device=DEV)
    ws.reserve(256), ws2.reserve(256)
    x, r, z = torch.empty(M, K, device=DEV), torch.empty(M, K, device=DEV), torch.empty(
        M, V, device=DEV)
    q, back = S.MXTensor.empty(M, K, S.SPEC_MX_E4M3, DEV), torch.empty(M, K, device=DEV)
    out = [S.TokenLogprobs.empty(M, 3, True, torch.device(DEV)) for _ in range(n)]
    backs = torch.empty(n, M, K, device=DEV)

    def chain(step):
        main = torch.cuda.current_stream()
        r.zero_()
        for i in range(n):
            x.copy_(xs[i])
            S.spec_rmsnorm_mx(x, head.norm_weight, residual=r, residual_out=r, out=q,
                              workspace=ws)
            step()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                S.spec_mx_dequantize(q, out=back, workspace=ws2)
                step()
                S.spec_mx_quantize(back, S.SPEC_MX_E4M3, out=q2, workspace=ws2)
                step()
                S.spec_mx_dequantize(q2, out=backs[i], workspace=ws2)
                step()
            S.spec_mx_logits(q, head.w, out=z, workspace=ws)
            step()
            S.spec_token_logprobs(z, tok[i], 1.0, top=3, out=out[i], workspace=ws)
            step()
            main.wait_stream(side)
            if i % 3 == 0:  # straight after both streams
                S.spec_token_logprobs(z, tok[i], 1.0, top=3, out=out[i], workspace=ws)
                step()

    q2 = S.MXTensor.empty(M, K, S.SPEC_MX_E4M3, DEV)

    def results():
        torch.cuda.synchronize()
        assert ws.status() == 0 and ws2.status() == 0
        return [getattr(o, f).clone() for o in out for f in S.TokenLogprobs.__slots__] + [
            backs.clone(), r.clone()]

    def spoil():
        for t in [x, r, z, back, backs] + [getattr(o, f) for o in out
                                           for f in S.TokenLogprobs.__slots__]:
            t.fill_(7)

    chain(torch.cuda.synchronize)
    want = results()
    for _ in range(20):
        spoil()
        chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for _ in range(20):
        spoil()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
