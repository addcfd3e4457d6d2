"""The vocabulary head's calls straight after the kernel that writes their inputs, without a wait
in between: their blocks start while that kernel still runs, and read what it wrote."""
import pytest
import torch

from draft_sampling_verification_markov_gb300 import spec as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTS = [torch.bfloat16, torch.float32]


def seeded(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def fields(q):
    return [q.codes.clone(), q.scales.clone()]


def lp(r):
    return [r.logp, r.rank, r.entropy, r.top_ids, r.top_logp]


def check(step, buf, news):
    """step(buf) for each of `news`, written into buf by the kernel before, equals step(new) of a
    buffer that nothing writes meanwhile."""
    want = []
    for x in news:
        torch.cuda.synchronize()
        want.append(step(x))
        torch.cuda.synchronize()
    got = []
    for x in news * 4:
        step(buf)            # the buffer's old contents are read by the same kernels
        buf.copy_(x)
        buf.mul_(2.0).mul_(0.5)   # in place: each value passes through the SM that rewrites it
        got.append(step(buf))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(news)])), i


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,K", [(1, 100), (3000, 1001), (700, 4096)])
def test_inputs_written_by_the_kernel_before(rows, K, dt):
    news = [seeded(rows, K, seed=s, dtype=dt) for s in range(4)]
    ws = S.Workspace(256, device=DEV)
    w = torch.ones(K, device=DEV)
    check(lambda x: fields(S.spec_mx_quantize(x, S.SPEC_MX_E4M3, workspace=ws)),
          torch.empty_like(news[0]), news)
    check(lambda x: fields(S.spec_rmsnorm_mx(x, w, workspace=ws)[1]),
          torch.empty_like(news[0]), news)
    tok = torch.randint(K, (rows,), device=DEV, dtype=torch.int32)
    check(lambda x: lp(S.spec_token_logprobs(x, tok, 0.7, top=5, workspace=ws)),
          torch.empty_like(news[0]), news)


@pytest.mark.parametrize("K", [999, 4096, 9001])
def test_weights_written_by_the_kernel_before(K):
    x = seeded(600, K, seed=9, dtype=torch.bfloat16)
    ws = S.Workspace(256, device=DEV)
    news = [1 + 0.2 * seeded(K, seed=s) for s in range(4)]
    check(lambda w: fields(S.spec_rmsnorm_mx(x, w, workspace=ws)[1]),
          torch.empty_like(news[0]), news)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,K,V", [(5, 320, 1003), (300, 1000, 5001)])
def test_calls_one_after_the_other(rows, K, V, dt):
    """In-place norm, quantised sum, product, read-back and log-probabilities in one chain, each
    reading what the call before wrote into buffers of the step before."""
    news = [seeded(rows, K, seed=s, dtype=dt) for s in range(4)]
    ws = S.Workspace(256, device=DEV)
    w = S.spec_mx_quantize(seeded(V, K, seed=20), workspace=ws)
    r = seeded(rows, K, seed=21, dtype=dt)
    g = torch.ones(K, device=DEV, dtype=dt)
    tok = torch.randint(V, (rows,), device=DEV, dtype=torch.int32)
    q = S.MXTensor.empty(rows, K, S.SPEC_MX_E4M3, DEV)
    q2 = S.MXTensor.empty(rows, K, S.SPEC_MX_E4M3, DEV)
    logits = torch.empty(rows, V, device=DEV, dtype=dt)
    back = torch.empty(rows, K, device=DEV, dtype=dt)
    h = torch.empty(rows, K, device=DEV, dtype=dt)

    def step(x):
        h.copy_(x)
        S.spec_rmsnorm_mx(h, g, residual=r, residual_out=h, out=q, workspace=ws)
        S.spec_mx_quantize(h, S.SPEC_MX_E4M3, out=q2, workspace=ws)
        S.spec_mx_dequantize(q2, out=back, workspace=ws)
        S.spec_mx_logits(q, w, out=logits, workspace=ws)
        out = lp(S.spec_token_logprobs(logits, tok, 1.0, top=3, workspace=ws))
        return [h.clone(), back.clone(), logits.clone()] + out

    want = []
    for x in news:               # with a wait after every call
        h.copy_(x)
        torch.cuda.synchronize()
        S.spec_rmsnorm_mx(h, g, residual=r, residual_out=h, out=q, workspace=ws)
        torch.cuda.synchronize()
        S.spec_mx_quantize(h, S.SPEC_MX_E4M3, out=q2, workspace=ws)
        torch.cuda.synchronize()
        S.spec_mx_dequantize(q2, out=back, workspace=ws)
        torch.cuda.synchronize()
        S.spec_mx_logits(q, w, out=logits, workspace=ws)
        torch.cuda.synchronize()
        out = lp(S.spec_token_logprobs(logits, tok, 1.0, top=3, workspace=ws))
        torch.cuda.synchronize()
        want.append([h.clone(), back.clone(), logits.clone()] + out)
    got = [step(x) for x in news * 4]
    torch.cuda.synchronize()
    for i, s in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(s, want[i % 4])), i
    assert ws.status() == 0
