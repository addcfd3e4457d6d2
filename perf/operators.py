"""Cases of the vocabulary-head operators and of the token log-probabilities, for timing.

The operators, as a speculative decoder meets them between its last layer and its proposal or
verification:

  quantize   a matrix written as block-scaled 4- or 8-bit floating point (32 elements share one
             power of two) and read back
  norm       residual addition, root-mean-square norm, output in 8 bits with block scales
  logits     the product of block-scaled rows with a block-scaled vocabulary matrix
  logprobs   log-probability and rank of given tokens, entropy, top alternatives

`own` false computes them with elementary torch operations in 32 bits; `own` true calls the
package. `exact` states each definition in 64 bits.
"""
import math

import torch

own = False

E2M1, E4M3 = 0, 1                       # element formats: 4 bits (largest value 6), 8 bits (448)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the draft's vocabulary matrix when it is loaded: quantised once, read back for a check
        dict(name="quantize_head", op="quantize", rows=129280, K=4096, dtype="bf16", fmt=E2M1),
        # activations of a ragged batch in 32 bits, neither size a multiple of a tile
        dict(name="quantize_ragged", op="quantize", rows=1001, K=1000, dtype="f32", fmt=E4M3),
        # one request drafting its next token
        dict(name="norm_token", op="norm", rows=1, K=4096, dtype="bf16"),
        # a verify window of 256 requests, 8 positions each
        dict(name="norm_window", op="norm", rows=2048, K=4096, dtype="bf16"),
        # the widest batch of the decoding loop: 1024 requests, 17 positions, 32-bit stream
        dict(name="norm_loop", op="norm", rows=17408, K=2048, dtype="f32"),
        # four requests, one drafted token each, on a small vocabulary: latency
        dict(name="logits_token", op="logits", rows=4, V=32000, K=2048, dtype="f32"),
        # 64 requests, one position: the vocabulary matrix is the traffic
        dict(name="logits_step", op="logits", rows=64, V=129280, K=4096, dtype="bf16"),
        # 256 requests, one position of a serial proposal
        dict(name="logits_batch", op="logits", rows=256, V=129280, K=4096, dtype="bf16"),
        # 256 requests, 7 draft positions at once: the tensor cores are the bound
        dict(name="logits_window", op="logits", rows=1792, V=129280, K=4096, dtype="bf16"),
        # four requests answering with log-probabilities: latency
        dict(name="logprobs_token", op="logprobs", rows=4, V=32000, dtype="f32", top=5,
             T=1.0, masked=0.0),
        # one grammar-masked step of 64 requests with 4 window rows each
        dict(name="logprobs_step", op="logprobs", rows=256, V=129280, dtype="bf16", top=20,
             T=0.7, masked=0.3),
        # every emitted token of 256 requests with 8 window rows each
        dict(name="logprobs_window", op="logprobs", rows=2048, V=129280, dtype="bf16", top=20,
             T=1.0, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "logits", "logits", "logprobs", "logprobs"])
    if op == "quantize":
        K = _log_int(rng, 32, 8192)
        rows = _log_int(rng, 1, min(129280, 129280 * 4096 // K))
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "f32"]),
                    fmt=rng.choice([E2M1, E4M3]))
    if op == "norm":
        K = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, min(17408, 17408 * 2048 // K))
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "f32"]))
    if op == "logits":
        V, K = _log_int(rng, 1000, 129280), _log_int(rng, 128, 4096)
        return dict(op=op, rows=_log_int(rng, 1, 1792), V=V, K=K,
                    dtype=rng.choice(["bf16", "f32"]))
    V = _log_int(rng, 1000, 129280)
    return dict(op=op, rows=_log_int(rng, 1, 1024), V=V, dtype=rng.choice(["bf16", "f32"]),
                top=rng.choice([0, 1, 5, 20, 32]), T=rng.choice([1.0, 0.7, 1.3]),
                masked=rng.choice([0.0, 0.0, 0.3, 0.9]))


# ------------------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + salt)


def _randn(shape, g, dtype, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        # weights and activations are near normal; each row has its own size
        x = _randn((case["rows"], case["K"]), _gen(seed, 1), torch.float32, 0.02)
        x *= torch.exp2(torch.randn(case["rows"], 1, generator=_gen(seed, 2), device=DEV))
        return dict(case=case, x=x.to(dt))
    if op == "norm":
        shape = (case["rows"], case["K"])
        return dict(case=case, x=_randn(shape, _gen(seed, 1), dt, 1.0),
                    residual=_randn(shape, _gen(seed, 2), dt, 4.0),
                    weight=_randn((case["K"],), _gen(seed, 3), torch.float32, 0.1).add_(1.0)
                    .to(dt))
    if op == "logits":
        # a user's program holds both operands quantised: the head since loading, the rows as
        # the norm wrote them
        a = _randn((case["rows"], case["K"]), _gen(seed, 1), torch.float32, 1.0)
        w = _randn((case["V"], case["K"]), _gen(seed, 2), torch.float32, 2.0 / case["K"] ** 0.5)
        return dict(case=case, a=_quantize(a, E4M3), w=_quantize(w, E2M1))
    rows, V = case["rows"], case["V"]
    x = _randn((rows, V), _gen(seed, 1), torch.float32, 2.0)
    # a few likely tokens a row, as a trained model's rows have
    at = torch.randint(V, (rows, 8), generator=_gen(seed, 2), device=DEV)
    x.scatter_add_(1, at, torch.rand(rows, 8, generator=_gen(seed, 3), device=DEV) * 10.0)
    tokens = at[:, 0].clone()
    other = torch.randint(V, (rows,), generator=_gen(seed, 4), device=DEV)
    tokens = torch.where(torch.arange(rows, device=DEV) % 4 == 3, other, tokens)
    if case["masked"]:
        g = _gen(seed, 5)
        out = torch.rand(rows, V, generator=g, device=DEV) < case["masked"]
        out.scatter_(1, tokens[:, None], False)
        x.masked_fill_(out, -math.inf)
    return dict(case=case, logits=x.to(dt), tokens=tokens.to(torch.int32))


# ------------------------------------------------------------------------------ plain forms
# Block-scaled matrices. Elements 32 b .. 32 b + 31 of a row share the scale 2^e, the smallest
# power of two for which none of them passes the format's largest value; e is stored with a bias
# of 127 (0 for a block of zeros). Rows are padded with zeros to a multiple of 128 elements.
# codes: [rows, Kp / 2] bytes (the lower half is the even element) or [rows, Kp] bytes.
# scales: [ceil(rows / 128), Kp / 128, 32, 4, 4] bytes: row r, block b of a 128-element group g
# is at [r // 128, g, r % 32, r % 128 // 32, b].

def _padded(K):
    return -(-K // 128) * 128


def _quantize(x, fmt):
    rows, K = x.shape
    Kp = _padded(K)
    x = torch.nn.functional.pad(x.float(), (0, Kp - K)).view(rows, Kp // 32, 32)
    frac, exp2 = torch.frexp(x.abs().amax(-1))
    top, shift = (0.75, 3) if fmt == E2M1 else (0.875, 9)      # 6 = 0.75 * 2^3, 448 = 0.875 * 2^9
    e = (exp2 - shift + (frac > top)).clamp(min=-127)
    e = torch.where(frac == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(x, -e[..., None]).view(rows, Kp)
    if fmt == E2M1:
        mag = y.abs()
        # ties of the rounding go to the even code
        code = ((mag > 0.25).to(torch.uint8) + (mag >= 0.75) + (mag > 1.25) + (mag >= 1.75)
                + (mag > 2.5) + (mag >= 3.5) + (mag > 5.0))
        code += torch.signbit(y).to(torch.uint8) * 8
        codes = code[:, 0::2] + code[:, 1::2] * 16
    else:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    tiles = -(-rows // 128)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, 0, 0, tiles * 128 - rows))
    s = s.view(tiles, 4, 32, Kp // 128, 4).permute(0, 3, 2, 1, 4).contiguous()
    return dict(codes=codes.contiguous(), scales=s, fmt=fmt, K=K)


def _values(q):
    """The numbers that a block-scaled matrix stands for, in 32 bits, without the padding."""
    codes, s = q["codes"], q["scales"]
    rows, tiles, groups = codes.shape[0], s.shape[0], s.shape[1]
    if q["fmt"] == E2M1:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
        table = torch.cat([table, -table])
        two = torch.stack([codes & 15, codes >> 4], -1).view(rows, -1)
        y = table[two.int()]
    else:
        y = codes.view(torch.float8_e4m3fn).float()
    e = s.permute(0, 3, 2, 1, 4).reshape(tiles * 128, groups * 4)[:rows].int() - 127
    y = torch.ldexp(y.view(rows, groups * 4, 32), e[..., None]).view(rows, groups * 128)
    return y[:, :q["K"]]


def _norm(x, residual, weight):
    h = (x.float() + residual.float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    return h, _values(_quantize(y, E4M3)).to(torch.bfloat16)


def _logprobs(logits, tokens, T, top):
    x = logits.float()
    at = x.gather(1, tokens.long()[:, None])
    z = x / T
    m = z.amax(1, keepdim=True)
    z = z - m
    p = torch.exp(z)
    s = p.sum(1, keepdim=True)
    log_s = torch.log(s)
    out = dict(logp=(at / T - m - log_s)[:, 0], rank=(x > at).sum(1).to(torch.int32) + 1,
               entropy=(log_s - torch.where(p > 0, p * z, 0.0).sum(1, keepdim=True) / s)[:, 0])
    if top:
        # larger logits first, then lower ids: one whole number a token
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * (1 << 32)
        order -= torch.arange(x.shape[1], device=DEV)
        ids = torch.topk(order, top, dim=1).indices
        lp = z.gather(1, ids) - log_s
        out["top_ids"] = torch.where(torch.isinf(lp), -1, ids).to(torch.int32)
        out["top_logp"] = lp
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "quantize":
        return _values(_quantize(state["x"], state["case"]["fmt"])).to(torch.bfloat16)
    if op == "norm":
        return _norm(state["x"], state["residual"], state["weight"])
    if op == "logits":
        dt = DTYPES[state["case"]["dtype"]]
        return torch.matmul(_values(state["a"]), _values(state["w"]).t()).to(dt)
    c = state["case"]
    return _logprobs(state["logits"], state["tokens"], c["T"], c["top"])


def _run_own(op, state):
    from draft_sampling_verification_markov_gb300 import spec
    c = state["case"]
    if op == "quantize":
        return spec.spec_mx_dequantize(spec.spec_mx_quantize(state["x"], c["fmt"]))
    if op == "norm":
        h, y = spec.spec_rmsnorm_mx(state["x"], state["weight"], 1e-6,
                                    residual=state["residual"])
        return h, spec.spec_mx_dequantize(y)
    if op == "logits":
        a, w = (spec.MXTensor(q["codes"], q["scales"], q["fmt"], q["K"])
                for q in (state["a"], state["w"]))
        return spec.spec_mx_logits(a, w, dtype=DTYPES[c["dtype"]])
    r = spec.spec_token_logprobs(state["logits"], state["tokens"], c["T"], top=c["top"])
    out = dict(logp=r.logp, rank=r.rank, entropy=r.entropy)
    if c["top"]:
        out.update(top_ids=r.top_ids, top_logp=r.top_logp)
    return out


# ------------------------------------------------------------------------------ work and exact

def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"]
    if op == "logprobs":
        n = rows * case["V"]
        return dict(bytes=n * size + rows * (16 + 8 * case["top"]), flops=4 * n)
    K, Kp = case["K"], _padded(case["K"])
    if op == "quantize":
        code = rows * Kp * (1 if case["fmt"] == E4M3 else 0.5) + rows * Kp // 32
        return dict(bytes=rows * K * (size + 2) + code, flops=3 * rows * K)
    if op == "norm":
        return dict(bytes=rows * K * (3 * size + 2) + rows * Kp * 33 // 32 + K * size,
                    flops=7 * rows * K)
    V = case["V"]
    return dict(bytes=V * Kp * 17 // 32 + rows * Kp * 33 // 32 + rows * V * size,
                flops=2 * rows * V * K)


def _exact_block_round(y, fmt):
    """y [rows, K] in 64 bits to the nearest values of the format under its block scales."""
    rows, K = y.shape
    big, low, bits = (6.0, 0, 1) if fmt == E2M1 else (448.0, -6, 3)
    pad = torch.zeros(rows, -K % 32, dtype=torch.float64, device=y.device)
    b = torch.cat([y, pad], 1).unflatten(1, (-1, 32))
    most = b.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(most.clamp(min=1e-300) / big))
    e = torch.where(most > big * torch.exp2(e), e + 1, e)          # log2's own rounding
    e = torch.where(most <= big * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
    v = b / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    return (torch.round(v / step) * step * torch.exp2(e)).flatten(1)[:, :K]


def _exact_decode(q):
    """Block-scaled values from their fields, in 64 bits."""
    rows = q["codes"].shape[0]
    c = q["codes"].to(torch.int64)
    if q["fmt"] == E2M1:
        c = torch.stack([c % 16, c // 16], 2).flatten(1)
        sign, ex, man = c // 8, c // 2 % 4, (c % 2).double() / 2
        mag = torch.where(ex > 0, (1 + man) * torch.exp2(ex.double() - 1), man)
    else:
        sign, ex, man = c // 128, c // 8 % 16, (c % 8).double() / 8
        mag = torch.where(ex > 0, (1 + man) * torch.exp2(ex.double() - 7), man * 2.0 ** -6)
    r = torch.arange(rows, device=c.device)[:, None]
    b = torch.arange(c.shape[1] // 32, device=c.device)[None, :]
    e = q["scales"][r // 128, b // 4, r % 32, r % 128 // 32, b % 4].double() - 127
    mag = mag.unflatten(1, (-1, 32)) * torch.exp2(e)[..., None]
    return (mag.flatten(1) * (1 - 2 * sign))[:, :q["K"]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # elements are rounded one block at a time: bands of rows bound the memory
        return torch.cat([_exact_block_round(p.double(), case["fmt"])
                          for p in s["x"].split(16384)])
    if op == "norm":
        h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + 1e-6)
        y = y * s["weight"].double()
        return h, torch.cat([_exact_block_round(p, E4M3) for p in y.split(4096)])
    if op == "logits":
        a = _exact_decode(s["a"])
        return torch.cat([a @ _exact_decode(dict(s["w"], codes=p, scales=q)).t()
                          for p, q in zip(s["w"]["codes"].split(16384),
                                          s["w"]["scales"].split(128))], 1)
    lp = [torch.log_softmax(p.double() / case["T"], 1) for p in s["logits"].split(256)]
    out = dict(logp=torch.cat([p[torch.arange(len(p), device=DEV), t.long()]
                               for p, t in zip(lp, s["tokens"].split(256))]),
               rank=None,
               entropy=torch.cat([torch.special.entr(p.exp()).sum(1) for p in lp]))
    if case["top"]:
        out["top_ids"] = None
        out["top_logp"] = torch.cat([p.topk(case["top"], 1).values for p in lp])
    return out
