"""Cases of the truncated-sampling operators and of the products with grouped 4-bit weights, for
timing.

The operators, as a speculative decoder's user meets them around the proposal and the verification:

  sample     one token a row from softmax(logits / T) restricted by top-k, top-p and min-p, from a
             given uniform: a request's first token, a draft without a Markov head
  truncate   logits with -inf outside that restriction, and the normalisers of what is left: the
             target rows that lossless verification is to reproduce
  w4         a few hidden rows (residual added, normalised where the case says so) times a matrix
             of 4-bit weights with a scale per group: the draft's vocabulary head and projections
  w4_pack    a matrix written as grouped 4-bit weights and read back

`own` false computes them with elementary torch operations; `own` true calls the package. `exact`
states each definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # four requests' next tokens on a small vocabulary: latency
        dict(name="sample_token", op="sample", rows=4, V=32000, dtype="f32", T=0.7, k=50, p=0.9,
             mp=0.0, per=0),
        # one step of 64 requests at a nucleus alone
        dict(name="sample_step", op="sample", rows=64, V=129280, dtype="bf16", T=1.0, k=0, p=0.95,
             mp=0.0, per=0),
        # 256 requests at a temperature alone: no token is ruled out
        dict(name="sample_plain", op="sample", rows=256, V=129280, dtype="bf16", T=1.0, k=0, p=1.0,
             mp=0.0, per=0),
        # 256 requests with 8 window rows each, every request with parameters of its own
        dict(name="sample_window", op="sample", rows=2048, V=129280, dtype="bf16", T=1.0, k=0,
             p=1.0, mp=0.0, per=8),
        # the verify window of one request, four drafts and the bonus row: latency
        dict(name="truncate_token", op="truncate", rows=5, V=32000, dtype="f32", T=0.7, k=20,
             p=0.8, mp=0.0, per=0),
        # the target rows of 256 requests before verification, parameters per request
        dict(name="truncate_window", op="truncate", rows=2048, V=129280, dtype="bf16", T=1.0, k=0,
             p=1.0, mp=0.0, per=8),
        # one request's next draft: residual, norm and the vocabulary head
        dict(name="w4_token", op="w4", rows=1, N=129280, K=4096, dtype="bf16", group=128,
             scale="bf16", zeros=False, norm=True),
        # the same of eight requests
        dict(name="w4_step", op="w4", rows=8, N=129280, K=4096, dtype="bf16", group=128,
             scale="bf16", zeros=False, norm=True),
        # embedding and hidden state of four requests onto one hidden width, zero points: latency
        dict(name="w4_project", op="w4", rows=4, N=4096, K=8192, dtype="bf16", group=64,
             scale="bf16", zeros=True, norm=False),
        # a window of 16 drafts and the anchor, 32-bit hidden states, small groups
        dict(name="w4_window", op="w4", rows=17, N=32000, K=2048, dtype="f32", group=32,
             scale="f32", zeros=False, norm=True),
        # the draft's vocabulary matrix when it is loaded
        dict(name="w4_pack_head", op="w4_pack", rows=129280, K=4096, dtype="bf16", group=128,
             scale="bf16"),
        # a small 32-bit matrix, neither size a multiple of anything
        dict(name="w4_pack_ragged", op="w4_pack", rows=1001, K=1000, dtype="f32", group=32,
             scale="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "truncate", "truncate", "w4", "w4", "w4_pack"])
    if op in ("sample", "truncate"):
        return dict(op=op, rows=_log_int(rng, 1, 1024), V=_log_int(rng, 1000, 129280),
                    dtype=rng.choice(["bf16", "f32"]), T=rng.choice([0.6, 0.7, 1.0, 1.3]),
                    k=rng.choice([0, 0, 1, 20, 50, 200, 1000]),
                    p=rng.choice([1.0, 1.0, 0.8, 0.9, 0.95, 0.99]),
                    mp=rng.choice([0.0, 0.0, 0.05, 0.1]), per=rng.choice([0, 0, 1]))
    if op == "w4":
        K = _log_int(rng, 128, 8192)
        N = _log_int(rng, 512, min(129280, 129280 * 4096 // K))
        return dict(op=op, rows=_log_int(rng, 1, 24), N=N, K=K, dtype=rng.choice(["bf16", "f32"]),
                    group=rng.choice([32, 64, 128]), scale=rng.choice(["bf16", "f32"]),
                    zeros=rng.choice([False, True]), norm=rng.choice([False, True]))
    K = _log_int(rng, 32, 8192)
    return dict(op=op, rows=_log_int(rng, 1, min(129280, 129280 * 2048 // K)), K=K,
                dtype=rng.choice(["bf16", "f32"]), group=rng.choice([32, 64, 128]),
                scale=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + salt)


def _randn(shape, g, dtype, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _pick(values, n, g, dtype):
    at = torch.randint(len(values), (n,), generator=g, device=DEV)
    return torch.tensor(values, dtype=dtype, device=DEV)[at]


def prepare(case, seed):
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op in ("sample", "truncate"):
        rows, V = case["rows"], case["V"]
        x = _randn((rows, V), _gen(seed, 1), torch.float32, 2.0)
        # a trained model's rows: some tokens stand out, in rows from near flat to sharply peaked
        at = torch.randint(V, (rows, 64), generator=_gen(seed, 2), device=DEV)
        peak = 8.0 + 12.0 * torch.rand(rows, 1, generator=_gen(seed, 3), device=DEV)
        x.scatter_add_(1, at, torch.rand(rows, 64, generator=_gen(seed, 4), device=DEV) * peak)
        s = dict(case=case, logits=x.to(dt))
        if op == "sample":
            s["u"] = torch.rand(rows, generator=_gen(seed, 5), device=DEV)
        if case["per"]:
            # one set of parameters a request, greedy ones among them
            n, f, i = -(-rows // case["per"]), torch.float32, torch.int32
            s.update(T=_pick([0.0, 0.7, 1.0, 1.3], n, _gen(seed, 6), f),
                     k=_pick([0, 0, 20, 50, 200], n, _gen(seed, 7), i),
                     p=_pick([1.0, 0.8, 0.95, 0.99], n, _gen(seed, 8), f),
                     mp=_pick([0.0, 0.0, 0.05], n, _gen(seed, 9), f))
        else:
            s.update(T=case["T"], k=case["k"], p=case["p"], mp=case["mp"])
        return s
    if op == "w4":
        M, N, K = case["rows"], case["N"], case["K"]
        s = dict(case=case, x=_randn((M, K), _gen(seed, 1), dt, 1.0))
        # what a user's program holds since loading: packed weights, with the checkpoint's zero
        # points where it has them
        w = _randn((N, K), _gen(seed, 2), torch.float32, K ** -0.5)
        s["w"] = _pack(w, case["group"], DTYPES[case["scale"]])
        if case["zeros"]:
            s["w"]["zeros"] = torch.randint(6, 11, s["w"]["scales"].shape, generator=_gen(seed, 3),
                                            device=DEV, dtype=torch.uint8)
        if case["norm"]:
            s["residual"] = _randn((M, K), _gen(seed, 4), dt, 4.0)
            s["weight"] = _randn((K,), _gen(seed, 5), torch.float32, 0.1).add_(1.0).to(dt)
        return s
    # weights are near normal; each row has its own size
    x = _randn((case["rows"], case["K"]), _gen(seed, 1), torch.float32, 0.02)
    x *= torch.exp2(torch.randn(case["rows"], 1, generator=_gen(seed, 2), device=DEV))
    return dict(case=case, x=x.to(dt))


# ------------------------------------------------------------------------------ plain forms
# Truncation. Tokens in descending order of their logits, ties to the lower id. Top-k leaves the
# first k (0: all), top-p of these, renormalised, those before which less than p has been reached,
# min-p those at least min_p times as likely as the first. T = 0 leaves the first token. The sums
# are in 64 bits: a border between two tokens is a matter of the last bits of 32.

def _rows_of(value, rows, dtype):
    v = torch.as_tensor(value, dtype=dtype, device=DEV).reshape(-1)
    return v.repeat_interleave(rows // v.numel() if rows % v.numel() == 0
                               else -(-rows // v.numel()))[:rows, None]


def _truncated(s):
    """Logits in descending order, their ids, weights exp(z - max z) and which ones are left."""
    x = s["logits"].float()
    rows, V = x.shape
    T = _rows_of(s["T"], rows, torch.float32)
    k, p = _rows_of(s["k"], rows, torch.int32), _rows_of(s["p"], rows, torch.float32).double()
    mp = _rows_of(s["mp"], rows, torch.float32).double()
    xs, ids = torch.sort(x + 0.0, dim=1, descending=True, stable=True)
    greedy = T == 0
    scale = torch.where(greedy, torch.ones_like(T), 1.0 / T).double()
    w = xs.double() * scale
    w = torch.exp(w - w[:, :1])
    limit = torch.where(greedy, torch.ones_like(k), torch.where(k > 0, k, torch.full_like(k, V)))
    left = (torch.arange(V, device=DEV) < limit) & (xs > -math.inf)
    wk = torch.where(left, w, torch.zeros_like(w))
    c = wk.cumsum(1)
    left &= (p >= 1) | (c - wk < p * c[:, -1:])
    left &= w >= mp
    return xs, ids, w, left, scale


def _sample(s):
    xs, ids, w, left, _ = _truncated(s)
    mass = torch.zeros_like(w).scatter_(1, ids, torch.where(left, w, torch.zeros_like(w)))
    c = mass.cumsum(1)
    total = c[:, -1:]
    # the first token, in order of the ids, whose cumulative mass passes u
    tok = (c <= s["u"].double()[:, None] * total).sum(1)
    last = xs.shape[1] - 1 - (mass > 0).flip(1).int().argmax(1)
    tok = torch.minimum(tok, last)
    logp = torch.log(mass.gather(1, tok[:, None])) - torch.log(total)
    return dict(tokens=tok.to(torch.int32), logp=logp[:, 0].float(),
                kept=left.sum(1).to(torch.int32))


def _truncate(s):
    xs, ids, w, left, scale = _truncated(s)
    mask = torch.zeros_like(left).scatter_(1, ids, left)
    out = s["logits"].masked_fill(~mask, -math.inf)
    z = torch.where(left, w, torch.zeros_like(w)).sum(1)
    stats = torch.stack([xs[:, 0].double() * scale[:, 0], torch.log(z)], 1).float()
    return dict(logits=out, kept=left.sum(1).to(torch.int32), stats=stats)


# Grouped 4-bit weights. Rows of K, padded with zeros to a multiple of 128; `group` consecutive
# elements share a scale s (and a zero point z, 8 without one): w = (code - z) s. Packing takes the
# least scale of its type with 7 s >= the group's largest magnitude, and codes rounded to the
# nearest, ties to even. codes: [N, Kp / 2] bytes, the lower half is the even element.

def _pack(x, group, scale_type):
    rows, K = x.shape
    Kp = -(-K // 128) * 128
    g = torch.nn.functional.pad(x.float(), (0, Kp - K)).view(rows, Kp // group, group).double()
    most = g.abs().amax(-1)
    s = (most / 7).to(scale_type)
    bits = s.view(torch.int16 if scale_type == torch.bfloat16 else torch.int32)
    s = torch.where(s.double() * 7 < most, (bits + 1).view(scale_type), s)
    code = torch.round(g / s.double()[..., None]).nan_to_num_(0.0) + 8
    code = code.to(torch.uint8).view(rows, Kp)
    return dict(codes=code[:, 0::2] + code[:, 1::2] * 16, scales=s, zeros=None, group=group, K=K)


def _values(q):
    """The numbers that grouped 4-bit weights stand for, in 32 bits, without the padding."""
    codes = q["codes"]
    rows = codes.shape[0]
    c = torch.stack([codes & 15, codes >> 4], -1).view(rows, -1, q["group"]).float()
    zero = 8.0 if q["zeros"] is None else q["zeros"].float()[..., None]
    return ((c - zero) * q["scales"].float()[..., None]).view(rows, -1)[:, :q["K"]]


def _w4(s):
    x, c = s["x"], s["case"]
    out = {}
    f = x.float()
    if c["norm"]:
        h = (f + s["residual"].float()).to(x.dtype)
        out["hidden"] = h
        f = h.float()
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out["logits"] = torch.matmul(f, _values(s["w"]).t()).to(x.dtype)
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(op, state)
    if op == "sample":
        return _sample(state)
    if op == "truncate":
        return _truncate(state)
    if op == "w4":
        return _w4(state)
    q = _pack(state["x"], case["group"], DTYPES[case["scale"]])
    return _values(q).to(state["x"].dtype)


def _run_own(op, s):
    from draft_sampling_verification_markov_gb300 import spec
    c = s["case"]
    if op == "sample":
        r = spec.spec_sample(s["logits"], s["u"], s["T"], top_k=s["k"], top_p=s["p"],
                             min_p=s["mp"])
        return dict(tokens=r.tokens, logp=r.logp, kept=r.kept)
    if op == "truncate":
        r = spec.spec_truncate(s["logits"], s["T"], top_k=s["k"], top_p=s["p"], min_p=s["mp"])
        return dict(logits=r.logits, kept=r.kept, stats=r.stats)
    if op == "w4":
        q = s["w"]
        w = spec.W4Tensor(q["codes"], q["scales"], q["group"], q["K"], zeros=q["zeros"])
        if not c["norm"]:
            return dict(logits=spec.spec_w4_logits(s["x"], w))
        h, y = spec.spec_w4_logits(s["x"], w, norm_weight=s["weight"], eps=EPS,
                                   residual=s["residual"])
        return dict(hidden=h, logits=y)
    q = spec.spec_w4_quantize(s["x"], c["group"], scale_dtype=DTYPES[c["scale"]])
    return spec.spec_w4_dequantize(q, dtype=s["x"].dtype)


# ------------------------------------------------------------------------------ work and exact

def work(case):
    op, size, rows = case["op"], 2 if case["dtype"] == "bf16" else 4, case["rows"]
    if op in ("sample", "truncate"):
        n = rows * case["V"]
        return dict(bytes=n * size * (1 if op == "sample" else 2) + rows * 16, flops=4 * n)
    K = case["K"]
    Kp = -(-K // 128) * 128
    N = case["N"] if op == "w4" else rows
    packed = N * Kp // 2 + N * (Kp // case["group"]) * (2 if case["scale"] == "bf16" else 4)
    if op == "w4_pack":
        return dict(bytes=2 * rows * K * size + packed, flops=3 * rows * K)
    if case["zeros"]:
        packed += N * (Kp // case["group"])
    x = rows * K * size * (3 if case["norm"] else 1) + (K * size if case["norm"] else 0)
    return dict(bytes=packed + x + rows * N * size, flops=2 * rows * N * K)


def _exact_order(x):
    """Ids by descending logit, then ascending id: whole numbers, one for each token."""
    b = (x.float() + 0.0).view(torch.int32).long()
    b = torch.where(b < 0, -(b & 0x7fffffff), b)
    return torch.argsort(b * (1 << 24) - torch.arange(x.shape[1], device=x.device), dim=1,
                         descending=True)


def _exact_rows(case, s, at):
    x = s["logits"][at]
    n, rows, V = x.shape[0], case["rows"], case["V"]

    def of(name):
        v = s[name]
        if not torch.is_tensor(v):
            return torch.full((n,), v, dtype=torch.float32, device=DEV).double()
        return v.double()[torch.arange(rows, device=DEV)[at] // case["per"]]

    T, k, p, mp = of("T"), of("k"), of("p"), of("mp")
    scale = torch.where(T > 0, 1.0 / T.float(), torch.ones(n, device=DEV)).double()
    order = _exact_order(x)
    z = x.double().gather(1, order) * scale[:, None]
    count = torch.isfinite(z).sum(1)
    count = torch.where(k > 0, torch.minimum(count, k.long()), count)
    count = torch.where(T > 0, count, torch.ones_like(count))
    place = torch.arange(V, device=DEV)[None, :]
    prob = torch.softmax(z.masked_fill(place >= count[:, None], -math.inf), 1)
    reach = prob.cumsum(1)
    by_p = 1 + (reach < p[:, None]).sum(1)
    count = torch.where(p < 1, torch.minimum(count, by_p), count)
    by_m = (z - z[:, :1] >= torch.log(mp)[:, None]).sum(1)
    count = torch.minimum(count, by_m)
    z = z.masked_fill(place >= count[:, None], -math.inf)
    by_id = torch.full_like(z, -math.inf).scatter_(1, order, z)
    return by_id, count, z[:, 0]


def _exact_weights(q):
    rows, group = q["codes"].shape[0], q["group"]
    c = q["codes"].to(torch.int64)
    c = torch.stack([c % 16, c // 16], 2).flatten(1)
    j = torch.arange(q["K"], device=c.device)
    zero = 8 if q["zeros"] is None else q["zeros"].long()[:, j // group]
    return (c[:, :q["K"]] - zero).double() * q["scales"].double()[:, j // group]


def _exact_pack(x, group, bits):
    rows, K = x.shape
    pad = torch.zeros(rows, -K % group, dtype=torch.float64, device=x.device)
    g = torch.cat([x, pad], 1).unflatten(1, (-1, group))
    a = g.abs().amax(2, keepdim=True)
    # scales of `bits` significant bits
    step = torch.exp2(torch.floor(torch.log2((a / 7).clamp(min=1e-300))) - (bits - 1))
    n = torch.ceil(a / 7 / step)
    n = torch.where(n * step * 7 < a, n + 1, n)
    n = torch.where((n - 1) * step * 7 >= a, n - 1, n)
    sc = n * step
    v = torch.where(a > 0, torch.round(g / sc), torch.zeros_like(g))
    return (v * sc).flatten(1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("sample", "truncate"):
        parts = [_exact_rows(case, s, slice(i, i + 256)) for i in range(0, case["rows"], 256)]
        kept = torch.cat([c for _, c, _ in parts]).to(torch.int32)
        if op == "truncate":
            x = torch.cat([torch.where(z > -math.inf, y.double(), z) for (z, _, _), y in
                           zip(parts, s["logits"].split(256))])
            lse = torch.cat([torch.logsumexp(z, 1) for z, _, _ in parts])
            m = torch.cat([m for _, _, m in parts])
            return dict(logits=x, kept=kept, stats=torch.stack([m, lse - m], 1))
        toks, lps = [], []
        for (z, _, _), u in zip(parts, s["u"].split(256)):
            prob = torch.softmax(z, 1)
            reach = prob.cumsum(1)
            t = torch.searchsorted(reach, (u.double() * reach[:, -1])[:, None], right=True)
            ids = torch.arange(z.shape[1], device=DEV)
            last = torch.where(prob > 0, ids, torch.zeros_like(ids)).amax(1, keepdim=True)
            t = torch.minimum(t, last)
            toks.append(t[:, 0])
            lps.append(torch.log_softmax(z, 1).gather(1, t)[:, 0])
        return dict(tokens=torch.cat(toks).to(torch.int32), logp=torch.cat(lps), kept=kept)
    if op == "w4":
        out = {}
        x = s["x"].double()
        if case["norm"]:
            h = (x + s["residual"].double()).to(s["x"].dtype)
            out["hidden"] = h.double()
            x = h.double() / torch.sqrt(h.double().square().sum(1, keepdim=True) / case["K"] + EPS)
            x = x * s["weight"].double()
        q = s["w"]
        cut = [dict(q, codes=c, scales=sc, zeros=z) for c, sc, z in zip(
            q["codes"].split(8192), q["scales"].split(8192),
            [None] * q["codes"].shape[0] if q["zeros"] is None else q["zeros"].split(8192))]
        out["logits"] = torch.cat([x @ _exact_weights(c).t() for c in cut], 1)
        return out
    bits = 8 if case["scale"] == "bf16" else 24
    return torch.cat([_exact_pack(p.double(), case["group"], bits) for p in s["x"].split(8192)])
