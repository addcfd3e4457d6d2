"""Definitions in 64 bits of the block-scaled formats, the norm and the token log-probabilities,
and the rounding bounds their kernels are held to."""
import numpy as np
import torch

E2M1, E4M3 = 0, 1
TOP = {E2M1: 6.0, E4M3: 448.0}
U32 = 2.0 ** -24          # half a step of fp32, relative


def code_values(fmt):
    """The value of every code, from its sign, exponent and significand."""
    if fmt == E2M1:
        mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
        return np.concatenate([mag, -mag])
    c = np.arange(128)
    ex, man = c >> 3, (c & 7) / 8.0
    mag = np.where(ex > 0, (1 + man) * 2.0 ** (ex - 7.0), man * 2.0 ** -6)
    mag[127] = np.nan
    return np.concatenate([mag, -mag])


def groups(K):
    return -(-K // 128)


def quantize(x, fmt):
    """codes [rows, G * 64 or G * 128], scales [tiles, G, 32, 4, 4] of x (fp64 [rows, K])."""
    rows, K = x.shape
    G = groups(K)
    b = np.zeros((rows, G * 128))
    b[:, :K] = x
    b = b.reshape(rows, G * 4, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(2)
    finite = np.isfinite(b).all(2)
    e = np.full(amax.shape, -127)
    ok = finite & (amax > 0)
    e[ok] = np.maximum(np.ceil(np.log2(amax[ok] / TOP[fmt])).astype(int), -127)
    e = np.where(ok & (amax > TOP[fmt] * 2.0 ** e), e + 1, e)
    e = np.where(ok & (e > -127) & (amax <= TOP[fmt] * 2.0 ** (e - 1.0)), e - 1, e)
    byte = np.where(finite, e + 127, 255)
    y = np.where(finite[..., None], b, 0.0) / 2.0 ** e[..., None].astype(float)
    mags = code_values(fmt)[:(8 if fmt == E2M1 else 127)]      # ascending, code = index
    a = np.abs(y)
    hi = np.clip(np.searchsorted(mags, a), 0, len(mags) - 1)   # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    # nearest; a tie goes to the even code
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == mags[hi], hi, code)
    code = (code + np.signbit(y) * (8 if fmt == E2M1 else 128)).astype(np.uint8)
    code = code.reshape(rows, G * 128)
    codes = code[:, 0::2] | code[:, 1::2] << 4 if fmt == E2M1 else code
    tiles = -(-rows // 128)
    s = np.zeros((tiles, G, 32, 4, 4), np.uint8)
    r = np.arange(rows)[:, None]
    k = np.arange(G * 4)[None, :]
    s[r // 128, k // 4, r % 32, r % 128 // 32, k % 4] = byte
    return codes, s


def dequantize(codes, scales, fmt, K):
    codes, scales = np.asarray(codes), np.asarray(scales)
    rows, G = codes.shape[0], groups(K)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(rows, -1) if fmt == E2M1 else codes
    r = np.arange(rows)[:, None]
    k = np.arange(G * 4)[None, :]
    byte = scales[r // 128, k // 4, r % 32, r % 128 // 32, k % 4].astype(float)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte - 127))
    return (code_values(fmt)[c].reshape(rows, G * 4, 32) * s[..., None]).reshape(rows, -1)[:, :K]


def check_rounded(q, scales, fmt, y, rel):
    """Block-scaled values q [rows, K] stand for y (fp64) known up to the relative error `rel`:
    each block's scale is the least that fits, each element within half a step."""
    rows, K = y.shape
    G = groups(K)
    pad = np.zeros((rows, G * 128))
    pad[:, :K] = np.abs(y)
    amax = pad.reshape(rows, G * 4, 32).max(2)
    r = np.arange(rows)[:, None]
    k = np.arange(G * 4)[None, :]
    byte = np.asarray(scales)[r // 128, k // 4, r % 32, r % 128 // 32, k % 4].astype(int)
    s = 2.0 ** (byte - 127.0)
    assert (amax * (1 - rel) <= TOP[fmt] * s).all(), "a block's scale is too small"
    assert ((byte == 0) | (amax * (1 + rel) > TOP[fmt] * s / 2)).all(), "a scale is too large"
    se = np.repeat(s, 32, 1)[:, :K]
    low, bits = (0, 1) if fmt == E2M1 else (-6, 3)
    v = np.abs(y) / se * (1 + rel)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(v, 1e-300))), low) - bits)
    assert (np.abs(q - y) <= se * step / 2 + np.abs(y) * rel + 1e-300).all()


def norm_rel(K):
    """Relative error of h * rstd * w in fp32: the sum of squares is a chain of at most
    8 * ceil(K / 2048) + 13 roundings a term (a thread's elements of a 256-thread block, two
    warp sums, the square itself), half of which passes the square root; division by K, + eps,
    the root, its reciprocal and two products are six more."""
    return (0.5 * (8 * -(-K // 2048) + 13) + 6) * U32


def token_logprobs(x, tokens, T, top):
    """logp, rank, entropy, top ids and log-probabilities of logits x (fp64 torch [rows, V])."""
    z = x / T
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    rows, V = x.shape
    out = {}
    if tokens is not None:
        t = tokens.long().clamp(0, V - 1)
        at = x.gather(1, t[:, None])
        out["logp"] = lp.gather(1, t[:, None])[:, 0]
        out["rank"] = (x > at).sum(1) + 1
    out["entropy"] = torch.special.entr(p).sum(1)
    out["spread"] = torch.where(p > 0, p * (z - z.amax(1, keepdim=True)).abs(),
                                torch.zeros_like(p)).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True)
    k = min(top, V)
    ids = torch.full((rows, top), -1, dtype=torch.int64)
    tl = torch.full((rows, top), -float("inf"), dtype=torch.float64)
    ids[:, :k] = order.indices[:, :k].cpu()
    tl[:, :k] = lp.gather(1, order.indices[:, :k]).cpu()
    ids[tl == -float("inf")] = -1
    out["top_ids"], out["top_logp"] = ids, tl
    return out


def logp_tol(V, zmax):
    """Absolute error of z_t - log S in fp32. z = (x - m) / T carries three roundings (the
    difference, 1 / T, the product), an exponential 2^-22, and S a chain of at most
    V / 256 + 32 additions (a thread's share of a row of at least 256 threads, then the tree);
    errors of S pass the logarithm relative to S. The logarithm and the last difference add two
    roundings of numbers up to |z_t| + log V."""
    return (V / 256 + 32 + 4 + 2 * 3 * zmax + 2 * (zmax + np.log(V))) * U32
