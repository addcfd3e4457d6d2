"""Grouped 4-bit weights in 64 bits, from their definition, on the CPU.

Tolerance of a product. The multiplied numbers are exact (24 bits of the rows, codes of 4 bits,
scales of at most 24), except that a 32-bit row times its norm weight is rounded once. What is left
are fp32 sums: a group's on the tensor cores (G / 16 steps of 16 products a column, each step off by
at most two units of 2^-23 of the running magnitude), one addition a group, up to 8 warps of up to 3
columns joined, and the norm's factor: a sum of squares (2^-20 at most for 2^15 elements added in 512
threads and a tree), a root and a division. All of it relative to sum |a w|.

For a bf16 product the numbers themselves are held in 11 bits, unless they are bf16 already: half a
step, 2^-12 of each, and so of sum |a w|."""
import torch


def padded(K):
    return -(-K // 128) * 128


def least_scale(most, dtype):
    """The least number of dtype with 7 s >= most (both as float64, by stepping)."""
    s = (most / 7).to(dtype)
    up = torch.nextafter(s, torch.full_like(s, float("inf")))
    s = torch.where(s.double() * 7 < most, up, s)
    down = torch.nextafter(s, torch.full_like(s, -float("inf")))
    return torch.where((s > 0) & (down.double() * 7 >= most), down, s)


def pack(x, group, scale_dtype):
    """(codes, scales) of x [rows, K]."""
    rows, K = x.shape
    g = torch.zeros(rows, padded(K), dtype=torch.float64)
    g[:, :K] = x.double()
    g = g.view(rows, -1, group)
    s = least_scale(g.abs().amax(2), scale_dtype)
    sd = s.double()[..., None]
    c = torch.where(sd > 0, torch.round(g / sd), torch.zeros_like(g)) + 8
    c = c.to(torch.uint8).view(rows, -1)
    return (c[:, 0::2] | c[:, 1::2] << 4).contiguous(), s


def values(codes, scales, group, K, zeros=None):
    rows = codes.shape[0]
    c = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1, group).double()
    z = 8.0 if zeros is None else (zeros & 127).double()[..., None]
    return ((c - z) * scales.double()[..., None]).view(rows, -1)[:, :K]


def product(x, w, K, norm=None, eps=0.0, residual=None):
    """(h, y, magnitude): x [M, K] as stored, w [N, K] in 64 bits."""
    h = x
    if residual is not None:
        h = (x.double() + residual.double()).to(x.dtype)
    a = h.double()
    if norm is not None:
        a = a / torch.sqrt((a * a).mean(1, keepdim=True) + eps) * norm.double()
    return h, a @ w.t(), a.abs() @ w.abs().t()


def tolerance(K, group, magnitude, y, dtype, exact=False):
    """`exact`: rows of bf16 without a norm."""
    steps = 2 * (group / 16) + padded(K) / group + 24
    half = torch.finfo(dtype).eps / 2
    held = 0.0 if exact or dtype == torch.float32 else 2.0 ** -12
    return (held + steps * 2.0 ** -23 + 2.0 ** -20) * magnitude + half * y.abs() + 1e-37
