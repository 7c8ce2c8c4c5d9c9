"""Plain 64-bit attention for the tests of the shared-prefix and scored calls, and seeded inputs."""
from __future__ import annotations

import math

import torch

D = 128


def gen(seed: int) -> torch.Generator:
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def nan_past(x, lengths):
    """Fills rows at and past each leading index's length with NaN, in place. x [N][H][cap][D]."""
    past = torch.arange(x.shape[2], device="cuda")[None, :] >= lengths[:, None]
    return x.masked_fill_(past[:, None, :, None], math.nan)


def ring(B, H, n, fill, g, seed=0):
    """(ring_k, ring_v, wp, fill): empty slots NaN."""
    fill = ints(fill)
    wp = torch.randint(0, n, (B,), generator=g, device="cuda", dtype=torch.int32)
    rk, rv = randn((B, H, n, D), g), randn((B, H, n, D), g)
    age = torch.remainder(wp[:, None].long() - 1 - torch.arange(n, device="cuda"), n) + 1
    empty = age > fill[:, None]
    rk.masked_fill_(empty[:, None, :, None], math.nan)
    rv.masked_fill_(empty[:, None, :, None], math.nan)
    return rk, rv, wp, fill


def slots_oldest_first(wp: int, fill: int, n: int):
    return torch.tensor([(wp - fill + j) % n for j in range(fill)], dtype=torch.long, device="cuda")


def attend(q, k, v, bias=None, softcap=0.0, scale=None):
    """q [T][D], k / v [K][D], bias [T][K] (-inf: not seen), all f64: out, lse, and sum of weight * |v|."""
    s = (q @ k.T) * (1.0 / math.sqrt(D) if scale is None else scale)
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    if bias is not None:
        s = s + bias
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    if s.shape[1] == 0:
        return out, lse, size
    some = ~torch.isneginf(s).all(1)
    lse[some] = torch.logsumexp(s[some], 1)
    w = torch.exp(s[some] - lse[some][:, None])
    out[some], size[some] = w @ v, w @ v.abs()
    return out, lse, size
