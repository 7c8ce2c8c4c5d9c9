"""Pair frequencies of rswa_rope_1d, made once on the host.

A rotary encoding of ``rot_dim`` dims turns pair i by pos * base^(-2i / rot_dim). Positions past
the trained length are brought back into it by changing the frequencies alone:

* ``"linear"``: every frequency divided by ``factor`` (positions squeezed evenly);
* ``"ntk"``: the base raised to base * factor^(rot_dim / (rot_dim - 2)), so that the slowest pair is
  divided by ``factor`` and the fastest is kept;
* ``"by_parts"``: by how often a pair turns within the trained length L (L f / 2 pi turns): at most
  ``slow`` turns: divided by ``factor``; at least ``fast``: kept; a linear ramp between. It
  comes with an attention factor 0.1 ln(factor) + 1 on cos and sin (``mscale``).
"""
from __future__ import annotations

import math

import torch


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               trained: int | None = None, slow: float = 1.0, fast: float = 32.0):
    """(inv_freq, mscale) for rswa_rope_1d: f64 [rot_dim / 2] on the CPU, and the factor on cos and sin."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and >= 2 (got {rot_dim})")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError("base must be finite and > 0")
    if scaling not in (None, "linear", "ntk", "by_parts"):
        raise ValueError(f"scaling: expected None, 'linear', 'ntk' or 'by_parts', got {scaling!r}")
    if scaling is not None and not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("factor must be finite and >= 1")
    if scaling == "ntk":
        if rot_dim == 2:
            raise ValueError("scaling 'ntk' needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = torch.tensor([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=torch.float64)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "by_parts":
        if trained is None or trained < 1:
            raise ValueError("scaling 'by_parts' needs the trained length")
        if not 0 <= slow < fast:
            raise ValueError("slow and fast turns must satisfy 0 <= slow < fast")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0
