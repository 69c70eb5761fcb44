"""Rotary frequency tables for cq_rope_qkv, scaled for contexts longer than the
one a model was trained on.  Host side, fp64, rounded to fp32 once.

Channel pair i of rot_dim / 2 turns by theta_i = base^(-2i / rot_dim) per
position.  With factor s = wanted context / trained context:

  none     theta_i
  linear   theta_i / s                    (positions interpolated)
  base     theta_i of base * s^(rot_dim / (rot_dim - 2)): the fastest pair is
           kept, the slowest is divided by s
  parts    with n_i = context * theta_i / (2 pi), the turns that pair i makes over
           the trained context, and g from 1 (kept) to 0 (divided by s):
           theta_i * (g + (1 - g) / s).  Two ramps for g, which differ by 40 % and
           more in pairs between their ends:
             turns   (n_i - slow_turns) / (fast_turns - slow_turns), clipped, as the
                     YaRN paper writes its interpolation by parts
             index   1 - (i - low) / (high - low), clipped: a line over the pair's
                     index from the last pair that makes fast_turns or more
                     (low) to the first that makes slow_turns or less (high).
                     Models released with YaRN scaling are run with this one: a
                     table for such a model needs ramp="index"
"""
from __future__ import annotations

import math

import numpy as np


def rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  context: int | None = None, slow_turns: float = 1.0,
                  fast_turns: float = 32.0, ramp: str = "turns") -> np.ndarray:
    """fp32 [rot_dim / 2] table of angles per position (see the module's text)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    theta = np.power(float(base), -2.0 * i / rot_dim)
    if scaling in ("none", "base"):
        pass
    elif scaling == "linear":
        theta = theta / factor
    elif scaling == "parts":
        if context is None or context <= 0:
            raise ValueError("scaling 'parts' needs the trained context")
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must exceed slow_turns")
        if ramp == "turns":
            turns = context * theta / (2.0 * math.pi)
            g = np.clip((turns - slow_turns) / (fast_turns - slow_turns), 0.0, 1.0)
        elif ramp == "index":
            if not base > 1 or not slow_turns > 0:
                raise ValueError("ramp 'index' needs base > 1 and slow_turns > 0")

            def index(n):  # where a pair makes n turns: context base^(-2i / rot_dim) = 2 pi n
                return rot_dim * math.log(context / (2.0 * math.pi * n)) / (2.0 * math.log(base))

            low = max(math.floor(index(fast_turns)), 0)
            high = min(math.ceil(index(slow_turns)), rot_dim - 1)
            g = 1.0 - np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        else:
            raise ValueError(f"unknown ramp {ramp!r}")
        theta = theta * (g + (1.0 - g) / factor)
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return theta.astype(np.float32)


def rope_attn_scale(factor: float) -> float:
    """The YaRN paper's attention temperature, as a factor on the turned q and
    k: 0.1 ln(s) + 1 for a context stretched by s > 1, else 1."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
