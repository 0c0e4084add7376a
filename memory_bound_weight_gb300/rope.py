"""Cosine and sine tables of rotary positions, for kv4_append.

Pair i of the R rotated dimensions turns by position * f_i, f_i = base^(-2i/R)
(rotary embedding of Su et al., "RoFormer", sec. 3.4.2). For contexts longer
than those trained on, `scaling` changes the frequencies:

  {"type": "linear", "factor": s}: f_i / s (position interpolation, Chen et
      al. 2023).
  {"type": "ntk", "factor": s}: base * s^(R/(R-2)), so that the slowest pair
      turns s times slower and the fastest as before.
  {"type": "yarn", "factor": s, "original_max": n, "beta_fast": 32, "beta_slow":
      1}: pairs that turn more than beta_fast times over n positions keep f_i,
      those that turn less than beta_slow times take f_i / s, a linear ramp over
      the pair's index between; cosines and sines times "attention_factor",
      0.1 ln s + 1 by default (Peng et al., "YaRN", sec. 3).
  {"type": "llama3", "factor": s, "original_max": n, "low_freq_factor": a,
      "high_freq_factor": b}: f_i where a turn takes fewer than n / b positions,
      f_i / s where it takes more than n / a, between them a mix linear in the
      number of turns over n positions (Llama 3.1's published configuration).

Angles are formed in 64 bits: at position 100,000 an fp32 angle is off by up
to 0.004.
"""
from __future__ import annotations

import math


def rope_frequencies(rotary_dim, base=10000.0, scaling=None):
    """(frequencies float64 (rotary_dim / 2,), factor on cosines and sines)."""
    import torch

    if rotary_dim < 16 or rotary_dim % 16:
        raise ValueError("rotary_dim must be a positive multiple of 16")
    if not base > 1:
        raise ValueError("base must be above 1")
    s = dict(scaling or {"type": "none"})
    kind = s.pop("type", None)
    pair = torch.arange(rotary_dim // 2, dtype=torch.float64)
    factor = float(s.pop("factor", 1.0))
    if not factor >= 1:
        raise ValueError("factor must be at least 1")
    if kind == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = torch.pow(torch.tensor(float(base), dtype=torch.float64), -2 * pair / rotary_dim)
    times = 1.0
    if kind == "linear":
        freq = freq / factor
    elif kind == "yarn":
        n = float(s.pop("original_max"))
        fast, slow = float(s.pop("beta_fast", 32)), float(s.pop("beta_slow", 1))
        times = float(s.pop("attention_factor", 0.1 * math.log(factor) + 1))

        def index(turns):  # the pair that turns so often over n positions
            return rotary_dim * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(index(fast)), 0)
        hi = min(math.ceil(index(slow)), rotary_dim - 1)
        ramp = ((pair - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
    elif kind == "llama3":
        n = float(s.pop("original_max"))
        a, b = float(s.pop("low_freq_factor", 1)), float(s.pop("high_freq_factor", 4))
        turns = n * freq / (2 * math.pi)
        keep = ((turns - a) / (b - a)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
    elif kind not in ("none", "ntk"):
        raise ValueError(f"unknown scaling type {kind!r}")
    if s:
        raise ValueError(f"unknown scaling keys {sorted(s)}")
    return freq, times


def rope_table(max_pos, rotary_dim, base=10000.0, scaling=None, device="cuda"):
    """fp32 (max_pos, rotary_dim): per position rotary_dim / 2 cosines, then the sines."""
    import torch

    if max_pos < 1:
        raise ValueError("max_pos must be positive")
    freq, times = rope_frequencies(rotary_dim, base, scaling)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq.to(device)
    return torch.cat((angle.cos() * times, angle.sin() * times), 1).float()
