"""Rotary position embedding as the append kernel takes it: frequencies (host numbers, 64 bits) and pair layout."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence


class _Rotary(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("gain", ctypes.c_float),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class Rotary:
    """Rotation of the first ``rotary_dim`` elements of a head: pair i turns by position * base^(-2 i / rotary_dim).

    Pairs are (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with ``interleaved``.  ``scaling`` stretches the positions for
    contexts longer than the model was trained on:

    * ``{"type": "linear", "factor": s}``: every frequency divided by s;
    * ``{"type": "ntk", "factor": s}``: base * s^(R / (R - 2)), which divides the slowest frequency by s and keeps the
      fastest;
    * ``{"type": "yarn", "factor": s, "original_max_position": n, "beta_fast": 32, "beta_slow": 1,
      "attention_factor": None}``: frequencies that make more than beta_fast turns in n positions stay, those that make
      fewer than beta_slow are divided by s, a ramp over the dimensions between; cosine and sine are multiplied by
      attention_factor (0.1 ln s + 1 unless given).
    """

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[dict] = None):
        rot, base = int(rotary_dim), float(base)
        if rot < 16 or rot % 16:
            raise ValueError(f"rotary_dim {rot} is not a positive multiple of 16")
        if not base > 1.0 or math.isinf(base):
            raise ValueError("base must be a finite number above 1")
        freq, gain = [base ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
        if scaling is not None:
            freq, gain = _scaled(rot, base, freq, dict(scaling))
        self._set(freq, interleaved, gain)

    @classmethod
    def from_frequencies(cls, inv_freq: Sequence[float], interleaved: bool = False, gain: float = 1.0) -> "Rotary":
        """Frequencies of one's own, radians a position: rotary_dim / 2 of them."""
        self = cls.__new__(cls)
        freq = [float(f) for f in inv_freq]
        if not freq or len(freq) % 8:
            raise ValueError("the number of frequencies must be a positive multiple of 8")
        self._set(freq, interleaved, gain)
        return self

    def _set(self, freq, interleaved, gain):
        if not all(math.isfinite(f) for f in freq) or not math.isfinite(gain):
            raise ValueError("frequencies and gain must be finite")
        self.inv_freq, self.interleaved, self.gain = tuple(freq), bool(interleaved), float(gain)
        self.rotary_dim = 2 * len(freq)
        self._array = (ctypes.c_double * len(freq))(*freq)
        self._struct = _Rotary(self.rotary_dim, int(self.interleaved), self.gain,
                               ctypes.cast(self._array, ctypes.POINTER(ctypes.c_double)))
        self._ref = ctypes.byref(self._struct)


def _scaled(rot, base, freq, s):
    kind, factor = s.pop("type", None), float(s.pop("factor", 0.0))
    if not factor >= 1.0 or math.isinf(factor):
        raise ValueError("scaling needs a finite factor of at least 1")
    if kind == "linear":
        out, gain = [f / factor for f in freq], 1.0
    elif kind == "ntk":
        wide = base * factor ** (rot / (rot - 2))
        out, gain = [wide ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    elif kind == "yarn":
        length = float(s.pop("original_max_position", 0))
        fast, slow = float(s.pop("beta_fast", 32.0)), float(s.pop("beta_slow", 1.0))
        given = s.pop("attention_factor", None)
        if not length >= 1 or not fast > slow > 0:
            raise ValueError("yarn scaling needs original_max_position and beta_fast > beta_slow > 0")

        def dim_of(turns):  # the (fractional) pair whose frequency makes this many turns in `length` positions
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(dim_of(fast)), 0)
        high = min(math.ceil(dim_of(slow)), rot - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        out = [f / factor * r + f * (1.0 - r) for f, r in zip(freq, ramp)]
        gain = 0.1 * math.log(factor) + 1.0 if given is None else float(given)
    else:
        raise ValueError(f"unknown scaling type {kind!r}")
    if s:
        raise ValueError(f"unknown scaling entries {sorted(s)}")
    return out, gain
