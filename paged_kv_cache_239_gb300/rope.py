"""``Rope``: rotary frequencies and pair layout for ``BlockPool.norm_rope_write_kv``.

Host data only (the kernel takes the frequencies as arguments), so one object
serves every layer, pool, stream and device.
"""
from __future__ import annotations

from typing import Optional, Sequence

from . import binding as B

_SCALINGS = {"none": B.PA_ROPE_PLAIN, "linear": B.PA_ROPE_LINEAR, "ntk": B.PA_ROPE_NTK,
             "parts": B.PA_ROPE_PARTS}


class Rope:
    """Rotation of the first ``rotary_dim`` elements of a head (a multiple of 16).

    ``interleaved``: the pairs are (2j, 2j + 1), else (j, j + rotary_dim / 2).
    ``scaling``: 'none'; 'linear' (positions divided by ``factor``); 'ntk' (a
    larger base); 'parts' (by wavelength: frequencies that turn at most ``low``
    times over ``original_len`` positions are divided by ``factor``, those that
    turn ``high`` times or more are kept, the rest blended).  ``frequencies``
    (rotary_dim / 2 numbers, radians per position) replaces all of these.
    ``amplitude`` scales the rotated elements.

    The blend of 'parts' is linear in the turns, as in YaRN's formula (low 1, high 32,
    amplitude 0.1 ln(factor) + 1).  Models are also trained with a blend that is linear
    in the pair's index j, between the pairs that turn ``high`` and ``low`` times: other
    numbers in between, which such a model needs given as ``frequencies``.
    """

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 4096,
                 low: float = 1.0, high: float = 4.0, amplitude: float = 1.0,
                 frequencies: Optional[Sequence[float]] = None):
        self.handle = None
        if frequencies is None:
            if scaling not in _SCALINGS:
                raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, not {scaling!r}")
            frequencies = B.pa_rope_frequencies(rotary_dim, base, _SCALINGS[scaling], factor,
                                                original_len, low, high)
        self.rotary_dim, self.interleaved = rotary_dim, bool(interleaved)
        self.amplitude, self.frequencies = float(amplitude), [float(f) for f in frequencies]
        self.handle = B.pa_rope_create(rotary_dim, interleaved, self.frequencies, amplitude)

    def close(self) -> None:
        if getattr(self, "handle", None):
            B.pa_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
