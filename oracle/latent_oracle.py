"""Plain CPU oracle for the latent cache in 16, 8 or 4 bits.

TEST INFRASTRUCTURE ONLY, like the other modules of this package.

What a cache row holds (include/misa_latent.h): 512 latent entries in 16 groups
of 32, each entry an element of e4m3 ("mx8") or e2m1 ("mx4") times its group's
power of two, and 64 rotary entries as they are.  Elements are found by looking
through the table of all of them, so that neither the bit tricks nor the
hardware conversions of the kernels are repeated here.  float64 throughout.
"""
from __future__ import annotations

import numpy as np

__all__ = ["latent_elements", "latent_bytes", "latent_values", "latent_quantise"]

DV, DQK, GROUP = 512, 576, 32
E_MIN, E_MAX = -117, {"mx8": 119, "mx4": 125}


def latent_elements(form: str) -> np.ndarray:
    """The non-negative elements by code: 0 .. 0x7E of e4m3 (0x7F is NaN), 0 .. 7 of e2m1."""
    man_bits, bias, last = (3, 7, 0x7E) if form == "mx8" else (1, 1, 7)
    out = []
    for code in range(last + 1):
        e, m = code >> man_bits, code & ((1 << man_bits) - 1)
        out.append(m * 2.0 ** (1 - bias - man_bits) if e == 0 else (1 + m / 2.0 ** man_bits) * 2.0 ** (e - bias))
    return np.array(out)


def _nearest(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Code of the table entry nearest to x >= 0; a tie goes to the even code."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dlo, dhi = x - table[lo], table[hi] - x
    return np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)


def latent_quantise(rows: np.ndarray, form: str):
    """rows [..., 576] float64 -> (codes [..., 512] with the sign in the top bit,
    scale bytes [..., 16], rotary part [..., 64])."""
    rows = np.asarray(rows, dtype=np.float64)
    table = latent_elements(form)
    sign_bit = 0x80 if form == "mx8" else 8
    codes = np.zeros(rows.shape[:-1] + (DV,), dtype=np.uint8)
    scales = np.zeros(rows.shape[:-1] + (DV // GROUP,), dtype=np.uint8)
    for g in range(DV // GROUP):
        x = rows[..., g * GROUP:(g + 1) * GROUP]
        ok = np.isfinite(x).all(-1)
        amax = np.where(ok, np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1), 0.0)
        e = np.full(amax.shape, E_MIN)
        for step in range(E_MIN, E_MAX[form]):       # the smallest e whose largest element covers amax
            e = np.where((e == step) & (amax > table[-1] * 2.0 ** step), step + 1, e)
        y = np.where(ok[..., None], x, 0.0) / 2.0 ** e[..., None].astype(np.float64)
        c = _nearest(np.abs(y), table).astype(np.uint8)
        codes[..., g * GROUP:(g + 1) * GROUP] = np.where(np.signbit(y), c | sign_bit, c)
        scales[..., g] = np.where(ok, e + 127, 255)
    return codes, scales, rows[..., DV:]


def latent_values(rows: np.ndarray, form: str) -> np.ndarray:
    """rows [..., 576] float64 -> the numbers a cache of this form holds of them."""
    rows = np.asarray(rows, dtype=np.float64)
    if form == "bf16":
        return rows.copy()
    codes, scales, rope = latent_quantise(rows, form)
    sign_bit = 0x80 if form == "mx8" else 8
    mag = latent_elements(form)[codes & (sign_bit - 1)]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    v = np.where(codes & sign_bit, -mag, mag) * np.repeat(s, GROUP, -1)
    return np.concatenate([v, rope], -1)


def latent_bytes(rows: np.ndarray, form: str) -> np.ndarray:
    """rows [..., 576] float64 (bf16 numbers) -> cache rows [..., 656 or 400] uint8."""
    codes, scales, rope = latent_quantise(rows, form)
    if form == "mx4":
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    bits = (np.ascontiguousarray(rope, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.concatenate([codes, scales, np.ascontiguousarray(bits).view(np.uint8)], -1)
