"""The 8-bit pool in numpy: e4m3 codes, quantisation of rows, and attention over what they stand for.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the definition, without any of
the library's code: codes are decoded from their bits, rounding is a search over the sorted code
values, and attention is the float64 definition over code * scale.
"""
from __future__ import annotations

import numpy as np

from . import attention as A

E4M3_MAX = 448.0
MIN_SCALE = np.float32(2.0 ** -126)


def _code_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent
    0 is subnormal, 0x7f and 0xff are NaN, there are no infinities."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


VALUES = _code_values()


def encode(x: np.ndarray) -> np.ndarray:
    """The nearest code of x, ties to the even mantissa, saturating at +-448; keeps the sign of
    zero.  x: finite float64."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    grid = VALUES[:127]                     # 0 .. 448, increasing, code = index
    hi = np.clip(np.searchsorted(grid, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = mag - grid[lo], grid[hi] - mag
    pick_hi = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    code = np.where(pick_hi, hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(bits: np.ndarray):
    """bf16 rows (bit patterns [..., 128]) -> codes uint8 [..., 128], scales float32 [...]: scale =
    max(a / 448, 2^-126), code = e4m3(x r), r = 448 / a (2^126 at the floor), all in float32; a row
    that is not finite: scale NaN, codes 0."""
    x = A.bf16_to_f64(bits).astype(np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(x).max(axis=-1)
        fine = np.isfinite(x).all(axis=-1)
        scale = np.maximum(a / np.float32(E4M3_MAX), MIN_SCALE)
        r = np.where(scale > MIN_SCALE, np.float32(E4M3_MAX) / a,
                     np.float32(1) / MIN_SCALE).astype(np.float32)
        y = x * r[..., None]
        codes = encode(np.where(fine[..., None], y, 0.0))
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What a pool's rows stand for, float64."""
    return VALUES[codes] * np.asarray(scales, np.float64)[..., None]


def attend_rows(q, keys, vals, vscale, visible, scale):
    """Attention of query rows over key rows, with what its error bounds need: o, lse, and per row
    the sum of p_j |v_j| (per column), the largest scale * sum_d |q_d k_jd| over the visible keys,
    and the largest p_j * vscale_j."""
    o, lse = A.attend(q, keys, vals, visible, scale)
    s = np.where(visible, scale * (q @ keys.T), -np.inf)
    p = np.exp(s - np.where(np.isfinite(lse), lse, 0.0)[:, None])
    sabs = np.where(visible, scale * (np.abs(q) @ np.abs(keys).T), 0.0).max(axis=1, initial=0.0)
    return o, lse, p @ np.abs(vals), sabs, (p * vscale[None, :]).max(axis=1, initial=0.0)


def extend(q, k, v, req_to_token, req_idx, prefix_len, extend_len, cu_q, scale):
    """As attention.extend over float64 pools k, v [P, Hkv, 128] (see `values`)."""
    n_rows, hq, d = q.shape
    gq = hq // k.shape[1]
    o, lse = np.full((n_rows, hq, d), np.nan), np.full((n_rows, hq), np.nan)
    for r in range(len(req_idx)):
        p, e = int(prefix_len[r]), int(extend_len[r])
        at = np.asarray(req_to_token[req_idx[r], :p + e], np.int64)
        rows = slice(int(cu_q[r]), int(cu_q[r]) + e)
        visible = np.arange(p + e)[None, :] <= (p + np.arange(e))[:, None]
        x = A.bf16_to_f64(q[rows])
        for h in range(hq):
            o[rows, h], lse[rows, h] = A.attend(x[:, h], k[at, h // gq], v[at, h // gq], visible,
                                                scale)
    return o, lse


def decode(q, k, v, req_to_token, req_idx, seq_len, scale):
    """As attention.decode over float64 pools k, v [P, Hkv, 128]."""
    n = len(req_idx)
    return extend(q, k, v, req_to_token, req_idx, np.asarray(seq_len) - 1, np.ones(n, np.int64),
                  np.arange(n + 1), scale)
