"""Oracle of the paged-cache operators -- TEST INFRASTRUCTURE ONLY, as ``oracle/attention.py``.

Plain NumPy definitions, one token or one query row at a time where that is the simplest way to
write them: the rotation in fp64, the 4-bit format from the numbers it can hold (nearest by search,
ties to the even code), and attention over a sequence's first tokens in fp64.  ``quantise_f32``
does the format's arithmetic in IEEE fp32, which is what the stored bytes are defined by.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values() -> np.ndarray:
    """Values of the 128 non-negative e4m3 codes (the last is NaN)."""
    c = np.arange(128)
    e, f = c >> 3, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return v


def nearest(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Index of the nearest of ascending ``values`` for each x >= 0, ties to the even index,
    saturating at the last."""
    x = np.asarray(x)
    mid = (values[:-1] + values[1:]) / 2            # exact: neighbours of a small format
    lo = np.searchsorted(mid, x, side="left")       # values[lo] is nearest, the lower one at a tie
    tie = (lo < len(mid)) & (x == mid[np.minimum(lo, len(mid) - 1)])
    return np.where(tie & (lo % 2 == 1), lo + 1, lo)


def quantise_f32(x: np.ndarray, descale: float):
    """(codes, scales) uint8 [..., d] and [..., d/16] of fp32 x, in fp32 arithmetic."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    d = np.float32(descale)
    s = nearest(np.abs(b).max(-1) / (np.float32(6) * d), e4m3_values()[:127]).astype(np.uint8)
    f = (e4m3_values()[s].astype(np.float32) * d)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(f > 0, np.abs(b) / f, np.float32(0))
    code = nearest(y, E2M1[:8]) + 8 * np.signbit(b)
    return code.astype(np.uint8).reshape(x.shape), s


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(packed: np.ndarray, scales: np.ndarray, descale: float) -> np.ndarray:
    """fp64 values of packed codes and scales (code * scale * the fp32 descale)."""
    code = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])
    s = np.concatenate((e4m3_values(), -e4m3_values()))[scales]
    return E2M1[code] * np.repeat(s, 16, -1) * np.float64(np.float32(descale))


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [heads, d] at one position; cos, sin [rotary/2]."""
    y = np.array(x, dtype=np.float64)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, a] = x[:, a] * cos[i] - x[:, b] * sin[i]
        y[:, b] = x[:, b] * cos[i] + x[:, a] * sin[i]
    return y


def rotate_f32(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """The same, each product and sum rounded to fp32."""
    x, c, s = (np.asarray(v, np.float32) for v in (x, cos, sin))
    y = x.copy()
    half = len(c)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def places(cu, seqlens, table, block_size):
    """[(token, sequence, position, page, row)] of every token that a sequence owns."""
    out = []
    for b in range(len(seqlens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = seqlens[b] - n + i
            out.append((cu[b] + i, b, p, int(table[b][p // block_size]), p % block_size))
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, seen):
    """Query rows q [n, d] over k, v [len, d] in fp64, row i over the first seen[i] keys.

    Returns (O [n, d], lse [n], bound_o [n, d], bound_lse [n]): the bounds on a result computed with
    fp32 scores and sums, weights rounded to fp16 and O to bf16:
      a score sums d products, each term off by at most (d + 2) 2^-24 of its size, so by e in all,
      a weight by e^(2e) - 1 <= 2.2 e of itself, and by 2^-11 in fp16 or half of fp16's smallest step,
      2^-25, where the row's largest weight is 2^7 or more (2^-32 of that one), exponentials and
      logarithms by 2^-21 more.
    """
    n, d = q.shape
    o, lse = np.zeros((n, d)), np.full(n, -np.inf)
    bo, bl = np.zeros((n, d)), np.zeros(n)
    for i in range(n):
        m = int(seen[i])
        if m <= 0:
            continue
        s = (k[:m] @ q[i]) * scale
        top = s.max()
        e = np.exp(s - top)
        l = e.sum()
        o[i] = (e / l) @ v[:m]
        lse[i] = top + np.log(l)
        err = (d + 4) * 2.0 ** -24 * scale * (np.abs(k[:m]) @ np.abs(q[i])).max() + 2.0 ** -21 + np.abs(s).max() * 2.0 ** -22
        weight = (e / l) @ np.abs(v[:m])
        tiny = 2.0 ** -32 * np.abs(v[:m]).sum(0) / l
        bo[i] = 2.0 ** -8 * np.abs(o[i]) + (2.2 * err + 2.0 ** -11 + 2.0 ** -20) * weight + tiny + 1e-30
        bl[i] = 1.1 * err + 2.0 ** -21 + np.abs(lse[i]) * 2.0 ** -22
    return o, lse, bo, bl
