"""Plain 64-bit forms of the serving operators: integer codes of rows, the
product in 8-bit integers, the quantized cache, attention over it.  Used by
the tests only; shares no code with the library."""
from __future__ import annotations

from fractions import Fraction
from typing import List, Sequence, Tuple

import numpy as np


def row_codes(x: np.ndarray, top: int) -> Tuple[np.ndarray, np.ndarray]:
    """Codes and fp32 scales of the rows (last axis) of fp32 x: the integer
    nearest to top x / max|x|, ties to even; rows of zeros: 0, 0; rows with a
    NaN or an infinity: codes 0, scale NaN.  The two sides of a rounding
    border, 2 top |x| and (2 k + 1) max|x|, are compared exactly (fp64 holds
    both)."""
    a = np.abs(x.astype(np.float64))
    bad = ~np.isfinite(a).all(axis=-1)
    a = np.where(bad[..., None], 0.0, a)
    most = a.max(axis=-1, keepdims=True)
    safe = np.where(most > 0, most, 1.0)
    k = np.floor(top * a / safe)
    k = np.where(top * a < k * safe, k - 1, np.where(top * a >= (k + 1) * safe, k + 1, k))  # exact floor
    border = (2 * k + 1) * safe
    up = (2 * top * a > border) | ((2 * top * a == border) & (k % 2 == 1))
    code = np.sign(np.where(np.isfinite(x), x, 0.0).astype(np.float64)) * (k + up)
    scale = (most[..., 0] / top).astype(np.float32)
    return code.astype(np.int64), np.where(bad, np.float32(np.nan), scale)


def row_codes_slow(x: Sequence[float], top: int) -> List[int]:
    """The same for one row in rational numbers."""
    most = max((abs(Fraction(float(v))) for v in x), default=Fraction(0))
    return [0 if most == 0 else round(Fraction(float(v)) * top / most) for v in x]  # round: half to even


def integer_matmul(codes: np.ndarray, scales: np.ndarray, w: np.ndarray, w_scales: np.ndarray,
                   offsets: np.ndarray) -> np.ndarray:
    """sx[t] sw[n] (sum cx w - off sum cx): the integers exact (fp64 holds them), the scales in fp64."""
    s = codes.astype(np.float64) @ w.astype(np.float64).T
    s = s - codes.sum(axis=1).astype(np.float64)[:, None] * offsets.astype(np.float64)[None, :]
    return s * scales.astype(np.float64)[:, None] * w_scales.astype(np.float64)[None, :]


def unpack_rows(held: np.ndarray, bits: int) -> np.ndarray:
    """Codes [..., head_dim] from a cache's bytes."""
    if bits == 8:
        return held.view(np.int8).astype(np.int64)
    u = held.view(np.uint8).astype(np.int64)
    return np.stack([u & 15, u >> 4], axis=-1).reshape(*u.shape[:-1], -1) - 8


def pack_rows(codes: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return codes.astype(np.int8)
    n = (codes + 8).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def cache_rows(held: np.ndarray, scales: np.ndarray, bits: int, pages: Sequence[int], head: int,
               n_keys: int) -> Tuple[np.ndarray, np.ndarray]:
    """Codes [n_keys, head_dim] and scales [n_keys] of one head along a sequence's pages."""
    c = np.concatenate([unpack_rows(held[p, head], bits) for p in pages], axis=0)[:n_keys]
    s = np.concatenate([scales[p, head] for p in pages], axis=0)[:n_keys]
    return c.astype(np.float64), s.astype(np.float64)


def attention(q: np.ndarray, k: Tuple[np.ndarray, np.ndarray], v: Tuple[np.ndarray, np.ndarray], scale: float,
              hidden: np.ndarray | None = None):
    """One sequence, one head: q [n, d] fp64, (codes, scales) of its L keys and
    values; token t sees the keys 0 .. L - n + t that are not hidden.  Returns
    out [n, d] and what the tests' bounds take: sum p |v|, sum p sv, and per
    row max_j over seen keys of scale sk_j sum_d |q_d| (|ck_jd| + 24) and max_j p_j."""
    (kc, ks), (vc, vs) = k, v
    n, L = q.shape[0], kc.shape[0]
    out, absv, plain = (np.zeros((n, vc.shape[1])) for _ in range(3))
    worst, peak = np.zeros(n), np.zeros(n)
    for t in range(n):
        see = np.arange(L) <= L - n + t
        if hidden is not None:
            see = see & ~hidden
        if not see.any():
            continue
        s = scale * (kc[see] @ q[t]) * ks[see]
        with np.errstate(invalid="ignore"):
            p = np.exp(s - s.max())
        p = p / p.sum()
        out[t] = (p * vs[see]) @ vc[see]
        absv[t] = (p * vs[see]) @ np.abs(vc[see])
        plain[t] = (p * vs[see]).sum()
        peak[t] = p.max()
        worst[t] = (scale * ks[see] * ((np.abs(kc[see]) + 24.0) @ np.abs(q[t]))).max()
    return out, absv, plain, worst, peak
