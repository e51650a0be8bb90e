"""Plain 64-bit forms of what stands between a served layer's products: the
root-mean-square norm with its codes, activations, and attention with capped
scores, a bias by distance and a prefix.  Used by the tests only; shares no
code with the library."""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

from .serving_oracle import row_codes


def added(x: np.ndarray, residual: Optional[np.ndarray]) -> np.ndarray:
    """h = x + residual as the definition rounds it, to fp32."""
    return x.astype(np.float32) if residual is None else x.astype(np.float32) + residual.astype(np.float32)


def norm_factor(h: np.ndarray, eps: float) -> np.ndarray:
    return 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(axis=-1) + float(np.float32(eps)))


def norm(h: np.ndarray, weight: Optional[np.ndarray], eps: float) -> np.ndarray:
    """The normed rows of fp32 h, in fp64."""
    w = 1.0 if weight is None else weight.astype(np.float64)
    return norm_factor(h, eps)[:, None] * h.astype(np.float64) * w


def norm_codes(h: np.ndarray, weight: Optional[np.ndarray], eps: float) -> Tuple[np.ndarray, np.ndarray]:
    """Codes of the rows u = h weight (fp32) and scales factor max|u| / 127 in fp64, NaN for rows that are not finite."""
    with np.errstate(all="ignore"):
        u = h if weight is None else h * weight.astype(np.float32)
        codes, _ = row_codes(u, 127)
        bad = ~np.isfinite(u).all(axis=-1)
        scale = norm_factor(h, eps) * np.abs(u.astype(np.float64)).max(axis=-1) / 127
    return codes, np.where(bad, np.nan, scale)


def _erfc(x: np.ndarray) -> np.ndarray:
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def activation(z: np.ndarray, name: Optional[str]) -> np.ndarray:
    z = z.astype(np.float64)
    if name is None:
        return z
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    t = z if name == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    e = np.exp(-np.abs(t))
    return z * np.where(t >= 0, 1.0, e) / (1.0 + e)


def attention(q: np.ndarray, place: int, k: Tuple[np.ndarray, np.ndarray], v: Tuple[np.ndarray, np.ndarray], scale: float,
              cap: Optional[float], slope: float, prefix: int, hidden: Optional[np.ndarray] = None):
    """One token (q [d]) at `place` of its sequence and one head over (codes, scales)
    of L keys and values: sees the keys j <= place and j < prefix that are not
    hidden.  None if it sees none, else a dict: out [d], p, the scores before and
    after the cap, the distances, the seen keys' value rows and reach
    scale sk_j sum_d |q_d| (|ck_jd| + 24)."""
    (kc, ks), (vc, vs) = k, v
    j = np.arange(kc.shape[0])
    see = (j <= place) | (j < prefix)
    if hidden is not None:
        see &= ~hidden
    if not see.any():
        return None
    z = scale * (kc[see] @ q) * ks[see]
    capped = z if cap is None else cap * np.tanh(z / cap)
    away = np.abs(place - j[see]).astype(np.float64)
    s = capped - slope * away
    p = np.exp(s - s.max())
    p /= p.sum()
    return {"out": (p * vs[see]) @ vc[see], "p": p, "z": z, "capped": capped, "away": away, "s": s, "vc": vc[see], "vs": vs[see],
            "reach": scale * ks[see] * ((np.abs(kc[see]) + 24.0) @ np.abs(q))}
