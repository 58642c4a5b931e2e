"""The paged key-value cache and the attention of one new token (test infrastructure only: the oracle).

ZONOS2 Technical Report digest, "method overview and architecture", item 5: grouped-query attention with
headwise gating and rotary positions; "Builds on" lists the rotary embedding and query/key norms.
Readings taken where the pages are silent: the rotation turns pair i of a head's first R columns by
p * inv_freq[i], the pairs being (i, i + R / 2) or (2 i, 2 i + 1); the optional norm is RMSNorm over a head
with a gain of the head's width, before the rotation; the gate is the sigmoid of one value per head on the
attention's output.  The cache is [n_pages, Hkv, page_size, D]; row p of a sequence lies in page
table[s, p // page_size], row p % page_size.  float64, plain loops over tokens and sequences.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from .embed import rmsnorm


def rotate(x: np.ndarray, pos: int, inv_freq: np.ndarray, interleaved: bool) -> np.ndarray:
    """The heads x [H, D] of one token at position pos, their first 2 len(inv_freq) columns turned."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        w = float(pos) * float(inv_freq[i])
        u, z = x[:, a].copy(), x[:, b].copy()
        x[:, a] = u * np.cos(w) - z * np.sin(w)
        x[:, b] = u * np.sin(w) + z * np.cos(w)
    return x


def append_rows(q, k, v, pos, inv_freq, interleaved=False, q_gamma=None, k_gamma=None, eps=1e-6):
    """The rows that one call stores: (q [T, Hq, D], k, v [T, Hkv, D]) float64, unrounded."""
    inv_freq = np.zeros(0) if inv_freq is None else np.asarray(inv_freq, np.float64)

    def one(x, gamma, t):
        y = np.asarray(x[t], np.float64)
        if gamma is not None:
            y = rmsnorm(y, gamma, eps)
        return rotate(y, int(pos[t]), inv_freq, interleaved)

    T = len(pos)
    qr = None if q is None else np.stack([one(q, q_gamma, t) for t in range(T)])
    return qr, np.stack([one(k, k_gamma, t) for t in range(T)]), np.asarray(v, np.float64)


def paged_rows(cache: np.ndarray, table_row: np.ndarray, n: int) -> np.ndarray:
    """The first n rows of a sequence, [n, Hkv, D], of a cache [n_pages, Hkv, page_size, D]."""
    page = cache.shape[2]
    return np.stack([cache[table_row[p // page], :, p % page] for p in range(n)])


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, gate: Optional[np.ndarray] = None):
    """One token's queries q [Hq, D] over k, v [n, Hkv, D]: (out [Hq, D], lse [Hq]); zeros and -inf for n = 0."""
    Hq, D = q.shape
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if len(k):
        G = Hq // k.shape[1]
        for i in range(Hq):
            s = scale * (k[:, i // G].astype(np.float64) @ q[i].astype(np.float64))
            top = s.max()
            p = np.exp(s - top)
            out[i] = (p / p.sum()) @ v[:, i // G].astype(np.float64)
            lse[i] = top + np.log(p.sum())
    if gate is not None:
        out = out / (1 + np.exp(-np.asarray(gate, np.float64)))[:, None]
    return out, lse
