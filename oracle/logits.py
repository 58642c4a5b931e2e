"""Adjusted codebook logits and their greedy ids (test infrastructure only: the oracle).

ZONOS2 page of the sglang-omni cookbook, request parameters (repetition penalty).  Reading taken: the penalty
divides a positive logit and multiplies another one; presence and frequency penalties, a bias per id and a
mask of allowed ids follow in that order; the ids counted are those of the same codebook in the stream's
history.  float64; the greedy id takes the lowest of the largest values among the allowed ones.
"""
from __future__ import annotations

import numpy as np


def adjust_logits(logits, history=None, hist_lens=None, repetition=None, presence=None, frequency=None, bias=None,
                  allowed=None) -> np.ndarray:
    """logits [T, N, V]; history [T, L, N]; allowed: truth values [T, N, V]."""
    z = np.array(logits, np.float64)
    T, N, V = z.shape
    for t in range(T):
        for n in range(N):
            counts = np.zeros(V)
            if history is not None:
                L = history.shape[1] if hist_lens is None else min(max(int(hist_lens[t]), 0), history.shape[1])
                for v in history[t, :L, n]:
                    if 0 <= v < V:
                        counts[v] += 1
            hit = counts > 0
            row = z[t, n]
            if repetition is not None:
                r = float(repetition[t])
                row = np.where(hit, np.where(row > 0, row / r, row * r), row)
            if frequency is not None:
                row = row - float(frequency[t]) * counts
            if presence is not None:
                row = np.where(hit, row - float(presence[t]), row)
            z[t, n] = row
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
    return z


def allowed_greedy(stored, allowed=None) -> np.ndarray:
    """The greedy ids [T, N] of values [T, N, V] as they are stored: -1 where no id is allowed and a number."""
    stored = np.asarray(stored, np.float64)
    can = ~np.isnan(stored) if allowed is None else allowed & ~np.isnan(stored)
    ids = np.full(stored.shape[:2], -1, np.int64)
    for t in range(stored.shape[0]):
        for n in range(stored.shape[1]):
            for v in np.flatnonzero(can[t, n]):
                if ids[t, n] < 0 or stored[t, n, v] > stored[t, n, ids[t, n]]:
                    ids[t, n] = v
    return ids


def mask_bits(allowed: np.ndarray) -> np.ndarray:
    """Truth values [T, N, V] -> int32 words [T, N, ceil(V / 32)], id v at bit v % 32 of word v // 32."""
    T, N, V = allowed.shape
    w = np.zeros((T, N, (V + 31) // 32), np.uint32)
    for v in range(V):
        w[:, :, v // 32] |= allowed[:, :, v].astype(np.uint32) << np.uint32(v % 32)
    return w.view(np.int32)
