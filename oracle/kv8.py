"""CPU oracle of the 8-bit block cache and the decode attention over it (test infrastructure).

Only the test suite may import this module; it shares no code with the GPU library.  A
sequence is the list of its tokens' 16-bit keys and values; everything a cache may hold of it
(codes, scales, means) follows from the definition block by block, whatever calls brought the
tokens.  Scales and quotients are fp32 by definition (numpy's IEEE division), the rest fp64.
Pinned by ``tests/test_oracle_kv8.py``.
"""
from __future__ import annotations

import numpy as np

from .proj import _f64

BLOCK = 64
TOP = {"e4m3": 448.0, "int8": 127.0}


def code_grid(y, code):
    """The nearest 8-bit value to y, ties to the even code."""
    y = np.asarray(y, np.float64)
    if code == "int8":
        return np.rint(y)
    # e4m3: 3 mantissa bits, exponents down to 2^-6, below that steps of 2^-9
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(y / step) * step


def quantise(x, code):
    """One head's block [64, D] -> (values of its codes, fp32 scale)."""
    x = np.asarray(_f64(x), np.float32)
    amax = np.abs(x).max()
    if not np.isfinite(amax):
        return np.zeros(x.shape), np.float32(np.nan)
    scale = np.maximum(amax * (np.float32(1) / np.float32(TOP[code])), np.float32(2.0 ** -126))
    return code_grid(x / scale, code), scale


def stored(x, code):
    """[S, Hkv, D] tokens -> the values the attention reads: whole blocks before the newest
    token's own block as their codes stand for, the own block as it is."""
    x = _f64(x).copy()
    own = (len(x) - 1) // BLOCK
    for j in range(own):
        for h in range(x.shape[1]):
            y, scale = quantise(x[j * BLOCK:(j + 1) * BLOCK, h], code)
            x[j * BLOCK:(j + 1) * BLOCK, h] = y * np.float64(scale)
    return x


def attend(q, g, k, v, *, code, window, scale=None, blocks=None):
    """The newest token's attention: q, g [Hq, D] (g may be None), k, v [S, Hkv, D] its
    sequence's tokens.  blocks: per KV head the earlier blocks to read.  Returns out [Hq, D], lse [Hq]
    and, for tolerances, the sums of |p v| [Hq, D] and the sums over blocks of their p times
    their largest |v| [Hq]."""
    q, kk, vv = _f64(q), stored(k, code), stored(v, code)
    S, Hkv, D = kk.shape
    scale = D ** -0.5 if scale is None else scale
    p = S - 1
    out, lse, mag, top = np.zeros(q.shape), np.zeros(len(q)), np.zeros(q.shape), np.zeros(len(q))
    for h in range(len(q)):
        kv = h // (len(q) // Hkv)
        seen = np.arange(S) > p - window
        if blocks is not None:
            keep = set(int(j) for j in blocks[kv] if j >= 0) | {p // BLOCK}
            seen &= np.isin(np.arange(S) // BLOCK, list(keep))
        s = kk[seen, kv] @ q[h] * scale
        m = s.max()
        e = np.exp(s - m)
        lse[h] = m + np.log(e.sum())
        w = e / e.sum()
        out[h] = w @ vv[seen, kv]
        mag[h] = w @ np.abs(vv[seen, kv])
        at = np.flatnonzero(seen) // BLOCK
        starts = np.flatnonzero(np.r_[True, at[1:] != at[:-1]])
        top[h] = (np.add.reduceat(w, starts) * np.maximum.reduceat(np.abs(vv[seen, kv]).max(1), starts)).sum()
    if g is not None:
        sg = 1.0 / (1.0 + np.exp(-_f64(g)))
        out, mag, top = out * sg, mag * sg, top * sg.max(1)
    return out, lse, mag, top


def select(q, mean, *, first_block, n_select, n_first, n_last):
    """q [Hq, D], mean [n, Hkv, D] of the candidates first_block ..: per KV head the chosen
    blocks, ascending, padded with -1."""
    q, mean = _f64(q), _f64(mean)
    n, Hkv, _ = mean.shape
    G = len(q) // Hkv
    got = np.full((Hkv, n_select), -1, np.int64)
    for h in range(Hkv):
        with np.errstate(invalid="ignore"):
            score = (mean[:, h] @ q[h * G:(h + 1) * G].T).astype(np.float64)
        score = np.where(np.isnan(score).any(1), -np.inf, score.max(1)) if n else np.zeros(0)
        order = sorted(range(n), key=lambda i: (not (i < n_first or i >= n - n_last), -score[i], i))
        take = sorted(order[:n_select])
        got[h, :len(take)] = np.asarray(take, np.int64) + first_block
    return got
