"""Float64 CPU oracle of the layer operators around the verify step: attention of
a round's positions over a shared prefix and a paged cache, the residual RMSNorm
with an 8-bit output, and the matrix product with bias, activation and residual.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see ``oracle/__init__.py``).  Arrays are
float64 (already widened from their storage type); it shares no code with the
CUDA path.

Readings:
  R32 the query at position i of sequence b is that of the token before draft
      i, so it sees the prefix and the own tokens 0 .. L_b + i - 1, where the
      drafts were written at L_b .. L_b + k_b - 1 (the convention of R29).  For
      position 0 to see itself L_b counts its token: a round that follows a
      commit writes the emitted token's keys and values at the committed length
      and passes that length plus one.  A query that sees nothing gets 0 and a
      log-sum of -inf.
  R33 an 8-bit row is e4m3 (4 exponent and 3 mantissa bits, largest value 448)
      with the scale max(max|y| / 448, 2^-126), so that dividing by it stays
      finite; a zero row has zero values.
"""

from __future__ import annotations

import math

import numpy as np

FLAG_BAD_K = 1
FLAG_BAD_N = 256
FLAG_BAD_PAGE = 512

E4M3_MAX = 448.0


def own_tokens(pool, table_row, page_size: int, n: int):
    """Tokens 0..n-1 of one sequence as [n, Hkv, D], page by page."""
    rows = [pool[int(table_row[t // page_size]), t % page_size] for t in range(n)]
    return np.array(rows).reshape((n,) + pool.shape[2:])


def sequence_flags(k: int, K: int, length: int, max_pages: int, page_size: int, table_row,
                   prefix_pages, num_pages: int) -> int:
    """The flag a sequence raises, 0 if it is sound."""
    if not 0 <= k <= K:
        return FLAG_BAD_K
    if length < 0 or length + k > max_pages * page_size:
        return FLAG_BAD_N
    used = -(-(length + k) // page_size)
    ids = list(table_row[:used]) + list(prefix_pages)
    return FLAG_BAD_PAGE if any(not 0 <= int(p) < num_pages for p in ids) else 0


def prefix_attention(q, prefix_k, prefix_v, own_k, own_v, length: int, scale: float):
    """One sequence: q [Q, Hq, D]; prefix [P, Hkv, D]; own [L + Q - 1, Hkv, D].
    Returns out [Q, Hq, D], lse [Q, Hq], weight [Q, Hq, D] = sum p |v| / sum p
    (the scale of the rounding bound) and spread [Q, Hq] = max_j scale sum |q k|."""
    Q, Hq, D = q.shape
    Hkv = own_k.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((Q, Hq, D)), np.full((Q, Hq), -np.inf)
    weight, spread = np.zeros((Q, Hq, D)), np.zeros((Q, Hq))
    for i in range(Q):
        ks = np.concatenate([prefix_k, own_k[: length + i]])
        vs = np.concatenate([prefix_v, own_v[: length + i]])
        if len(ks) == 0:
            continue
        for h in range(Hkv):
            s = scale * (q[i, h * G:(h + 1) * G] @ ks[:, h].T)          # [G, n]
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(axis=1, keepdims=True)
            out[i, h * G:(h + 1) * G] = (p / total) @ vs[:, h]
            weight[i, h * G:(h + 1) * G] = (p / total) @ np.abs(vs[:, h])
            lse[i, h * G:(h + 1) * G] = (m + np.log(total))[:, 0]
            spread[i, h * G:(h + 1) * G] = abs(scale) * (
                np.abs(q[i, h * G:(h + 1) * G]) @ np.abs(ks[:, h]).T).max(axis=1)
    return out, lse, weight, spread


def rmsnorm_residual(x, residual, w, eps: float):
    """(s, y) of one batch of rows."""
    s = x if residual is None else x + residual
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * w[None]
    return s, y


def row_scale(y):
    return np.maximum(np.abs(y).max(axis=1) / E4M3_MAX, 2.0 ** -126)


def e4m3_values():
    """Every finite e4m3 value >= 0, ascending."""
    vals = [m * 2.0 ** -9 for m in range(8)]                            # subnormal
    vals += [(8 + m) / 8 * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)
             if not (e == 15 and m == 7)]
    return np.array(vals)


def activation(z, act: int):
    if act == 1:
        return np.maximum(z, 0)
    if act == 2:
        return z / (1 + np.exp(-z))
    if act == 3:
        return 0.5 * z * (1 + np.vectorize(math.erf)(z / math.sqrt(2)))
    if act == 4:
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(x, W, sx, sw, bias, act: int, residual):
    """(out, absp): the result and sum_k |x W| sx sw, the scale of its rounding."""
    scale = (1.0 if sx is None else sx[:, None]) * (1.0 if sw is None else sw[None])
    z = (x @ W.T) * scale
    absp = (np.abs(x) @ np.abs(W).T) * np.abs(scale)
    if bias is not None:
        z = z + bias[None]
    out = activation(z, act)
    return (out if residual is None else out + residual), absp
