"""Plain 64-bit references (numpy, CPU) of the norm, of 8-bit activations and their
product with ternary weights, and of the routing, written from their definitions,
with the error bounds that their tests use."""
from __future__ import annotations

import numpy as np
import torch

from mx_util import EPS, TINY, assert_close, dense, f64, pack_ternary  # noqa: F401

STEP = 2.0 ** -24   # half a step of fp32


def rounded(v: np.ndarray, dtype) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(v)).to(dtype).double().numpy()


def stream(x: torch.Tensor, residual):
    """What the residual stream holds after the addition, in 64 bits."""
    if residual is None:
        return f64(x)
    # one rounding of the exact sum: fp32 sums of 16-bit values are exact where they lie near a border
    return rounded(f64(x) + f64(residual), residual.dtype)


def blocks(v: np.ndarray, group: int) -> np.ndarray:
    M, K = v.shape
    return v.reshape(M, K // group, group) if group else v.reshape(M, 1, K)


def quantize(v: np.ndarray, factor: np.ndarray, group: int):
    """(codes [M,K], scales [M,G] in 64 bits) of v, whose rows are meant times factor [M]."""
    M, K = v.shape
    b = blocks(v, group)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        a = np.abs(b).max(-1).astype(np.float32).astype(np.float64)
        bad = ~np.isfinite(a)
        safe = np.where(bad | (a == 0), 1.0, a)
        q = np.rint(127.0 * b / safe[..., None])
        q = np.where((bad | (a == 0))[..., None], 0.0, q)
        s = np.where(bad, np.nan, np.where(a == 0, np.where(np.isnan(factor), np.nan, 0.0)[:, None],
                                           a * factor[:, None] / 127.0))
    return q.reshape(M, K).astype(np.int8), s


def norm(x: torch.Tensor, weight, eps: float, residual):
    """(h, y, v, f): the stream, the normed values, h w and the rows' factors."""
    h = stream(x, residual)
    w = f64(weight) if weight is not None else np.ones(h.shape[1])
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        f = 1.0 / np.sqrt((h * h).sum(-1) / h.shape[1] + np.float64(np.float32(eps)))
        return h, h * f[:, None] * w, h * w, f


def norm_bound(y: np.ndarray, dtype) -> np.ndarray:
    """The factor's rounding and two products in fp32, then the output's rounding; what
    those products lose below fp32's normal range is less than its smallest number."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.abs(y) * (4 * STEP + EPS[dtype] * (1 + 4 * STEP)) + TINY[dtype] + 2.0 ** -126 * EPS[torch.float32]


def product(q: np.ndarray, xs: np.ndarray, packed: np.ndarray, ws: np.ndarray, dtype):
    """(y, bound).  A block's sum is an exact integer; it meets the activations' and the
    weights' scale (two roundings), the sum over blocks takes one addition each, in any
    order, and one rounding to the output type."""
    M, K = q.shape
    N, G = ws.shape
    t = dense(packed, np.ones((N, G)))
    qg = q.astype(np.float64).reshape(M, G, 128)
    tg = t.reshape(N, G, 128)
    y = np.zeros((M, N))
    B = np.zeros((M, N))
    with np.errstate(invalid="ignore", over="ignore"):
        for g in range(G):
            d = qg[:, g] @ tg[:, g].T
            term = d * xs[:, g if xs.shape[1] > 1 else 0][:, None] * ws[:, g].astype(np.float64)[None, :]
            y += term
            B += np.abs(term)
        bound = (G + 8) * STEP * B
        return y, bound + EPS[dtype] * (np.abs(y) + bound) + TINY[dtype]


def route(logits: np.ndarray, top_k: int, score: str, bias, groups: int, keep: int, best: int, renorm: bool,
          scale: float):
    """(ids [T,k], weights [T,k])."""
    T, E = logits.shape
    per = E // groups
    ids = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))

    def key(v):   # NaN first, then the largest
        return (0, 0.0) if np.isnan(v) else (1, -v)

    for t in range(T):
        l = logits[t]
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                top = l.max() if not np.isnan(l).any() else np.nan
                p = np.where(l == -np.inf, 0.0, np.exp(l - top))
                s = p / p.sum() if p.sum() != 0 else p
            else:
                s = 1.0 / (1.0 + np.exp(-l))
        c = s + bias if bias is not None else l
        sums = s + bias if bias is not None else (s if best == 2 else l)
        open_ = (l != -np.inf) & (c != -np.inf)
        if groups > 1:
            totals = []
            for g in range(groups):
                mine = sorted((e for e in range(g * per, (g + 1) * per) if open_[e]), key=lambda e: key(sums[e]))[:best]
                totals.append(sum(sums[e] for e in mine) if mine else -np.inf)
            has = [any(open_[g * per:(g + 1) * per]) for g in range(groups)]
            order = sorted(range(groups), key=lambda g: (not has[g],) + key(totals[g]) + (g,))
            for g in order[keep:]:
                open_[g * per:(g + 1) * per] = False
        chosen = sorted((e for e in range(E) if open_[e]), key=lambda e: key(c[e]) + (e,))[:top_k]
        ids[t, :len(chosen)] = chosen
        v = s[chosen]
        total = v.sum() if renorm else 1.0
        with np.errstate(invalid="ignore", divide="ignore"):
            w[t, :len(chosen)] = 0.0 if total == 0 else v / total * scale
    return ids, w
