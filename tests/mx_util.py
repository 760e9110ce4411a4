"""Plain 64-bit references (numpy, CPU) of the microscaled 4-bit operators and
of the mixture-of-experts layer, written from their definitions, and the
error bounds that their tests use."""
from __future__ import annotations

import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def quantize(x: np.ndarray):
    """(code values 0..15 [M,K], exponent bytes [M,K/32]) of float64 x holding fp32 values."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(b).max(-1)
        bad = ~np.isfinite(b).all(-1)
        _, e = np.frexp(np.where(bad, 1.0, amax))   # amax in [2^(e-1), 2^e)
        E = np.where(amax > 0, e - 1 - 2, -127)
        E = np.maximum(E, -127)
        v = np.where(bad[..., None], 0.0, b) / np.exp2(E)[..., None].astype(np.float64)
    a = np.minimum(np.abs(v), 6.0)
    hi = np.searchsorted(GRID, a)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code + 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code)
    exps = np.where(bad, 255, E + 127)
    return code.reshape(M, K).astype(np.uint8), exps.astype(np.uint8)


def pack_nibbles(code: np.ndarray) -> np.ndarray:
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def values(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """float64 values of packed codes [R,K/2] and exps [R,K/32]."""
    R, half = codes.shape
    c = np.empty((R, half, 2), dtype=np.int64)
    c[..., 0], c[..., 1] = codes & 15, codes >> 4
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127))
    return (v.reshape(R, -1, 32) * s[..., None]).reshape(R, 2 * half)


def product_bound(x: np.ndarray, w: np.ndarray, y: np.ndarray, dtype) -> np.ndarray:
    """K fp32 additions, each off by at most a step (2^-23, which also allows
    truncation) of a partial sum that is at most sum |x w|; the products are
    exact; one rounding to the output type, by half a step."""
    K = x.shape[1]
    B = K * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    return B + EPS[dtype] * (np.abs(y) + B) + TINY[dtype]


def assert_close(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, what=""):
    g = f64(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    bad = ~(np.abs(g - want) <= bound)
    if bad.any():
        at = np.argwhere(bad)[:6].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first {at}: "
                             f"got {g[bad][:6]}, want {want[bad][:6]}, bound {bound[bad][:6]}")


# --- ternary experts ------------------------------------------------------------

def pack_ternary(t: np.ndarray) -> np.ndarray:
    c = np.where(t == 1, 1, np.where(t == -1, 2, 0)).astype(np.uint8)
    return c[..., 0::4] | (c[..., 1::4] << 2) | (c[..., 2::4] << 4) | (c[..., 3::4] << 6)


def dense(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 t * s of packed [..., K/4], scales [..., K/128]."""
    c = np.stack([(packed >> (2 * i)) & 3 for i in range(4)], -1)
    t = (c == 1).astype(np.float64) - (c == 2)
    t = t.reshape(packed.shape[:-1] + (packed.shape[-1] * 4,))
    return t * np.repeat(scales.astype(np.float64), 128, axis=-1)


def route(logits: np.ndarray, k: int, renorm: bool):
    """(chosen [T,E], weights [T,E]) by rank, in 64 bits."""
    T, E = logits.shape
    key = np.where(np.isnan(logits), np.inf, logits)
    nan = np.isnan(logits)
    chosen = np.zeros((T, E), dtype=bool)
    for t in range(T):
        # NaN first, then by value; equal ones by index (a stable sort keeps it)
        order = sorted(range(E), key=lambda e: (not nan[t, e], -key[t, e], e))
        chosen[t, order[:k]] = True
    chosen &= ~(logits == -np.inf)
    w = np.zeros((T, E))
    with np.errstate(invalid="ignore"):
        for t in range(T):
            if not chosen[t].any():
                continue
            pool = chosen[t] if renorm else ~(logits[t] == -np.inf)
            m = np.max(logits[t][pool])
            p = np.exp(logits[t] - m)
            w[t] = np.where(chosen[t], p / p[pool].sum(), 0.0)
    return chosen, w


def moe(x, logits, gate_up, gus, down, ds, k, renorm, dtype):
    """(y, bound) in 64 bits.  The bound carries fp32 sums (a step per addition),
    the hidden values' two bf16 terms (2^-16), exp and the weights' division
    (a few steps each, 2^-19 in all), and the final rounding."""
    T, H = x.shape
    E, F = gate_up.shape[0], down.shape[2] * 4
    chosen, w = route(logits, k, renorm)
    y = np.zeros((T, H))
    B = np.zeros((T, H))
    A = np.zeros((T, H))
    u32 = 2.0 ** -23
    for e in range(E):
        rows = np.where(chosen[:, e])[0]
        if rows.size == 0:
            continue
        Wgu, Wd = dense(gate_up[e], gus[e]), dense(down[e], ds[e])
        gu = x[rows] @ Wgu.T
        dgu = H * u32 * (np.abs(x[rows]) @ np.abs(Wgu).T)
        g, u, dg, du = gu[:, :F], gu[:, F:], dgu[:, :F], dgu[:, F:]
        with np.errstate(over="ignore"):
            sig = 1.0 / (1.0 + np.exp(-g))
        h = g * sig * u
        # |silu'| <= 1.1
        dh = (1.1 * dg) * (np.abs(u) + du) + np.abs(g * sig) * du + (2.0 ** -20 + 2.0 ** -16) * np.abs(h)
        part = h @ Wd.T
        dpart = dh @ np.abs(Wd).T + F * u32 * ((np.abs(h) + dh) @ np.abs(Wd).T)
        wt = w[rows, e][:, None]
        y[rows] += wt * part
        B[rows] += wt * dpart + 2.0 ** -19 * wt * np.abs(part)
        A[rows] += wt * (np.abs(part) + dpart)
    B += k * u32 * A
    return y, B + EPS[dtype] * (np.abs(y) + B) + TINY[dtype]
