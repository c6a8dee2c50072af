"""64-bit references of the feed-forward operators, and checks of codes
against a 64-bit value whose fp32 computation may be off by a known amount."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24  # unit roundoff of fp32


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").double().numpy()


def padded(rows: int, cols: int, dtype: torch.dtype, extra: int = 0, device="cuda") -> torch.Tensor:
    """[rows][cols] of NaN inside a wider buffer: row stride a multiple of 16 bytes, `extra` such units wider."""
    per = 16 // dtype.itemsize
    ld = (-(-max(cols, 1) // per) + extra) * per
    fill = 0x7f if dtype == torch.uint8 else float("nan")
    return torch.full((max(rows, 1), ld), fill, dtype=dtype, device=device)[:rows, :cols]


def place(a: np.ndarray, dtype: torch.dtype, extra: int = 0) -> torch.Tensor:
    t = padded(a.shape[0], a.shape[1], dtype, extra)
    t.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dtype))
    return t


def bf16_half_ulp(x: np.ndarray) -> np.ndarray:
    ax = np.maximum(np.abs(x), 2.0 ** -126)
    return np.exp2(np.floor(np.log2(ax)) - 8)


def assert_close(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, what: str):
    """|got - want| <= bound, and half a unit in the last place of a bf16 result on top."""
    if got.dtype == torch.bfloat16:
        bound = bound + bf16_half_ulp(np.abs(want) + bound)
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} out of bound; first at {tuple(np.argwhere(bad)[0])}: "
                           f"{g[bad][0]!r} wanted {want[bad][0]!r} +- {bound[bad][0]!r}")


def decode(q: torch.Tensor) -> np.ndarray:
    return f64(q.contiguous().view(torch.float8_e4m3fn).float())


def _half_step(v: np.ndarray) -> np.ndarray:
    """Half the distance between neighbouring E4M3 values at magnitude |v|."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -9)))
    return np.exp2(np.maximum(e, -6.0) - 4.0)


def assert_codes_of(q: torch.Tensor, s: torch.Tensor, v: np.ndarray, err: np.ndarray, pow2: bool, what: str):
    """1x128 codes q[rows][cols] and scales s[groups][rows] of values within `err` of v: the scale belongs to a tile
    maximum inside that interval, and each code is a nearest E4M3 value of something inside its own."""
    rows, cols = v.shape
    q64, s64 = decode(q), f64(s)
    assert q64.shape == v.shape and s64.shape == (-(-cols // 128), rows), (what, q64.shape, s64.shape)
    assert np.isfinite(q64).all() and np.isfinite(s64).all(), what
    for j in range(s64.shape[0]):
        a, e = np.abs(v[:, 128 * j:128 * j + 128]), err[:, 128 * j:128 * j + 128]
        lo, hi = np.maximum(a - e, 0).max(axis=1) / 448.0, (a + e).max(axis=1) / 448.0
        if pow2:
            hi = np.where(hi > 0, np.maximum(2.0 ** np.ceil(np.log2(np.maximum(hi, 1e-300))), 2.0 ** -127), 0.0)
        ok = (s64[j] >= lo * (1 - 2 * U) - 2.0 ** -149) & (s64[j] <= hi * (1 + 2 * U) + 2.0 ** -149)
        assert ok.all(), f"{what}: scale of tile {j}, row {np.argmin(ok)}: {s64[j][~ok][0]!r} in [{lo[~ok][0]!r}, {hi[~ok][0]!r}]"
    sc = np.repeat(s64.T, 128, axis=1)[:, :cols]
    room = np.where(sc > 0, err + sc * _half_step((np.abs(v) + err) / np.where(sc > 0, sc, 1)) * (1 + 8 * U), err)
    bad = np.abs(q64 * sc - v) > room + 4 * U * np.abs(v)
    assert not bad.any(), (f"{what}: {int(bad.sum())} codes off; first at {tuple(np.argwhere(bad)[0])}: "
                           f"{(q64 * sc)[bad][0]!r} for {v[bad][0]!r} (scale {sc[bad][0]!r})")


# ------------------------------------------------------------------ layer norm

def layernorm(x, gamma, beta, eps, layer):
    """y, mean, rstd in 64 bits, and bounds of the fp32 result.

    A sum of a row adds at most 32 values in a thread, 6 steps in a wave and 16 waves, one rounding each, plus the
    rounding of the terms: 64 U of the sum of magnitudes.  The variance is a sum of squares (64 U relative) with the
    mean's error entering squared, so rstd is good to 40 U; y then has the error of the mean and 48 U of its product."""
    mean = x.mean(axis=1, keepdims=True) if layer else np.zeros((x.shape[0], 1))
    d = x - mean
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    y = d * rstd * gamma + beta
    e_mean = 64 * U * np.abs(x).mean(axis=1, keepdims=True) if layer else 0 * mean
    # a mean that is off by e shifts every deviation by e and adds e^2 to the variance
    e_rstd = rstd * (40 * U + 0.5 * (e_mean * rstd) ** 2)
    e_y = (e_mean + U * np.abs(d)) * rstd * np.abs(gamma) + np.abs(d * gamma) * e_rstd + 8 * U * (
        np.abs(d * rstd * gamma) + np.abs(beta))
    return y, mean[:, 0], rstd[:, 0], e_y, e_mean[:, 0] + U * np.abs(mean[:, 0]), e_rstd[:, 0]


def layernorm_backward(dy, x, gamma, mean, rstd, skip, layer):
    """dx, dgamma, dbeta in 64 bits for the given statistics, and bounds of the fp32 result (see layernorm; the sums
    over rows add up to rows/512 + 128 + 8 partial results one after the other)."""
    rows, cols = x.shape
    m = mean[:, None] if layer else 0.0
    r = rstd[:, None]
    xh = (x - m) * r
    w = dy * gamma
    c2 = (w * xh).mean(axis=1, keepdims=True)
    c1 = w.mean(axis=1, keepdims=True) if layer else 0.0
    dx = r * (w - xh * c2 - c1) + skip
    a2, a1 = np.abs(w * xh).mean(axis=1, keepdims=True), np.abs(w).mean(axis=1, keepdims=True)
    # xh itself has two roundings
    e = 80 * U * r * (np.abs(w) + np.abs(xh) * a2 + (a1 if layer else 0.0)) + 2 * U * (np.abs(skip) + np.abs(dx))
    n = (rows / 512 + 144) * U
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0), e, n * np.abs(dy * xh).sum(axis=0), n * np.abs(dy).sum(axis=0)


# ------------------------------------------------------------------ SwiGLU

def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u):
    """h and its fp32 bound: exp(-g) is good to (4 + 2|g|) U of itself (its argument's rounding and its own), the
    quotient and the products add a rounding each."""
    s = _sigmoid(g)
    h = g * s * u
    return h, np.abs(h) * (8 + 2 * np.abs(g)) * U + _tiny(g, u, 1.0)


def _tiny(g, u, dh):
    # exp(-g) beyond the largest fp32 makes the sigmoid 0 where it is below 2^-126
    return 2.0 ** -124 * (1 + np.abs(g)) * (1 + np.abs(u)) * (np.abs(dh) + 2.0 ** -20)


def swiglu_backward(g, u, dh):
    """dg, du and their fp32 bounds."""
    s = _sigmoid(g)
    es = (6 + 2 * np.abs(g)) * U
    du, dg = dh * g * s, dh * u * s * (1 + g * (1 - s))
    e_du = np.abs(du) * (es + 2 * U)
    # 1 - s loses s's absolute error; the sum with 1 and the products round once each
    e_dg = np.abs(dh * u) * s * ((1 + np.abs(g) * (1 - s)) * (es + 6 * U) + np.abs(g) * (s * es + 2 * U))
    return dg, du, e_dg + _tiny(g, u, dh), e_du + _tiny(g, u, dh)


def checkpoint_values(q: torch.Tensor, s: torch.Tensor) -> np.ndarray:
    """fl32(dec(q) * s) as float64."""
    d = q.contiguous().view(torch.float8_e4m3fn).float().cpu()
    sc = s.cpu().t().repeat_interleave(128, dim=1)[:, : q.shape[1]]
    return (d * sc).double().numpy()


# ------------------------------------------------------------------ mixture of experts

def chosen(logits: np.ndarray, top_k: int, renormalize: bool):
    """For each token a list of (expert, probability), or None where a logit is NaN or +inf."""
    out = []
    for row in logits:
        if np.isnan(row).any() or np.isposinf(row).any():
            out.append(None)
            continue
        ids = [e for e in sorted(range(len(row)), key=lambda e: (-row[e], e))[:top_k] if row[e] > -np.inf]
        if not ids:
            out.append([])
            continue
        with np.errstate(under="ignore"):
            p = np.exp(row - row[ids[0]])
        total = p[ids].sum() if renormalize else p.sum()
        out.append([(e, p[e] / total) for e in ids])
    return out


def block_values(q: torch.Tensor, s: torch.Tensor) -> np.ndarray:
    return decode(q) * np.repeat(np.repeat(f64(s), 128, axis=0), 128, axis=1)


def moe(x, logits, w_gu, s_gu, w_down, s_down, top_k, renormalize):
    """y in 64 bits and the bound of the fp32 result: 1e-5 of the sum of magnitudes for each product (a chunk's 128
    products, up to 64 chunks and 4 waves are added in fp32), 2^-16 for h's two bf16 halves, and 16 + 2|g| roundings
    of the SwiGLU and the weight."""
    tokens, hidden = x.shape
    y, e = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    cache = {}
    for t, picks in enumerate(chosen(logits, top_k, renormalize)):
        if picks is None:
            y[t] = np.nan
            continue
        for ex, p in picks:
            if ex not in cache:
                cache[ex] = (block_values(w_gu[ex], s_gu[ex]), block_values(w_down[ex], s_down[ex]))
            wg, wd = cache[ex]
            a, ea = wg @ x[t], 1e-5 * (np.abs(wg) @ np.abs(x[t]))
            n = len(a) // 2
            g, u = a[:n], a[n:]
            s = _sigmoid(g)
            h = g * s * u
            # |d silu| <= 1.1
            eh = 1.1 * ea[:n] * (np.abs(u) + ea[n:]) + np.abs(g * s) * ea[n:] + np.abs(h) * (2.0 ** -16 + (16 + 2 * np.abs(g)) * U)
            y[t] += p * (wd @ h)
            e[t] += p * (np.abs(wd) @ (eh + 1e-5 * np.abs(h)))
    return y, e
