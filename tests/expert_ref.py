"""Plain 64-bit forms of the experts' weight gradients and of the AdamW step, on the CPU (numpy), with the bounds of
the fp32 evaluation.  Nothing here uses the package."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def e4m3(q):
    """float64 values of E4M3 codes (uint8 array)"""
    q = q.astype(np.int64)
    exp, man = (q >> 3) & 15, q & 7
    v = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp.astype(np.float64) - 10))
    v = np.where((q & 0x7F) == 0x7F, np.nan, v)
    return np.where(q & 0x80, -v, v)


def clamped(offsets, rows):
    """The offsets as the kernels take them."""
    off = np.clip(np.asarray(offsets, dtype=np.int64), 0, rows)
    return np.maximum.accumulate(off)


def first_chunks(off):
    """First chunk of every group in the padded layout, and one past the last."""
    return np.concatenate([[0], np.cumsum(-(-np.diff(off) // 128))])


def wgrad(qa, sa, qb, sb, off, start=None):
    """(dW, T) [G][N][K] from operands in the padded layout: T = the sum of the terms' magnitudes."""
    G = len(off) - 1
    first = first_chunks(off)
    dw = np.zeros((G, qa.shape[0], qb.shape[0]))
    t = np.zeros_like(dw)
    for g in range(G):
        for c in range(first[g], first[g + 1]):
            a = e4m3(qa[:, 128 * c: 128 * c + 128]) * sa[c][:, None].astype(np.float64)
            b = e4m3(qb[:, 128 * c: 128 * c + 128]) * sb[c][:, None].astype(np.float64)
            dw[g] += a @ b.T
            t[g] += np.abs(a) @ np.abs(b).T
    if start is not None:
        dw += start
        t += np.abs(start)
    return dw, t


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random_16(n, seed, place, step):
    """The two 16-bit numbers of every element of the tensor at `place` in the list."""
    m32 = 0xFFFFFFFF
    key = int(mix((int(mix((seed + 0x9E3779B9 * place) & m32)) + step) & m32))
    h = mix((np.arange(n, dtype=np.uint64) & np.uint64(m32)) ^ np.uint64(key))
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def round_random(y, r):
    """fp32 y >= 0 and 16-bit numbers: unit * floor(fl32(y / unit + (r + 1/2) / 2^16)), at most 448"""
    y = y.astype(np.float32)
    unit = (2.0 ** (np.maximum(np.frexp(y)[1] - 1, -6) - 3.0)).astype(np.float32)
    t = np.floor(y / unit + ((r + 0.5) / 65536.0).astype(np.float32))
    return np.minimum(t * unit, np.float32(448.0))


def moments_8bit(qm, sm, qv, sv, g, beta1, beta2, seed, place, step):
    """New (codes' magnitudes and signs of m, sm, codes' values of sqrt(v), sv), in fp32 operations as defined."""
    f = np.float32
    n = g.size
    m = e4m3(qm).astype(f) * np.repeat(sm, 128)[:n]
    r = e4m3(qv).astype(f) * np.repeat(sv, 128)[:n]
    g = g.astype(f)
    m = m * f(beta1) + g * f(1.0 - beta1)
    v = r * r * f(beta2) + g * g * f(1.0 - beta2)
    r = np.sqrt(v)
    low, high = random_16(n, seed, place, step)
    out = []
    for x, bits in ((m, low), (r, high)):
        t = np.zeros(-(-n // 128) * 128, f)
        t[:n] = np.abs(x)
        s = t.reshape(-1, 128).max(axis=1) * (f(1.0) / f(448.0))
        d = np.repeat(np.where(s > 0, s, f(1.0)), 128)[:n]
        c = np.where(np.repeat(s, 128)[:n] > 0, round_random(np.abs(x) / d, bits), f(0.0))
        out += [c, s]
    out[2] = np.where(r > 0, np.maximum(out[2], f(2.0 ** -9)), out[2])
    out[0] = np.copysign(out[0], m)
    return out


def adamw(p, g, m, v, lr, beta1, beta2, eps, decay, step, scale=1.0):
    """New (p, m, v), and bounds of the fp32 evaluation's distance from them.  All arrays float64.
    v is a sum of positive terms: rest2, two products and the fused sum round, and beta2: 5 U relative, 6 with the
    gradient's factor twice in x^2 (7 in all).  m: the same count on the magnitudes of its two terms (4).  The
    denominator: half of v's, the square root (2), its factor and the fused sum (3), eps: 9 U in all; the quotient by
    a hardware reciprocal (2) and a product (1), the rate (1): 14 U of the update beside m's own, taken as 16."""
    x = g * scale
    m1 = beta1 * m + (1 - beta1) * x
    mag = beta1 * np.abs(m) + (1 - beta1) * np.abs(x)
    v1 = beta2 * v + (1 - beta2) * x * x
    d = np.sqrt(v1 / (1 - beta2 ** step)) + eps
    rate = lr / (1 - beta1 ** step)
    p1 = p * (1 - lr * decay) - rate * m1 / d
    em = 4 * U * mag + 1e-44
    ev = 7 * U * v1 + 3e-45
    ep = 3 * U * (np.abs(p) + np.abs(p1)) + rate / d * (em + 16 * U * mag)
    return p1, m1, v1, ep, em, ev
