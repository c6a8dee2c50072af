"""SwiGLU at the ends of the number range against 64-bit references: tiles whose
gates are all closed (down to the lowest finite value), infinite gates, NaN and
infinities beside tiles of zeros, and the agreement of the two passes."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
MODES = [0, 1]  # fp32 and power-of-two scales
CLOSED = [-60.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -92.0, -100.0, -104.0, -200.0, -1e4, -1e30, -1e38]
U = R.U


def _silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def _room(h, g, u):
    """The fp32 bound of ffn_ref.swiglu, and an absolute one that does not grow with the gate: a result or a factor
    below the smallest normal number 2^-126 may be off by that much, times u."""
    return np.abs(h) * (8 + 2 * np.minimum(np.abs(g), 200.0)) * U + 2.0 ** -125 * (1 + np.abs(u))


def _closed(dtype, lowest=True):
    gates = CLOSED + [-3.3e38, float(torch.finfo(dtype).min)] if lowest else CLOSED
    rng = np.random.default_rng(1)
    u = rng.standard_normal((len(gates), 256))
    u[:, 128:] *= 1e6
    return R.place(np.repeat(np.array(gates)[:, None], 256, axis=1), dtype), R.place(u, dtype)


@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_closed_gates_forward(fp8q, dtype, mode):
    """Every gate of a tile far below zero: h goes to zero with exp(g), it does not grow with g."""
    say(f"swiglu closed gates {dtype} mode {mode}")
    g, u = _closed(dtype)
    qh, sh, _ = fp8q.swiglu_quantize(g, u, scale_mode=mode)
    g64, u64 = R.f64(g), R.f64(u)
    h = _silu(g64) * u64
    R.assert_codes_of(qh, sh, h, _room(h, g64, u64), mode == 1, "h")
    q2, s2, _ = fp8q.swiglu_quantize(g, u, checkpoint=False, scale_mode=mode)
    assert torch.equal(q2, qh) and torch.equal(s2, sh)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_infinite_gates_forward(fp8q, dtype):
    """g = +inf gives h = inf * u, which its tile's scale shows; every other tile keeps its bits."""
    say(f"swiglu infinite gates {dtype}")
    rng = np.random.default_rng(2)
    g, u = R.place(rng.standard_normal((9, 384)), dtype), R.place(rng.uniform(0.5, 2.0, (9, 384)), dtype)
    clean = fp8q.swiglu_quantize(g, u)
    g[4, 200] = float("inf")
    for checkpoint in (True, False):
        qh, sh, _ = fp8q.swiglu_quantize(g, u, checkpoint=checkpoint)
        assert float(sh[1, 4]) == float("inf")
        others = torch.ones((3, 9), dtype=torch.bool, device="cuda")
        others[1, 4] = False
        assert torch.equal(sh[others], clean[1][others])
        tiles = others.t().repeat_interleave(128, dim=1)
        assert torch.equal(qh[tiles], clean[0][tiles])


def _backward_bounds(g, u, dh):
    """dg, du, h in 64 bits and bounds: those of ffn_ref with an absolute part that does not grow with the gate beyond
    the factors g, u and dh that the formula itself multiplies by."""
    s = R._sigmoid(g)
    h, du, dg = g * s * u, dh * g * s, dh * u * s * (1 + g * (1 - s))
    es = (6 + 2 * np.minimum(np.abs(g), 200.0)) * U
    tiny = 2.0 ** -124
    e_du = np.abs(du) * (es + 2 * U) + tiny * (1 + np.abs(dh))
    e_dg = np.abs(dh * u) * s * ((1 + np.abs(g) * (1 - s)) * (es + 6 * U) + np.abs(g) * (s * es + 2 * U)) + tiny * (
        1 + np.abs(dh)) * (1 + np.abs(u))
    return (dg, e_dg), (du, e_du), (h, np.abs(h) * (es + 2 * U) + tiny * (1 + np.abs(u)))


@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_closed_gates_backward(fp8q, dtype, mode):
    """The backward pass at closed gates, with gradients large enough that dg and du are normal numbers where the sigmoid
    is barely one; the recomputed h is the forward pass's at the checkpoint's values."""
    say(f"swiglu closed gates backward {dtype} mode {mode}")
    g, u = _closed(dtype, lowest=False)
    kept = fp8q.swiglu_quantize(g, u, scale_mode=mode)[2]
    dh = R.place(np.random.default_rng(3).standard_normal(tuple(g.shape)) * 1e6, dtype)
    g64, u64 = R.checkpoint_values(kept.qg, kept.sg), R.checkpoint_values(kept.qu, kept.su)
    assert np.isfinite(g64).all()
    want_dg, want_du, want_h = _backward_bounds(g64, u64, R.f64(dh))
    dg, du = fp8q.swiglu_backward(kept, dh)
    R.assert_close(dg, *want_dg, "dg")
    R.assert_close(du, *want_du, "du")
    o = fp8q.swiglu_backward_quantize(kept, dh, scale_mode=mode)
    R.assert_codes_of(o.qdg, o.sdg, *want_dg, mode == 1, "dg codes")
    R.assert_codes_of(o.qdu, o.sdu, *want_du, mode == 1, "du codes")
    R.assert_codes_of(o.qht, o.sht, *(np.ascontiguousarray(a.T) for a in want_h), mode == 1, "h transposed")


def _shown(q, s):
    """[rows][cols] of truth values: where codes times scale are no finite numbers (1x128 tiles of q[rows][cols])."""
    v = q.contiguous().view(torch.float8_e4m3fn).float() * s.t().repeat_interleave(128, dim=1)[:, : q.shape[1]]
    return ~torch.isfinite(v)


@pytest.mark.parametrize("value", [float("nan"), -float("nan"), float("inf")], ids=["nan", "-nan", "inf"])
@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_nonfinite_shows_forward(fp8q, dtype, mode, value):
    """One NaN or infinity in u beside tiles of zeros (a padded token): its tile's codes and scale show it, with a
    checkpoint and without; every other tile keeps its bits."""
    say(f"swiglu non-finite forward {dtype} mode {mode} {value}")
    rng = np.random.default_rng(4)
    g, u = R.place(rng.standard_normal((12, 512)), dtype), R.place(rng.standard_normal((12, 512)), dtype)
    g[5], u[5] = 0, 0
    g[:, 128:256], u[:, 128:256] = 0, 0
    clean = fp8q.swiglu_quantize(g, u, scale_mode=mode)
    u[4, 300] = value
    others = torch.ones((4, 12), dtype=torch.bool, device="cuda")
    others[2, 4] = False
    tiles = others.t().repeat_interleave(128, dim=1)
    for checkpoint in (True, False):
        qh, sh, kept = fp8q.swiglu_quantize(g, u, checkpoint=checkpoint, scale_mode=mode)
        shown = _shown(qh, sh)
        assert bool(shown[4, 300]) and not bool(shown[tiles].any())
        assert torch.equal(sh[others], clean[1][others]) and torch.equal(qh[tiles], clean[0][tiles])
        if mode == 0:
            assert not bool(torch.isfinite(sh[2, 4]))
        if kept is not None:
            assert bool(_shown(kept.qu, kept.su)[4, 300])
            assert torch.equal(kept.su[others], clean[2].su[others]) and torch.equal(kept.qg, clean[2].qg)


@pytest.mark.parametrize("value", [float("nan"), -float("nan"), float("inf")], ids=["nan", "-nan", "inf"])
@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_nonfinite_shows_backward(fp8q, dtype, mode, value):
    """One NaN or infinity in the incoming gradient beside zero gradients: every operand's tile that holds it shows it,
    in both orientations; the recomputed h and every other tile keep their bits."""
    say(f"swiglu non-finite backward {dtype} mode {mode} {value}")
    rng = np.random.default_rng(5)
    g, u = R.place(rng.standard_normal((140, 384)), dtype), R.place(rng.standard_normal((140, 384)), dtype)
    dh = R.place(rng.standard_normal((140, 384)), dtype)
    dh[8:12] = 0
    dh[:, 40] = 0
    kept = fp8q.swiglu_quantize(g, u)[2]
    clean = fp8q.swiglu_backward_quantize(kept, dh, scale_mode=mode)
    dh[9, 200] = value
    plain = fp8q.swiglu_backward(kept, dh)
    o = fp8q.swiglu_backward_quantize(kept, dh, scale_mode=mode)
    assert torch.equal(o.qht, clean.qht) and torch.equal(o.sht, clean.sht)
    for p, q, s, qt, st, cq, cs, cqt, cst in (
            (plain[0], o.qdg, o.sdg, o.qdgt, o.sdgt, clean.qdg, clean.sdg, clean.qdgt, clean.sdgt),
            (plain[1], o.qdu, o.sdu, o.qdut, o.sdut, clean.qdu, clean.sdu, clean.qdut, clean.sdut)):
        assert not bool(torch.isfinite(p[9, 200])) and int((~torch.isfinite(p)).sum()) == 1
        for a, b, ca, cb, at in ((q, s, cq, cs, (9, 200)), (qt, st, cqt, cst, (200, 9))):
            others = torch.ones(b.shape, dtype=torch.bool, device="cuda")
            others[at[1] // 128, at[0]] = False
            tiles = others.t().repeat_interleave(128, dim=1)[:, : a.shape[1]]
            shown = _shown(a, b)
            assert bool(shown[at]) and not bool(shown[tiles].any())
            assert torch.equal(b[others], cb[others]) and torch.equal(a[tiles], ca[tiles])
