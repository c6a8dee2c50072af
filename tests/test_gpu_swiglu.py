"""SwiGLU with 8-bit checkpoints, forward and backward, against 64-bit
references: one row to many, one column to wide, odd sizes, padded strides
with NaN beyond each row, gates from -200 to 200, zero tiles.  The checkpoint
equals the activation quantizer's codes, and the fused backward's codes equal
the quantizers' on the plain backward's fp32 gradients, bit for bit."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (1, 2048), (3, 16), (4, 127), (128, 128), (129, 128), (7, 129), (64, 512), (200, 520), (33, 1000),
         (257, 384), (2, 7168), (1000, 24)]
DTYPES = [torch.bfloat16, torch.float32]
MODES = [0, 1]  # fp32 and power-of-two scales


def _gates(rng, rows, cols):
    g = rng.standard_normal((rows, cols)) * rng.choice([0.5, 2.0, 8.0], (rows, 1))
    g.flat[rng.integers(0, g.size, max(1, g.size // 50))] = rng.choice([-200.0, -90.0, -20.0, 0.0, 20.0, 200.0])
    return g


def _halves(rng, rows, cols, dtype):
    """g and u: two halves of a fused product where its halves can be aligned, else two padded tensors"""
    g, u = _gates(rng, rows, cols), rng.standard_normal((rows, cols))
    if cols % 8 == 0:
        both = R.place(np.concatenate([g, u], axis=1), dtype, 1)
        return both[:, :cols], both[:, cols:]
    return R.place(g, dtype, 1), R.place(u, dtype, 1)


@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(fp8q, rows, cols, dtype, mode):
    say(f"swiglu forward {rows}x{cols} {dtype} mode {mode}")
    g, u = _halves(np.random.default_rng(rows + cols), rows, cols, dtype)
    qh, sh, kept = fp8q.swiglu_quantize(g, u, scale_mode=mode)
    h, e = R.swiglu(R.f64(g), R.f64(u))
    R.assert_codes_of(qh, sh, h, e, mode == 1, "h")
    for q, s, v in ((kept.qg, kept.sg, g), (kept.qu, kept.su, u)):
        wq, ws = fp8q.quantize_act(R.place(v.float().cpu().numpy(), dtype), scale_mode=mode)
        assert torch.equal(q, wq) and torch.equal(s, ws)
    q2, s2, none = fp8q.swiglu_quantize(g, u, checkpoint=False, scale_mode=mode)
    assert none is None and torch.equal(q2, qh) and torch.equal(s2, sh)


def _kept(fp8q, rows, cols, dtype, seed, mode=0):
    rng = np.random.default_rng(seed)
    g, u = _halves(rng, rows, cols, dtype)
    kept = fp8q.swiglu_quantize(g, u, scale_mode=mode)[2]
    dh = R.place(rng.standard_normal((rows, cols)) * 1e-3, dtype, 1)
    return kept, dh


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(fp8q, rows, cols, dtype):
    say(f"swiglu backward {rows}x{cols} {dtype}")
    kept, dh = _kept(fp8q, rows, cols, dtype, 5 * rows + cols)
    dg, du = fp8q.swiglu_backward(kept, dh)
    g, u = R.checkpoint_values(kept.qg, kept.sg), R.checkpoint_values(kept.qu, kept.su)
    wg, wu, eg, eu = R.swiglu_backward(g, u, R.f64(dh))
    R.assert_close(dg, wg, eg, "dg")
    R.assert_close(du, wu, eu, "du")


@pytest.mark.parametrize("mode", MODES, ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward_quantize(fp8q, rows, cols, dtype, mode):
    say(f"swiglu backward quantize {rows}x{cols} {dtype} mode {mode}")
    kept, dh = _kept(fp8q, rows, cols, dtype, rows + 9 * cols)
    o = fp8q.swiglu_backward_quantize(kept, dh, scale_mode=mode)
    plain = fp8q.swiglu_backward(kept, R.place(dh.float().cpu().numpy(), torch.float32))
    for d, q, s, qt, st in zip(plain, (o.qdg, o.qdu), (o.sdg, o.sdu), (o.qdgt, o.qdut), (o.sdgt, o.sdut)):
        d = R.place(d.cpu().numpy(), torch.float32)
        wq, ws = fp8q.quantize_act(d, scale_mode=mode)
        assert torch.equal(q, wq) and torch.equal(s, ws), "1x128"
        wq, ws = fp8q.quantize_act(d, fp8q.FP8Q_TILE_128x1, scale_mode=mode)
        assert torch.equal(qt, wq) and torch.equal(st, ws), "128x1"
    h, e = R.swiglu(R.checkpoint_values(kept.qg, kept.sg), R.checkpoint_values(kept.qu, kept.su))
    R.assert_codes_of(o.qht, o.sht, np.ascontiguousarray(h.T), np.ascontiguousarray(e.T), mode == 1, "h transposed")
    if cols % 128 == 0:
        q, s, qt, st = o.gate_up()
        assert torch.equal(q, torch.cat([o.qdg, o.qdu], 1)) and torch.equal(s, torch.cat([o.sdg, o.sdu]))
        assert torch.equal(qt, torch.cat([o.qdgt, o.qdut])) and torch.equal(st, torch.cat([o.sdgt, o.sdut], 1))
    else:
        with pytest.raises(ValueError, match="multiple of 128"):
            o.gate_up()


def test_backward_against_differences(fp8q):
    """dg and du against central differences of h in 64 bits at the checkpoint's values."""
    say("swiglu differences")
    kept, _ = _kept(fp8q, 40, 200, torch.float32, 2)
    one = torch.ones((40, 200), device="cuda")
    dg, du = fp8q.swiglu_backward(kept, one)
    g, u = R.checkpoint_values(kept.qg, kept.sg), R.checkpoint_values(kept.qu, kept.su)
    step = 1e-5
    for d, f in ((dg, lambda t: R.swiglu(g + t, u)[0]), (du, lambda t: R.swiglu(g, u + t)[0])):
        want = (f(step) - f(-step)) / (2 * step)
        # h^2 f'''/6 <= 1e-10 |u|, rounding 1e-16 |h| / step; fp32 (16 + 2|g|) U of each product's size
        room = 1e-9 * (1 + np.abs(g)) * (1 + np.abs(u)) + (16 + 2 * np.abs(g)) * R.U * (1 + np.abs(g)) * (1 + np.abs(u))
        assert (np.abs(R.f64(d) - want) <= room).all()


def test_zero_tiles_and_empty(fp8q):
    say("swiglu zero tiles, no rows")
    g = torch.zeros((130, 256), dtype=torch.bfloat16, device="cuda")
    u = torch.randn((130, 256), device="cuda").to(torch.bfloat16)
    qh, sh, kept = fp8q.swiglu_quantize(g, u)
    assert not sh.any() and not (qh & 0x7f).any()
    o = fp8q.swiglu_backward_quantize(kept, u)
    assert not o.sdu.any() and not o.sht.any() and bool(o.sdg.all())
    q0, s0, k0 = fp8q.swiglu_quantize(g[:0], u[:0])
    assert q0.shape == (0, 256) and s0.shape == (2, 0)
    assert fp8q.swiglu_backward(k0, u[:0])[0].shape == (0, 256)
    assert fp8q.swiglu_backward_quantize(k0, u[:0]).qht.shape == (256, 0)


def test_rows_past_32_bit_offsets(fp8q):
    """A row stride that puts the last rows beyond 2^32 bytes."""
    say("swiglu: far rows")
    ld = 1 << 29
    buf = torch.zeros(9 * ld, dtype=torch.bfloat16, device="cuda")
    g, u = buf.as_strided((9, 256), (ld, 1)), buf[512:].as_strided((9, 256), (ld, 1))
    vg, vu = (torch.randn((9, 256), device="cuda").to(torch.bfloat16) for _ in range(2))
    g.copy_(vg)
    u.copy_(vu)
    a, b = fp8q.swiglu_quantize(g, u), fp8q.swiglu_quantize(vg, vu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(i, j) for i, j in zip(a[2], b[2]))
    far = buf[1024:].as_strided((9, 256), (ld, 1))
    far.copy_(vu)
    assert all(torch.equal(i, j) for i, j in zip(fp8q.swiglu_backward(a[2], far), fp8q.swiglu_backward(a[2], vu)))
    assert all(torch.equal(i, j) for i, j in zip(fp8q.swiglu_backward_quantize(a[2], far),
                                                 fp8q.swiglu_backward_quantize(a[2], vu)))
