"""What the feed-forward operators write: every element of their outputs, and
nothing around them (before and behind the array, between a row's end and the
next row), at odd sizes and strides, through the C entry points; a workspace of
exactly the bytes asked for."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
GUARD = 4096


class Out:
    """[rows][cols] of `dtype` with row stride ld inside a buffer of 0xa5."""

    def __init__(self, rows, cols, dtype, ld):
        size = dtype.itemsize
        self.shape, self.size = (rows, cols, ld), size
        self.raw = torch.full((2 * GUARD + rows * ld * size,), 0xa5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:].view(dtype)[: rows * ld].view(rows, ld)[:, :cols] if rows * ld else None
        self.ptr, self.ld = self.raw.data_ptr() + GUARD, ld

    def check(self, what):
        rows, cols, ld = self.shape
        b = self.raw.cpu().numpy()
        assert (b[:GUARD] == 0xa5).all() and (b[len(b) - GUARD:] == 0xa5).all(), f"{what}: written outside"
        body = b[GUARD:len(b) - GUARD].reshape(rows, ld, self.size)
        assert (body[:, cols:] == 0xa5).all(), f"{what}: written between the rows"
        if self.size > 1:  # a code may be 0xa5
            assert not (body[:, :cols] == 0xa5).all(axis=2).any(), f"{what}: left unwritten"


def _ld(n, per, extra):
    return (-(-n // per) + extra) * per


def _stream():
    return torch.cuda.current_stream().cuda_stream


SIZES = [(1, 1), (3, 127), (5, 136), (17, 513), (130, 1001), (257, 2049), (9, 4100), (3, 8201), (1030, 700), (2051, 1500)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norms(fp8q, rows, cols, dtype):
    say(f"bounds norm {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    code, per = (1 if dtype == torch.bfloat16 else 0), 16 // dtype.itemsize
    x, dy = (R.place(rng.standard_normal((rows, cols)) + 0.1, dtype, 1) for _ in range(2))
    groups = -(-cols // 128)
    for eps in (1e-5, 0.0):
        y, q, s = (Out(rows, cols, dtype, _ld(cols, per, 2)), Out(rows, cols, torch.uint8, _ld(cols, 16, 1)),
                   Out(groups, rows, torch.float32, rows + 3))
        mean, rstd = Out(1, rows, torch.float32, rows), Out(1, rows, torch.float32, rows)
        assert fp8q.fp8q_layernorm(x.data_ptr(), code, rows, cols, x.stride(0), None, None, 0, eps, 0, y.ptr, code, y.ld,
                                   q.ptr, q.ld, s.ptr, s.ld, 0, mean.ptr, rstd.ptr, _stream()) == 0
        for what, o in (("q", q), ("s", s), ("mean", mean), ("rstd", rstd), ("y", y)):
            o.check(what)
    need = fp8q.fp8q_layernorm_backward_workspace(rows, cols)
    ws, dx = Out(1, need, torch.uint8, need), Out(rows, cols, dtype, _ld(cols, per, 1))
    dgamma, dbeta = Out(1, cols, torch.float32, cols), Out(1, cols, torch.float32, cols)
    assert fp8q.fp8q_layernorm_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), code, rows, cols, None, 0,
                                        mean.ptr, rstd.ptr, 0, None, 0, dx.ptr, dx.ld, dgamma.ptr, dbeta.ptr, 0, ws.ptr,
                                        need, _stream()) == 0
    for what, o in (("dx", dx), ("dgamma", dgamma), ("dbeta", dbeta)):
        o.check(what)
    b = ws.raw.cpu().numpy()
    assert (b[:GUARD] == 0xa5).all() and (b[GUARD + need:] == 0xa5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (129, 136), (17, 513), (130, 1001), (257, 384), (1030, 140)])
def test_swiglu(fp8q, rows, cols, dtype):
    say(f"bounds swiglu {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    code, per = (1 if dtype == torch.bfloat16 else 0), 16 // dtype.itemsize
    g, u, dh = (R.place(rng.standard_normal((rows, cols)) + 0.1, dtype, 1) for _ in range(3))
    groups, tgroups = -(-cols // 128), -(-rows // 128)

    def codes(n, m, extra):
        return Out(n, m, torch.uint8, _ld(m, 16, extra))

    def scales(n, m, extra):
        return Out(n, m, torch.float32, m + extra)

    qh, sh, qg, qu, sg, su = (codes(rows, cols, 1), scales(groups, rows, 1), codes(rows, cols, 2), codes(rows, cols, 2),
                              scales(groups, rows, 5), scales(groups, rows, 5))
    assert fp8q.fp8q_swiglu_quantize(g.data_ptr(), u.data_ptr(), code, g.stride(0), rows, cols, qh.ptr, qh.ld, sh.ptr,
                                     sh.ld, qg.ptr, qu.ptr, qg.ld, sg.ptr, su.ptr, sg.ld, 0, _stream()) == 0
    for what, o in (("qh", qh), ("sh", sh), ("qg", qg), ("qu", qu), ("sg", sg), ("su", su)):
        o.check(what)
    kept = (qg.ptr, qu.ptr, qg.ld, sg.ptr, su.ptr, sg.ld, dh.data_ptr(), code, dh.stride(0), rows, cols)
    dg, du = (Out(rows, cols, dtype, _ld(cols, per, 1)) for _ in range(2))
    assert fp8q.fp8q_swiglu_backward(*kept, dg.ptr, du.ptr, dg.ld, _stream()) == 0
    dg.check("dg")
    du.check("du")
    o = dict(qdg=codes(rows, cols, 1), qdu=codes(rows, cols, 1), sdg=scales(groups, rows, 2), sdu=scales(groups, rows, 2),
             qdgt=codes(cols, rows, 1), qdut=codes(cols, rows, 1), sdgt=scales(tgroups, cols, 3),
             sdut=scales(tgroups, cols, 3), qht=codes(cols, rows, 2), sht=scales(tgroups, cols, 1))
    p = {n: v.ptr for n, v in o.items()}
    assert fp8q.fp8q_swiglu_backward_quantize(
        *kept, p["qdg"], p["qdu"], o["qdg"].ld, p["sdg"], p["sdu"], o["sdg"].ld, p["qdgt"], p["qdut"], o["qdgt"].ld,
        p["sdgt"], p["sdut"], o["sdgt"].ld, p["qht"], o["qht"].ld, p["sht"], o["sht"].ld, 0, _stream()) == 0
    for n, v in o.items():
        v.check(n)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,E,top_k,H,I", [(1, 1, 1, 128, 128), (3, 5, 7, 256, 384), (5, 64, 8, 384, 128),
                                           (17, 12, 4, 256, 128), (40, 6, 6, 128, 256), (64, 70, 2, 256, 128)])
def test_moe(fp8q, T, E, top_k, H, I, out):
    say(f"bounds moe T={T} E={E} k={top_k} H={H} I={I} {out}")
    from tests.test_gpu_moe import _layer
    x, logits, w_gu, s_gu, w_down, s_down = _layer(T + E, T, E, H, I, pad=1)
    l = torch.from_numpy(logits).cuda()
    need = fp8q.fp8q_moe_decode_workspace(T, H, I, E, top_k)
    ws, y = Out(1, need, torch.uint8, need), Out(T, H, out, H + 16)
    assert fp8q.fp8q_moe_decode(
        x.data_ptr(), x.stride(0), T, H, l.data_ptr(), E, E, top_k, 1, I, w_gu.data_ptr(), w_gu.stride(1), w_gu.stride(0),
        s_gu.data_ptr(), s_gu.stride(1), s_gu.stride(0), w_down.data_ptr(), w_down.stride(1), w_down.stride(0),
        s_down.data_ptr(), s_down.stride(1), s_down.stride(0), y.ptr, 1 if out == torch.bfloat16 else 0, y.ld, ws.ptr, need,
        _stream()) == 0
    y.check("y")
    b = ws.raw.cpu().numpy()
    assert (b[:GUARD] == 0xa5).all() and (b[GUARD + need:] == 0xa5).all()
    assert torch.equal(y.t, fp8q.moe_decode(x, l, w_gu, s_gu, w_down, s_down, top_k, out_dtype=out))
