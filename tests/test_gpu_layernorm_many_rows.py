"""Norms of so many rows that every team of lanes works through several of them
(rows loaded ahead, sums that take turns, weights' gradients added over a
team's rows), in every layout of a row, with whole and with partial groups of
eight columns, against 64-bit references."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import assert_codes_equal, assert_scales_equal, host_u8, say

pytestmark = pytest.mark.gpu
EPS = 1e-5
DTYPES = [torch.bfloat16, torch.float32]
KINDS = ["layer", "rms"]
# 256 compute units: teams of 16 lanes, of a wave (one, two and four groups a lane), of two and of four waves
FORWARD = [(33000, 24), (8300, 136), (6200, 520), (6200, 1000), (2051, 1000), (4500, 1304), (4500, 1999), (2100, 2504),
           (4099, 4090), (2051, 4104), (2051, 4999)]
WIDE = [(2600, 7168), (2600, 7001)]
# more rows than 256 work-groups of 1024 lanes hold at once
BACKWARD = [(16500, 40), (33000, 100), (4200, 300), (2100, 1001), (1100, 1032), (600, 2104), (1100, 3001), (300, 4104),
            (777, 7168), (600, 7001), (300, 8200), (600, 16384)]


def _kind(fp8q, kind):
    return fp8q.FP8Q_NORM_LAYER if kind == "layer" else fp8q.FP8Q_NORM_RMS


def _inputs(rows, cols, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * rng.choice([0.1, 1.0, 30.0], (rows, 1)) + rng.standard_normal((rows, 1)) * 2
    gamma = torch.from_numpy(rng.standard_normal(cols) * 0.2 + 1).float().cuda()
    beta = torch.from_numpy(rng.standard_normal(cols) * 0.2).float().cuda()
    return R.place(x, dtype, 1), gamma, beta, rng


def _forward(fp8q, oracle, rows, cols, dtype, kind, pow2):
    say(f"layernorm forward {rows}x{cols} {dtype} {kind}")
    x, gamma, beta, _ = _inputs(rows, cols, dtype, rows + cols)
    k = _kind(fp8q, kind)
    o = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=k, out_dtype=torch.float32)
    y, mean, rstd, e_y, e_m, e_r = R.layernorm(R.f64(x), R.f64(gamma), R.f64(beta), EPS, kind == "layer")
    R.assert_close(o.y, y, e_y, "y")
    R.assert_close(o.rstd, rstd, e_r, "rstd")
    if kind == "layer":
        R.assert_close(o.mean, mean, e_m, "mean")
    q, s = oracle.quantize_act_1x128(o.y.cpu().numpy())
    assert_codes_equal(host_u8(o.q), q, "codes")
    assert_scales_equal(o.s.cpu().numpy(), s.T, "scales")
    values = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=k, quantize=False, out_dtype=dtype)
    assert torch.equal(values.y, o.y.to(dtype)) and torch.equal(values.rstd, o.rstd)
    alone = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=k)
    assert torch.equal(alone.q, o.q) and torch.equal(alone.s, o.s)
    if pow2:
        p = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=k, scale_mode=fp8q.FP8Q_SCALE_POW2)
        qp, sp = fp8q.quantize_act(R.place(o.y.cpu().numpy(), torch.float32), scale_mode=fp8q.FP8Q_SCALE_POW2)
        assert torch.equal(p.q, qp) and torch.equal(p.s, sp)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", FORWARD)
def test_forward(fp8q, oracle, rows, cols, dtype, kind):
    _forward(fp8q, oracle, rows, cols, dtype, kind, True)


@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, "rms"), (torch.float32, "layer")], ids=["bf16-rms", "f32-layer"])
@pytest.mark.parametrize("rows,cols", WIDE)
def test_forward_wide(fp8q, oracle, rows, cols, dtype, kind):
    _forward(fp8q, oracle, rows, cols, dtype, kind, False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", BACKWARD)
def test_backward(fp8q, rows, cols, dtype, kind):
    say(f"layernorm backward {rows}x{cols} {dtype} {kind}")
    x, gamma, _, rng = _inputs(rows, cols, dtype, 3 * rows + cols)
    layer, k = kind == "layer", _kind(fp8q, kind)
    dy = R.place(rng.standard_normal((rows, cols)) * 0.01, dtype)
    skip = R.place(rng.standard_normal((rows, cols)) * 0.01, dtype, 2)
    f = fp8q.layernorm(x, gamma, eps=EPS, kind=k)
    dx, dgamma, dbeta = fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd, skip=skip, kind=k)
    w = R.layernorm_backward(R.f64(dy), R.f64(x), R.f64(gamma), R.f64(f.mean) if layer else None, R.f64(f.rstd),
                             R.f64(skip), layer)
    # a team adds rows / (256 * teams) rows one after the other: no more than rows / 256 of the roundings that
    # ffn_ref counts as rows / 512
    more = rows / 512 * R.U
    R.assert_close(dx, w[0], w[3], "dx")
    R.assert_close(dgamma, w[1], w[4] + more * np.abs(w[4]) / ((rows / 512 + 144) * R.U), "dgamma")
    if layer:
        R.assert_close(dbeta, w[2], w[5] + more * np.abs(w[5]) / ((rows / 512 + 144) * R.U), "dbeta")
    # dx over dy, and no skip, through the C entry
    need = fp8q.fp8q_layernorm_backward_workspace(rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    code, st = (1 if dtype == torch.bfloat16 else 0), torch.cuda.current_stream().cuda_stream
    for add in (skip, None):
        want = (dx, dgamma, dbeta) if add is not None else fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd, kind=k)
        over = R.place(R.f64(dy), dtype)
        dg = torch.empty(cols, device="cuda")
        assert fp8q.fp8q_layernorm_backward(
            over.data_ptr(), over.stride(0), x.data_ptr(), x.stride(0), code, rows, cols, gamma.data_ptr(), 0,
            f.mean.data_ptr() if layer else None, f.rstd.data_ptr(), k, None if add is None else add.data_ptr(),
            0 if add is None else add.stride(0), over.data_ptr(), over.stride(0), dg.data_ptr(), None, 0, ws.data_ptr(),
            need, st) == 0
        assert torch.equal(over, want[0]) and torch.equal(dg, want[1])
