"""Layer norm and RMS norm, forward and backward, against 64-bit references:
widths from one column to the largest, odd ones, one row to many, padded row
strides with NaN beyond each row, rows of equal values, large offsets, tiny
and huge values; the codes equal the quantizer's on the same fp32 values bit
for bit."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import assert_codes_equal, assert_scales_equal, host_u8, say

pytestmark = pytest.mark.gpu
EPS = 1e-5
SIZES = [(1, 1), (1, 7168), (3, 8), (5, 127), (4, 128), (2, 129), (33, 512), (7, 513), (9, 1000), (17, 2048), (6, 2056),
         (3, 4097), (2, 7168), (5, 8192), (3, 8200), (2, 16384), (3000, 40), (1030, 264)]
DTYPES = [torch.bfloat16, torch.float32]
KINDS = ["layer", "rms"]


def _kind(fp8q, kind):
    return fp8q.FP8Q_NORM_LAYER if kind == "layer" else fp8q.FP8Q_NORM_RMS


def _inputs(rows, cols, dtype, seed, extra=1):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * rng.choice([0.1, 1.0, 30.0], (rows, 1)) + rng.standard_normal((rows, 1)) * 2
    return R.place(x, dtype, extra), rng


def _weights(rng, cols, dtype=torch.float32):
    g = torch.from_numpy(rng.standard_normal(cols) * 0.2 + 1).to(dtype).cuda()
    b = torch.from_numpy(rng.standard_normal(cols) * 0.2).to(dtype).cuda()
    return g, b


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(fp8q, oracle, rows, cols, dtype, kind):
    say(f"layernorm forward {rows}x{cols} {dtype} {kind}")
    x, rng = _inputs(rows, cols, dtype, rows + 7 * cols)
    wt = DTYPES[(rows + cols) % 2]
    gamma, beta = _weights(rng, cols, wt)
    o = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=_kind(fp8q, kind), out_dtype=torch.float32)
    y, mean, rstd, e_y, e_m, e_r = R.layernorm(R.f64(x), R.f64(gamma), R.f64(beta), EPS, kind == "layer")
    R.assert_close(o.y, y, e_y, "y")
    R.assert_close(o.rstd, rstd, e_r, "rstd")
    assert (o.mean is None) == (kind == "rms")
    if o.mean is not None:
        R.assert_close(o.mean, mean, e_m, "mean")
    q, s = oracle.quantize_act_1x128(o.y.cpu().numpy())
    assert_codes_equal(host_u8(o.q), q, "codes")
    assert_scales_equal(o.s.cpu().numpy(), s.T, "scales")
    # each output alone, and the rounded values
    b = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=_kind(fp8q, kind), quantize=False, out_dtype=torch.bfloat16)
    assert b.q is None and b.s is None and torch.equal(b.y, o.y.to(torch.bfloat16))
    p = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=_kind(fp8q, kind), scale_mode=fp8q.FP8Q_SCALE_POW2)
    qp, sp = fp8q.quantize_act(R.place(o.y.cpu().numpy(), torch.float32), scale_mode=fp8q.FP8Q_SCALE_POW2)
    assert p.y is None and torch.equal(p.q, qp) and torch.equal(p.s, sp)


def test_forward_without_weights_and_at_extremes(fp8q):
    """No gamma or beta; rows of one value (variance 0), around 2^60 (whose squares add up
    beyond the largest fp32), around 2^-60, of zeros, and with an offset of 1000."""
    say("layernorm extremes")
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 1024))
    x[0] = 3.25
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -60
    x[3] = 0
    x[4] += 1000.0
    xt = R.place(x, torch.float32)
    x = R.f64(xt)
    for layer, kind in ((True, fp8q.FP8Q_NORM_LAYER), (False, fp8q.FP8Q_NORM_RMS)):
        o = fp8q.layernorm(xt, eps=EPS, kind=kind, out_dtype=torch.float32)
        y, _, rstd, e_y, _, e_r = R.layernorm(x, np.ones(1024), np.zeros(1024), EPS, layer)
        R.assert_close(o.y, y, e_y, f"y layer={layer}")
        R.assert_close(o.rstd, rstd, e_r, "rstd")
    zero = fp8q.layernorm(xt, eps=EPS)
    assert not zero.q[0].any() and not zero.s[:, 0].any() and not zero.q[3].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(fp8q, rows, cols, dtype, kind):
    say(f"layernorm backward {rows}x{cols} {dtype} {kind}")
    x, rng = _inputs(rows, cols, dtype, 3 * rows + cols)
    dy = R.place(rng.standard_normal((rows, cols)) * 0.01, dtype, 2)
    skip = R.place(rng.standard_normal((rows, cols)) * 0.01, dtype, 0) if cols % 2 else None
    gamma, beta = _weights(rng, cols, DTYPES[rows % 2])
    k, layer = _kind(fp8q, kind), kind == "layer"
    f = fp8q.layernorm(x, gamma, beta, eps=EPS, kind=k)
    dx, dgamma, dbeta = fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd, skip=skip, kind=k)
    w = R.layernorm_backward(R.f64(dy), R.f64(x), R.f64(gamma), R.f64(f.mean) if layer else None, R.f64(f.rstd),
                             0.0 if skip is None else R.f64(skip), layer)
    R.assert_close(dx, w[0], w[3], "dx")
    R.assert_close(dgamma, w[1], w[4], "dgamma")
    assert (dbeta is None) == (not layer)
    if layer:
        R.assert_close(dbeta, w[2], w[5], "dbeta")
    # the same bits again, and added to what is there
    again = fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd, skip=skip, kind=k)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)
    start = torch.full((cols,), 0.5, device="cuda")
    acc = fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd, skip=skip, kind=k, dgamma=start.clone(),
                                  dbeta=start.clone() if layer else None, accumulate=True)
    assert torch.equal(acc[1], start + dgamma) and (not layer or torch.equal(acc[2], start + dbeta))


@pytest.mark.parametrize("kind", KINDS)
def test_backward_against_differences(fp8q, kind):
    """dx, dgamma, dbeta against central differences of the forward formula in 64 bits."""
    say(f"layernorm differences {kind}")
    rows, cols, layer = 3, 24, kind == "layer"
    rng = np.random.default_rng(8)
    x, g, b = rng.standard_normal((rows, cols)), rng.standard_normal(cols), rng.standard_normal(cols)
    c = rng.standard_normal((rows, cols))
    xt, ct = R.place(x, torch.float32), R.place(c, torch.float32)
    gt, bt = torch.from_numpy(g).float().cuda(), torch.from_numpy(b).float().cuda()
    x, c, g, b = R.f64(xt), R.f64(ct), R.f64(gt), R.f64(bt)
    k = _kind(fp8q, kind)
    f = fp8q.layernorm(xt, gt, bt, eps=EPS, kind=k)
    dx, dg, db = fp8q.layernorm_backward(ct, xt, gt, f.mean, f.rstd, kind=k)

    def loss(x, g, b):
        return (R.layernorm(x, g, b, EPS, layer)[0] * c).sum()

    def differences(a, at):
        d, h = np.zeros_like(a), 1e-5
        for i in np.ndindex(a.shape):
            up, down = a.copy(), a.copy()
            up[i] += h
            down[i] -= h
            d[i] = (at(up) - at(down)) / (2 * h)
        return d

    # differences: h^2 f'''/6 and rounding 1e-16/h, both below 1e-8 of these O(10) losses; the kernel's own fp32
    # error is below 1e-5
    assert np.abs(R.f64(dx) - differences(x, lambda v: loss(v, g, b))).max() < 2e-5
    assert np.abs(R.f64(dg) - differences(g, lambda v: loss(x, v, b))).max() < 2e-5
    if layer:
        assert np.abs(R.f64(db) - differences(b, lambda v: loss(x, g, v))).max() < 2e-5


def test_in_place_partial_outputs_and_no_rows(fp8q):
    """dx written over dy; only one of the weights' gradients through the C entry; no rows at all."""
    say("layernorm backward: in place, partial outputs, no rows")
    x, rng = _inputs(50, 600, torch.bfloat16, 5, extra=0)
    dy = R.place(rng.standard_normal((50, 600)), torch.bfloat16)
    gamma, beta = _weights(rng, 600)
    f = fp8q.layernorm(x, gamma, beta)
    dx, dgamma, dbeta = fp8q.layernorm_backward(dy, x, gamma, f.mean, f.rstd)
    need = fp8q.fp8q_layernorm_backward_workspace(50, 600)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    only = torch.empty(600, device="cuda")
    inplace = dy.clone(memory_format=torch.preserve_format)
    buf = torch.empty((50, 600), dtype=torch.bfloat16, device="cuda")
    buf.copy_(inplace)
    args = (x.data_ptr(), x.stride(0), 1, 50, 600, gamma.data_ptr(), 0, f.mean.data_ptr(), f.rstd.data_ptr(), 0, None, 0)
    assert fp8q.fp8q_layernorm_backward(buf.data_ptr(), 600, *args, buf.data_ptr(), 600, None, only.data_ptr(), 0,
                                        ws.data_ptr(), need, st) == 0
    assert torch.equal(buf, dx) and torch.equal(only, dbeta)
    out = torch.empty_like(buf)
    assert fp8q.fp8q_layernorm_backward(dy.data_ptr(), dy.stride(0), *args, out.data_ptr(), 600, None, None, 0, None, 0,
                                        st) == 0
    assert torch.equal(out, dx)
    none = x[:0]
    f0 = fp8q.layernorm(none, gamma, beta, out_dtype=torch.bfloat16)
    d0 = fp8q.layernorm_backward(none, none, gamma, f0.mean, f0.rstd)
    assert d0[0].shape == (0, 600) and not d0[1].any() and not d0[2].any()
    keep = torch.ones(600, device="cuda")
    fp8q.layernorm_backward(none, none, gamma, f0.mean, f0.rstd, dgamma=keep, dbeta=keep.clone(), accumulate=True)
    assert bool((keep == 1).all())


def test_rows_past_32_bit_offsets(fp8q):
    """A row stride that puts the last row beyond 2^32 bytes."""
    say("layernorm: far rows")
    ld = 1 << 29
    buf = torch.zeros(9 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((9, 256), (ld, 1))
    v = torch.randn((9, 256), device="cuda").to(torch.bfloat16)
    x.copy_(v)
    far, near = fp8q.layernorm(x, out_dtype=torch.float32), fp8q.layernorm(v, out_dtype=torch.float32)
    assert torch.equal(far.y, near.y) and torch.equal(far.q, near.q)
    d = torch.randn((9, 256), device="cuda").to(torch.bfloat16)
    a = fp8q.layernorm_backward(d, x, None, far.mean, far.rstd)
    b = fp8q.layernorm_backward(d, v, None, near.mean, near.rstd)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_more_rows_than_one_grid_dimension_holds(fp8q):
    """Wide rows with a work-group of 1024 threads each, past the 2^32 threads of one grid dimension."""
    say("layernorm: 2^22 + 3 rows")
    rows, cols = (1 << 22) + 3, 8200
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GB of device memory")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    ends = [0, (1 << 20) - 1, 1 << 20, (1 << 22) - 1, 1 << 22, rows - 1]
    some = torch.randn((len(ends), cols), generator=torch.Generator().manual_seed(5)).to(x)
    x[ends] = some
    big, few = fp8q.layernorm(x), fp8q.layernorm(some)
    for name in ("q", "mean", "rstd"):
        assert torch.equal(getattr(big, name)[ends], getattr(few, name)), name
    assert torch.equal(big.s[:, ends], few.s)
    assert not big.q[1].any() and float(big.rstd[1]) == pytest.approx(1e-5 ** -0.5)
    del x, big
    torch.cuda.empty_cache()
