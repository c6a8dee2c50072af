"""Norms at the ends of the number range: tiny and huge rows with eps = 0, NaN
and infinities beside rows of zeros, no columns at all."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
KINDS = ["layer", "rms"]
# one shape for each layout of a row: 16 lanes, a wave, several waves of a team, a work-group
SHAPES = [(40, 100), (14, 400), (2100, 700), (2100, 1800), (2100, 2504), (2100, 6001), (12, 2000), (12, 8000), (12, 12000)]


def _kind(fp8q, kind):
    return fp8q.FP8Q_NORM_LAYER if kind == "layer" else fp8q.FP8Q_NORM_RMS


@pytest.mark.parametrize("eps", [0.0, 1e-37])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_of_any_magnitude(fp8q, rows, cols, dtype, kind, eps):
    """Rows of 2^-115 to 2^100, whose squares leave the range of fp32 on either side: the statistics do not."""
    say(f"layernorm magnitudes {rows}x{cols} {dtype} {kind} eps={eps}")
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((rows, cols))
    for i, e in enumerate((-115, -90, -70, -60, -50, -20, 0, 50, 60, 64, 80, 100)):
        x[i if rows < 100 else 170 * i] *= 2.0 ** e
    x = R.place(x, dtype)
    o = fp8q.layernorm(x, eps=eps, kind=_kind(fp8q, kind), out_dtype=torch.float32)
    y, _, rstd, e_y, _, e_r = R.layernorm(R.f64(x), np.ones(cols), np.zeros(cols), float(np.float32(eps)), kind == "layer")
    R.assert_close(o.rstd, rstd, e_r, "rstd")
    R.assert_close(o.y, y, e_y, "y")


@pytest.mark.parametrize("mode", [0, 1], ids=["fp32", "pow2"])
@pytest.mark.parametrize("value", [float("nan"), -float("nan"), float("inf"), -float("inf")], ids=["nan", "-nan", "inf", "-inf"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(40, 100), (10, 400), (2100, 700), (2100, 2504), (12, 2000), (12, 12000)])
def test_nonfinite_shows(fp8q, rows, cols, kind, value, mode):
    """One NaN or infinity in a row: codes and scale show every result of that row that is no finite number; other rows
    keep their bits, those of zeros beside it too."""
    say(f"layernorm non-finite {rows}x{cols} {kind} {value} mode {mode}")
    x = R.place(np.random.default_rng(7).standard_normal((rows, cols)), torch.bfloat16)
    x[6] = 0
    call = dict(kind=_kind(fp8q, kind), scale_mode=mode)
    clean = fp8q.layernorm(x, **call)
    x[5, cols // 2] = value
    o, y = fp8q.layernorm(x, **call), fp8q.layernorm(x, out_dtype=torch.float32, **call).y
    bad = ~torch.isfinite(y)
    assert bool(bad[5].any()) and int(bad.any(dim=1).sum()) == 1
    v = o.q.contiguous().view(torch.float8_e4m3fn).float() * o.s.t().repeat_interleave(128, dim=1)[:, :cols]
    assert bool((~torch.isfinite(v[5]))[bad[5]].all())
    keep = torch.arange(rows, device="cuda") != 5
    assert torch.equal(o.q[keep], clean.q[keep]) and torch.equal(o.s[:, keep], clean.s[:, keep])


def test_no_columns(fp8q):
    """Rows without columns have no mean and no variance: NaN, as the mean of nothing is, and never what the memory held."""
    say("layernorm: no columns")
    torch.full((1 << 16,), 7.0, device="cuda")
    o = fp8q.layernorm(torch.empty((300, 0), dtype=torch.float32, device="cuda"), out_dtype=torch.float32)
    assert o.q.shape == (300, 0) and o.s.shape == (0, 300) and o.y.shape == (300, 0)
    assert bool(torch.isnan(o.mean).all()) and bool(torch.isnan(o.rstd).all())
