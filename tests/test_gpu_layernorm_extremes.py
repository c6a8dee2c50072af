"""Norms at the ends of the number range: NaN and infinities beside rows of zeros."""
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
