"""Norms around the number of rows at which teams of lanes take over from a
work-group per row (four to eight for each compute unit, by the row's layout):
both sides of it."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [520, 1001, 2000, 2048, 2049, 2504, 4097, 7168])
def test_both_sides_of_the_change(fp8q, cols, dtype, kind):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    layer = kind == "layer"
    k = fp8q.FP8Q_NORM_LAYER if layer else fp8q.FP8Q_NORM_RMS
    rng = np.random.default_rng(cols)
    rows = (5 if cols <= 1024 else 8 if cols <= 2048 else 4 if cols <= 4096 else 6) * cus
    say(f"layernorm {rows - 1} and {rows} x {cols} {dtype} {kind}")
    x = R.place(rng.standard_normal((rows, cols)) + 0.5, dtype, 1)
    gamma = torch.from_numpy(rng.standard_normal(cols) * 0.2 + 1).float().cuda()
    y, mean, rstd, e_y, e_m, e_r = R.layernorm(R.f64(x), R.f64(gamma), np.zeros(cols), 1e-5, layer)
    for n in (rows - 1, rows):
        o = fp8q.layernorm(x[:n], gamma, eps=1e-5, kind=k, out_dtype=torch.float32)
        R.assert_close(o.y, y[:n], e_y[:n], "y")
        R.assert_close(o.rstd, rstd[:n], e_r[:n], "rstd")
        R.assert_codes_of(o.q, o.s, y[:n], e_y[:n], False, "codes")
