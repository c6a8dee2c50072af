"""The SwiGLU's backward pass into FP8 operands over more than one band of
eight row tiles, the last band full, short or a single partial tile, against
the plain backward pass and the quantizers, bit for bit."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [0, 1], ids=["fp32", "pow2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1024, 384), (1025, 384), (1300, 520), (2176, 256), (3100, 200), (2048, 1000)])
def test_backward_quantize(fp8q, rows, cols, dtype, mode):
    say(f"swiglu backward bands {rows}x{cols} {dtype} mode {mode}")
    rng = np.random.default_rng(rows + cols)
    g, u, dh = (R.place(rng.standard_normal((rows, cols)) * f, dtype, 1) for f in (2.0, 1.0, 1e-3))
    kept = fp8q.swiglu_quantize(g, u, scale_mode=mode)[2]
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
