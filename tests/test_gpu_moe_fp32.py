"""An fp32 result of the mixture-of-experts layer is good to fp32: nothing
between its inputs and its output is held in fewer bits."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say
from tests.test_gpu_moe import _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,top_k,H,I", [
    (1, 4, 2, 256, 2048), (4, 8, 2, 384, 1024), (8, 64, 3, 256, 512), (16, 16, 4, 256, 1024), (33, 12, 3, 256, 512),
    (64, 8, 8, 384, 512), (64, 64, 8, 1024, 512)])
def test_error_of_an_fp32_result(fp8q, T, E, top_k, H, I):
    """Of the roundings of 2^-24 on the way to a result (a chunk's products in four matrix instructions, at most 16 chunks
    and four waves one after the other, in each of two products; six of the SwiGLU; three and top_k sums at the end) the
    independent ones add up as their root: below sqrt(2 * 24 + 6 + 3 + top_k) = 8 for the first product's, which pass
    through a factor of at most 1.1, and the rest.  20 * 2^-24 of the result in the 2-norm is allowed; two bf16 numbers in
    place of h are 40."""
    say(f"moe fp32 T={T} E={E} k={top_k} H={H} I={I}")
    x, logits, w_gu, s_gu, w_down, s_down = _layer(5 * T + E, T, E, H, I)
    y = fp8q.moe_decode(x, torch.from_numpy(logits).cuda(), w_gu, s_gu, w_down, s_down, top_k, out_dtype=torch.float32)
    want, _ = R.moe(R.f64(x), logits.astype(np.float64), w_gu, s_gu, w_down, s_down, top_k, True)
    off = np.linalg.norm(R.f64(y) - want) / np.linalg.norm(want)
    say(f"  {off / R.U:.1f} * 2^-24")
    assert off <= 20 * R.U
