"""The mixture-of-experts layer for at most eight tokens, on both sides of the
choice between a work-group for all active experts (few of them, or little to
read) and one for each, with short and long contractions of the down
projection."""
import pytest
import torch

from tests.parity import say
from tests.test_gpu_moe import _check, _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,E,top_k,H,I", [
    (1, 2, 2, 128, 16512), (1, 1, 1, 256, 20480), (2, 4, 2, 128, 4224), (8, 8, 3, 128, 2176), (4, 8, 2, 384, 128),
    (8, 9, 3, 128, 640), (1, 64, 8, 256, 1024), (1, 64, 9, 256, 256), (2, 64, 4, 128, 2048), (8, 64, 1, 256, 384),
    (8, 128, 32, 128, 128), (3, 24, 4, 256, 256)])
def test_few_tokens(fp8q, T, E, top_k, H, I, out_dtype):
    say(f"moe few T={T} E={E} k={top_k} H={H} I={I} {out_dtype}")
    _check(fp8q, _layer(T + 3 * E, T, E, H, I, pad=T % 3), top_k, bool(T % 2), out_dtype)
