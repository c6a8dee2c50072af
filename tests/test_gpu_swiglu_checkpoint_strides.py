"""The row stride of a checkpoint's scales as the backward helpers take it: a
single group may carry any, groups that overlap are refused."""
import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
ESHAPE = 2


def _kept(fp8q, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    g, u, dh = (torch.randn((rows, cols), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    return fp8q.swiglu_quantize(g, u)[2], dh


@pytest.mark.parametrize("stride", [0, 1, 1 << 40])
def test_one_group(fp8q, stride):
    say(f"swiglu checkpoint of one group, stride {stride}")
    kept, dh = _kept(fp8q, 33, 128)
    view = kept._replace(**{n: getattr(kept, n).as_strided((1, 33), (stride, 1)) for n in ("sg", "su")})
    for call in (fp8q.swiglu_backward, fp8q.swiglu_backward_quantize):
        assert all(torch.equal(a, b) for a, b in zip(call(view, dh), call(kept, dh)))


def test_overlapping_groups_are_refused(fp8q):
    """One row of scales shared by all groups (row stride 0) is no array that the kernels read: refused, not read with
    another stride."""
    say("swiglu checkpoint with shared scales")
    kept, dh = _kept(fp8q, 33, 384)
    for stride in (0, 32):
        shared = kept._replace(**{n: getattr(kept, n).as_strided((3, 33), (stride, 1)) for n in ("sg", "su")})
        for call in (fp8q.swiglu_backward, fp8q.swiglu_backward_quantize):
            with pytest.raises(fp8q.Fp8qError) as e:
                call(shared, dh)
            assert e.value.status == ESHAPE
