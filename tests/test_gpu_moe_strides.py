"""Axes of one element carry no stride: mixture-of-experts operands whose single
expert or single block row has whatever stride a view left it."""
import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 3, 20])
@pytest.mark.parametrize("E,H,I", [(1, 256, 128), (4, 128, 256), (1, 128, 128)])
def test_strides_of_single_elements(fp8q, T, E, H, I):
    say(f"moe single elements T={T} E={E} H={H} I={I}")
    gen = torch.Generator(device="cuda").manual_seed(E + H)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    w = [torch.randint(0, 0x70, s, generator=gen, device="cuda", dtype=torch.uint8) for s in ((E, 2 * I, H), (E, H, I))]
    s = [torch.rand((E, t.shape[1] // 128, t.shape[2] // 128), generator=gen, device="cuda") * 1e-3 for t in w]
    want = fp8q.moe_decode(x, logits, w[0], s[0], w[1], s[1], 2)

    def single(t, stride):
        return t.as_strided(t.shape, [stride if n == 1 else old for n, old in zip(t.shape, t.stride())])

    for stride in (0, 1, 1 << 40):
        a = [single(t, stride) for t in (w[0], s[0], w[1], s[1])]
        assert torch.equal(fp8q.moe_decode(x, single(logits, stride), *a, 2), want)
