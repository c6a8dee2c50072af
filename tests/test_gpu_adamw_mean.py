"""The mean of 8-bit second moments beside that of fp32 ones: as far above it as the header says."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("beta2,steps,above", [(0.9, 100, 0.014), (0.95, 150, 0.024), (0.99, 600, 0.048)])
def test_mean_second_moment(fp8q, beta2, steps, above):
    """Six time constants of the moving average and more.  The header's figures have two digits, and the mean of 2^16
    elements, each within a third of its own value, one of a thousand: 0.005 is allowed."""
    n = 1 << 16
    gen = torch.Generator(device=DEV).manual_seed(61)
    ps, g = [torch.zeros(n, device=DEV) for _ in range(2)], torch.zeros(n, device=DEV)
    sts = [fp8q.adamw_state(p, bits) for p, bits in zip(ps, (32, 8))]
    plans = [fp8q.adamw_tensors([p], [g], [st]) for p, st in zip(ps, sts)]
    ratios = []
    for step in range(1, steps + 1):
        g.copy_(torch.randn(n, generator=gen, device=DEV))
        for plan in plans:
            fp8q.adamw(plan, step=step, lr=0.0, beta2=beta2, seed=6, weight_decay=0.0)
        if step > steps - 20:
            root = sts[1].v.view(torch.float8_e4m3fn).double().view(-1, 128) * sts[1].sv.double()[:, None]
            ratios.append(float(root.square().mean() / sts[0].v.double().mean()))
    mean = sum(ratios) / len(ratios)
    assert abs(mean - 1.0 - above) <= 0.005, mean
