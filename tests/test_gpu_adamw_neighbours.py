"""An element's step does not depend on the values beside it, and its quotient is the rounded one."""
import numpy as np
import pytest
import torch

from tests.test_gpu_adamw import DEV, H, _tensor

pytestmark = pytest.mark.gpu


def _f32(x):
    return torch.tensor(x, dtype=torch.float32, device=DEV)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("coded", [False, True])
def test_an_element_and_its_neighbours(fp8q, bits, coded):
    """The same tensor with one element's gradient zero, tiny or huge: every other element's p is the same, bit for bit
    (its moments before the rounding are its own; codes of the others change with their tile's maximum)."""
    shape, at = ((256, 256), (129, 77)) if coded else ((8192,), (4990,))  # all 64 lanes have elements
    results = []
    for value in (1e-3, 0.0, 1e-30, 1e15):
        p, g = torch.zeros(shape, device=DEV), _tensor(shape, torch.float32, 51)[1]
        g[g == 0] = 3e-4
        g[at] = value
        st = fp8q.adamw_state(p, bits)
        codes = [fp8q.weight_codes(p)] if coded else None
        fp8q.adamw(fp8q.adamw_tensors([p], [g], [st], codes), step=1, seed=5, **H)
        p[at] = 0.0
        results.append(p)
    for other in results[1:]:
        assert torch.equal(other, results[0])


def test_the_quotient_is_rounded_to_nearest(fp8q):
    """With p = 0, no decay and lr / (1 - beta1) = 1 the step is -fl32(m' / (fl32(sqrt(v')) root + eps)), each
    operation rounded once."""
    n = 1 << 18
    rng = np.random.default_rng(52)
    g = (rng.standard_normal(n) * np.exp(rng.uniform(-12, 12, n))).astype(np.float32)
    g[g == 0] = 1.0
    p = torch.zeros(n, device=DEV)
    st = fp8q.adamw_state(p)
    fp8q.adamw(fp8q.adamw_tensors([p], [_f32(g)], [st]), step=1, lr=0.5, beta1=0.5, beta2=0.75, eps=1e-8, weight_decay=0.0)
    f = np.float32
    m, v = st.m.cpu().numpy(), st.v.cpu().numpy()
    assert np.array_equal(m, g * f(0.5)) and np.array_equal(v, g * g * f(0.25))
    d = np.sqrt(v) * f(2.0) + f(1e-8)  # sqrt(1 - 3/4) = 1/2
    assert np.array_equal(p.cpu().numpy(), -(m / d))


def test_sums_of_fp32_moments_round_once(fp8q):
    """m' = fl32(fl32(beta1 m) + (1 - beta1) x) and v' = fl32(fl32(beta2 v) + (1 - beta2) fl32(x^2)): with 5/8 and 3/8 the
    factors are exact, and the sums are exact in 64 bits (numbers within 2^+-10)."""
    n = 1 << 16
    rng = np.random.default_rng(53)
    g, m, v = (np.exp(rng.uniform(-3, 3, n)).astype(np.float32) for _ in range(3))
    g[::2] *= -1
    p = torch.zeros(n, device=DEV)
    st = fp8q.adamw_state(p)
    st.m.copy_(_f32(m))
    st.v.copy_(_f32(v))
    fp8q.adamw(fp8q.adamw_tensors([p], [_f32(g)], [st]), step=3, lr=0.5, beta1=0.625, beta2=0.625)
    f, d = np.float32, np.float64
    assert np.array_equal(st.m.cpu().numpy(), ((m * f(0.625)).astype(d) + 0.375 * g.astype(d)).astype(f))
    assert np.array_equal(st.v.cpu().numpy(), ((v * f(0.625)).astype(d) + 0.375 * (g * g).astype(d)).astype(f))
