"""How far 8-bit moments can move an element that is tiny beside its tile's largest."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_movement_of_tiny_elements(fp8q):
    """Gradients of 1e-6 beside one of 1, then none.  A step moves an element by
        lr C (b1 M + (1 - b1) g) / sqrt(b2 R^2 + (1 - b2) g^2),  C = sqrt(1 - b2^t) / (1 - b1^t)
    at most, with M and R what is held of m and sqrt(v).  M of a tiny element is at most two of the smallest codes: 1e-6
    is less than one of them (amax / 448 / 512 > 2e-6 from the third step on, and 1e-6 (1 - b1^t) against 4e-6 (1 - b1^t)
    before), so from one code's value on it falls; and one is above it by a rounding's error.  R is at least one of its
    smallest codes.  For the tile's largest, whose codes are 448 exactly, it is the quotient of exact moments, at most
    (1 - b1) / sqrt((1 - b2) (1 - b1^2 / b2)).  20 fp32 roundings."""
    b1, b2, tiny, n = 0.9, 0.95, 1e-6, 128 * 64
    g = torch.full((n,), tiny, device=DEV)
    g[::128] = 1.0
    large = torch.zeros(n, dtype=torch.bool, device=DEV)
    large[::128] = True
    p = torch.zeros(n, device=DEV)
    st = fp8q.adamw_state(p, 8)
    plan = fp8q.adamw_tensors([p], [g], [st])
    slack = 1 + 20 * 2.0 ** -24
    for step in range(1, 40):
        if step == 20:
            g.zero_()
        sm, sv = (s.double().repeat_interleave(128) for s in (st.sm, st.sv))
        p.zero_()
        fp8q.adamw(plan, step=step, lr=1.0, beta1=b1, beta2=b2, weight_decay=0.0, seed=4)
        c = math.sqrt(1 - b2 ** step) / (1 - b1 ** step)
        x = g.double()
        most = c * (b1 * 2 * 2.0 ** -9 * sm + (1 - b1) * x) / (b2 * (2.0 ** -9 * sv).square() + (1 - b2) * x * x).sqrt()
        most[large] = c * (1 - b1) / math.sqrt((1 - b2) * (1 - b1 * b1 / b2))
        assert (p.double().abs() <= most * slack).all(), (step, float((p.double().abs() / most).max()))
        assert ((st.m & 0x7F)[~large] <= 2).all() and (st.v[~large] >= 1).all()
        assert ((st.m & 0x7F)[large] == 0x7E).all() and (st.v[large] == 0x7E).all()
