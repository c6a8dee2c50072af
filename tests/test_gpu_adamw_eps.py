"""AdamW with an eps of zero, or near it: the rows that a weight's last band of 128x128 blocks lacks have nothing to
say, and a positive eps stays positive."""
import pytest
import torch

from tests.test_gpu_adamw import DEV, H, _check_codes, _tensor, _Want

pytestmark = pytest.mark.gpu


def _no_zeros(fp8q, shape, gdtype, bits):
    """Gradients that are nowhere zero, so that no second moment is."""
    p, g = _tensor(shape, gdtype, 41)
    g[g == 0] = 3e-4
    return p, g, fp8q.adamw_state(p, bits)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-46])
@pytest.mark.parametrize("shape", [(1, 128), (16, 384), (77, 256), (130, 128), (3, 77, 256), (128, 128)])
def test_codes_of_weights(fp8q, bits, eps, shape):
    for gdtype in (torch.float32, torch.bfloat16):
        for mode in (fp8q.FP8Q_SCALE_FP32, fp8q.FP8Q_SCALE_POW2):
            p, g, st = _no_zeros(fp8q, shape, gdtype, bits)
            c = fp8q.weight_codes(p, scale_mode=mode)
            want = _Want(p, g, st, 1, 5, 0, eps=eps)
            fp8q.adamw(fp8q.adamw_tensors([p], [g], [st], [c]), step=1, seed=5, scale_mode=mode, **{**H, "eps": eps})
            want.check(p, st)
            _check_codes(fp8q, p, c, mode)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_over_zero_shows_in_its_element_and_its_block(fp8q, bits):
    """Where eps, m and v are all zero the formula is 0 / 0: NaN in that element and in the scale of its block, as the
    quantizer has it; every other element is as if it were not there."""
    p, g, st = _no_zeros(fp8q, (200, 256), torch.float32, bits)
    other, so = p.clone(), fp8q.adamw_state(p, bits)
    c, co = fp8q.weight_codes(p), fp8q.weight_codes(other)
    go = g.clone()
    g[130, 5] = 0.0
    for args in ((p, g, st, c), (other, go, so, co)):
        fp8q.adamw(fp8q.adamw_tensors(*([a] for a in args)), step=1, seed=5, **{**H, "eps": 0.0})
    at = torch.zeros_like(p, dtype=torch.bool)
    at[130, 5] = True
    assert p[at].isnan().all() and torch.equal(p[~at], other[~at])
    q, s = fp8q.quantize_weight(p)
    assert c.s.isnan().tolist() == [[False, False], [True, False]] == s.isnan().tolist()
    assert torch.equal(c.s.nan_to_num(7.0), s.nan_to_num(7.0))
    assert torch.equal(c.st.t().nan_to_num(7.0), s.nan_to_num(7.0))
    live = torch.ones_like(p, dtype=torch.bool)
    live[128:, :128] = False  # the codes of that block multiply a NaN
    assert torch.equal(c.q[live], q[live]) and torch.equal(c.q[live], co.q[live])


def test_flat_tensors(fp8q):
    """Lengths that end inside a work-group, a tile and a lane's eight elements."""
    for bits in (32, 8):
        for n in (1, 7, 130, 2049):
            p, g, st = _no_zeros(fp8q, (n,), torch.float32, bits)
            want = _Want(p, g, st, 2, 5, 0, eps=0.0)
            fp8q.adamw(fp8q.adamw_tensors([p], [g], [st]), step=2, seed=5, **{**H, "eps": 0.0})
            want.check(p, st)
            assert torch.isfinite(p).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-46, 5e-324, 1e-40, 2.0 ** -149])
def test_small_eps_is_not_zero(fp8q, bits, eps):
    """No gradient and no moments: 0 / eps is 0 for every positive eps, so only the decay is left."""
    p = torch.randn((77, 256), device=DEV)
    before, st = p.clone(), fp8q.adamw_state(p, bits)
    c = fp8q.weight_codes(p)
    vec = torch.randn(300, device=DEV)
    vec_before, vec_st = vec.clone(), fp8q.adamw_state(vec, bits)
    plan = fp8q.adamw_tensors([p, vec], [torch.zeros_like(p), torch.zeros_like(vec)], [st, vec_st], [c, None])
    fp8q.adamw(plan, step=1, lr=0.5, weight_decay=0.5, eps=eps)
    assert torch.equal(p, before * 0.75) and torch.equal(vec, vec_before * 0.75)
    _check_codes(fp8q, p, c)
