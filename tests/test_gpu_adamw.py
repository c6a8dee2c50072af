"""The AdamW step over many tensors against its 64-bit form, within bounds of the fp32 evaluation (expert_ref.py)."""
import numpy as np
import pytest
import torch

from tests import expert_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
H = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _tensor(shape, gdtype, seed):
    rng = np.random.default_rng(seed)
    p = rng.standard_normal(shape) * 0.05
    g = rng.standard_normal(shape) * np.exp(rng.uniform(-4, 4, shape)) * 1e-3
    g[rng.random(shape) < 0.05] = 0.0
    return (torch.from_numpy(p).float().to(DEV), torch.from_numpy(g).to(gdtype).to(DEV))


def _state(fp8q, p, bits, seed):
    st = fp8q.adamw_state(p, bits)
    rng, n = np.random.default_rng(seed), p.numel()
    if bits == 32:
        st.m.copy_(torch.from_numpy(rng.standard_normal(n) * 1e-3))
        st.v.copy_(torch.from_numpy(np.exp(rng.uniform(-20, -8, n))))
        st.v[rng.random(n) < 0.03] = 0.0
    else:
        qm = rng.integers(0, 256, n).astype(np.uint8)
        qm[(qm & 0x7F) == 0x7F] = 0
        st.m.copy_(torch.from_numpy(qm))
        st.v.copy_(torch.from_numpy(rng.integers(0, 0x7F, n).astype(np.uint8)))
        for s in (st.sm, st.sv):
            s.copy_(torch.from_numpy(np.exp(rng.uniform(-12, -9, s.numel()))))
            s[rng.random(s.numel()) < 0.1] = 0.0
    return st


def _moments(st):
    """(m, v) in 64 bits"""
    if st.sm is None:
        return st.m.double().cpu().numpy(), st.v.double().cpu().numpy()
    n = st.m.numel()
    m, r = (R.e4m3(q.cpu().numpy()) * np.repeat(s.double().cpu().numpy(), 128)[:n] for q, s in ((st.m, st.sm), (st.v, st.sv)))
    return m, r * r


class _Want:
    """What one tensor's step gives: 64 bits with bounds, and the 8-bit moments bit for bit."""

    def __init__(self, p, g, st, step, seed=0, place=0, scale=1.0, **kw):
        h = {**H, **kw}
        m, v = _moments(st)
        g = g.double().cpu().numpy().reshape(-1)
        self.plain = R.adamw(p.double().cpu().numpy().reshape(-1), g, m, v, h["lr"], h["beta1"], h["beta2"], h["eps"],
                             h["weight_decay"], step, scale)
        self.coded = None
        if st.sm is not None:
            args = [t.cpu().numpy() for t in (st.m, st.sm, st.v, st.sv)]
            self.coded = R.moments_8bit(*args, g * scale, h["beta1"], h["beta2"], seed, place, step)

    def check(self, p, st):
        p1, m1, v1, ep, em, ev = self.plain
        got = p.double().cpu().numpy().reshape(-1)
        assert (np.abs(got - p1) <= ep).all(), float(np.max(np.abs(got - p1) / ep))
        if self.coded is None:
            assert (np.abs(st.m.double().cpu().numpy() - m1) <= em).all()
            assert (np.abs(st.v.double().cpu().numpy() - v1) <= ev).all()
            return
        cm, sm, cv, sv = self.coded
        assert np.array_equal(st.sm.cpu().numpy(), sm) and np.array_equal(st.sv.cpu().numpy(), sv)
        for q, c in ((st.m, cm), (st.v, cv)):
            bits = q.cpu().numpy()
            assert np.array_equal(R.e4m3(bits), c.astype(np.float64))
            assert np.array_equal((bits & 0x80) != 0, np.signbit(c))


SIZES = [1, 2, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 4096, 33333]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step", [1, 5, 100000])
def test_vectors(fp8q, bits, gdtype, step):
    ts = [_tensor((n,), gdtype, i) for i, n in enumerate(SIZES)]
    sts = [_state(fp8q, p, bits, 100 + i) for i, (p, _) in enumerate(ts)]
    want = [_Want(p, g, st, step, 77, i) for i, ((p, g), st) in enumerate(zip(ts, sts))]
    plan = fp8q.adamw_tensors([p for p, _ in ts], [g for _, g in ts], sts)
    fp8q.adamw(plan, step=step, seed=77, **H)
    for (p, _), st, w in zip(ts, sts, want):
        w.check(p, st)


def _check_codes(fp8q, p, c, mode=0):
    """The codes are those of the quantizer and the transposer on the new weights."""
    mats = p.reshape((-1,) + tuple(p.shape[-2:]))
    lead = (mats.shape[0],)
    for e in range(mats.shape[0]):
        q, s = fp8q.quantize_weight(mats[e], scale_mode=mode)
        assert torch.equal(c.q.reshape(lead + tuple(q.shape))[e], q)
        assert torch.equal(c.s.reshape(lead + tuple(s.shape))[e], s)
        if c.qt is not None:
            qt, st = fp8q.transpose_weight(q, s)
            assert torch.equal(c.qt[e] if p.dim() == 3 else c.qt, qt)
            assert torch.equal(c.st.reshape(lead + tuple(st.shape))[e], st)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shape", [(128, 128), (1, 128), (130, 384), (3, 77, 256), (2, 256, 128), (5, 16, 640)])
@pytest.mark.parametrize("transposed", [True, False])
def test_weights_with_codes(fp8q, bits, shape, transposed):
    for gdtype in (torch.float32, torch.bfloat16):
        for mode in (fp8q.FP8Q_SCALE_FP32, fp8q.FP8Q_SCALE_POW2):
            p, g = _tensor(shape, gdtype, 3)
            st = _state(fp8q, p, bits, 4)
            c = fp8q.weight_codes(p, transposed=transposed, scale_mode=mode)
            _check_codes(fp8q, p, c, mode)
            vec, vg = _tensor((300,), gdtype, 5)
            vst = _state(fp8q, vec, bits, 6)
            want = [_Want(vec, vg, vst, 9, 5, 0), _Want(p, g, st, 9, 5, 1)]
            plan = fp8q.adamw_tensors([vec, p], [vg, g], [vst, st], [None, c])
            fp8q.adamw(plan, step=9, seed=5, scale_mode=mode, **H)
            want[0].check(vec, vst)
            want[1].check(p, st)
            _check_codes(fp8q, p, c, mode)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(fp8q, bits):
    """Vectors and weights mixed, several launches of each kind."""
    shapes = [(1 + 37 * i,) if i % 2 else (1 + i % 5, 128) for i in range(150)]
    ts = [_tensor(s, torch.float32, i) for i, s in enumerate(shapes)]
    sts = [_state(fp8q, p, bits, i) for i, (p, _) in enumerate(ts)]
    codes = [fp8q.weight_codes(p) if p.dim() == 2 else None for p, _ in ts]
    want = [_Want(p, g, st, 3, 1, i) for i, ((p, g), st) in enumerate(zip(ts, sts))]
    fp8q.adamw(fp8q.adamw_tensors([p for p, _ in ts], [g for _, g in ts], sts, codes), step=3, seed=1, **H)
    for i, ((p, _), st, w) in enumerate(zip(ts, sts, want)):
        w.check(p, st)
        if codes[i] is not None:
            _check_codes(fp8q, p, codes[i])


def test_scalars_on_the_device(fp8q):
    """step, lr and the gradients' factor read when the step runs: the same as given from the host."""
    a, g = _tensor((5000,), torch.float32, 8)
    b = a.clone()
    sa, sb = _state(fp8q, a, 8, 9), _state(fp8q, b, 8, 9)
    want = _Want(a, g, sa, 12, 3, scale=0.25)
    fp8q.adamw(fp8q.adamw_tensors([a], [g], [sa]), step=12, seed=3, grad_scale=torch.tensor([0.25], device=DEV), **H)
    want.check(a, sa)
    h = {**H, "lr": torch.tensor(H["lr"], device=DEV)}
    fp8q.adamw(fp8q.adamw_tensors([b], [g], [sb]), step=torch.tensor(12, device=DEV), seed=3,
               grad_scale=torch.tensor([0.25], device=DEV), **h)
    assert (a - b).abs().max() <= 4 * R.U * a.abs().max()  # lr is an fp32 number there
    assert torch.equal(sa.m, sb.m) and torch.equal(sa.sv, sb.sv)


def test_captured_step_with_eager_steps_between(fp8q):
    p, g = _tensor((3, 100, 256), torch.float32, 10)
    ref = p.clone()
    st, sr = fp8q.adamw_state(p, 8), fp8q.adamw_state(ref, 8)
    c, cr = fp8q.weight_codes(p), fp8q.weight_codes(ref)
    step, lr = torch.zeros((), dtype=torch.int64, device=DEV), torch.tensor(1e-3, device=DEV)
    plan, plan_ref = fp8q.adamw_tensors([p], [g], [st], [c]), fp8q.adamw_tensors([ref], [g], [sr], [cr])
    h = {k: v for k, v in H.items() if k != "lr"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        fp8q.adamw(plan, step=step, lr=lr, seed=2, **h)
    for i in range(1, 5):
        g.copy_(torch.randn(g.shape, device=DEV) * 1e-3 * i)
        lr.fill_(1e-3 / i)
        graph.replay()
        fp8q.adamw(plan_ref, step=torch.tensor(i, device=DEV), lr=lr, seed=2, **h)
        torch.cuda.synchronize()
        assert torch.equal(p, ref) and torch.equal(st.m, sr.m) and torch.equal(st.v, sr.v)
        assert torch.equal(c.q, cr.q) and torch.equal(c.qt, cr.qt) and torch.equal(c.st, cr.st)


def test_rounding_is_unbiased_and_small_moments_move(fp8q):
    """A gradient whose moments stand still in exact arithmetic: the mean of many roundings is the value.  The mean of
    n numbers that are one of two grid points a step apart has a deviation of at most step / (2 sqrt n)."""
    n = 1 << 16
    p, g = torch.zeros(n, device=DEV), torch.full((n,), 0.3, device=DEV)
    g[::128] = 1.0  # the tiles' maxima
    st = fp8q.adamw_state(p, 8)
    fp8q.adamw(fp8q.adamw_tensors([p], [g], [st]), step=1, lr=0.0, beta1=0.9, beta2=0.99, seed=11, weight_decay=0.0)
    live = np.arange(n) % 128 != 0
    for q, s, x in ((st.m, st.sm, 0.1 * 0.3), (st.v, st.sv, np.sqrt(0.01) * 0.3)):
        y = R.e4m3(q.cpu().numpy())[live]
        want = x / float(s[0])
        assert len(np.unique(y)) == 2
        step = 2.0 ** (np.floor(np.log2(want)) - 3)
        assert abs(y.mean() - want) <= 6 * step / (2 * np.sqrt(live.sum()))


def test_moments_never_leave_a_zero_under_a_nonzero(fp8q):
    """Gradients of tiny elements beside large ones: their sqrt(v) keeps a code, and a later step with no gradient
    moves no element by more than the moments allow: |m| / sqrt(v) is at most its bound for exact moments,
    (1 - b1) / sqrt((1 - b2) (1 - b1^2 / b2)), plus one step of a code of each, over the bias corrections."""
    n = 128 * 64
    g = torch.full((n,), 1e-6, device=DEV)
    g[::128] = 1.0
    p = torch.zeros(n, device=DEV)
    st = fp8q.adamw_state(p, 8)
    plan = fp8q.adamw_tensors([p], [g], [st])
    for step in range(1, 40):
        if step == 20:
            g.zero_()
        before = p.clone()
        fp8q.adamw(plan, step=step, lr=1.0, beta1=0.9, beta2=0.95, weight_decay=0.0, seed=4)
        assert (st.v != 0).all()
        assert torch.isfinite(p).all() and (p - before).abs().max() < 40.0


def test_not_finite_gradients_show_where_they_are(fp8q):
    for bits in (32, 8):
        p, g = _tensor((4, 128), torch.float32, 12)
        g[1, 5] = float("nan")
        g[2, 7] = float("inf")
        st = fp8q.adamw_state(p, bits)
        ref, sr = p.clone(), fp8q.adamw_state(p, bits)
        gr = g.clone()
        gr[1, 5] = gr[2, 7] = 0.0
        fp8q.adamw(fp8q.adamw_tensors([p], [g], [st]), step=1, **H)
        fp8q.adamw(fp8q.adamw_tensors([ref], [gr], [sr]), step=1, **H)
        keep = torch.ones_like(p, dtype=torch.bool)
        keep[1, 5] = keep[2, 7] = False
        assert torch.equal(p[keep], ref[keep]) and p[~keep].isnan().all()
        if bits == 8:
            assert not torch.isfinite(st.sm[1:3]).any() and not torch.isfinite(st.sv[1:3]).any()
            assert torch.isfinite(st.sm[[0, 3]]).all()


def test_zero_gradients_from_the_start(fp8q):
    for bits in (32, 8):
        p = torch.randn(1000, device=DEV)
        st, before = fp8q.adamw_state(p, bits), p.clone()
        fp8q.adamw(fp8q.adamw_tensors([p], [torch.zeros_like(p)], [st]), step=1, lr=0.5, weight_decay=0.5)
        assert torch.equal(p, before * 0.75) and not st.m.any() and not st.v.any()


def test_step_follows_the_loss_downhill(fp8q):
    """With zero moments the first step moves p by lr against the gradient's sign; 16 roundings of the update
    (expert_ref.adamw) and two of p."""
    p, g = _tensor((777,), torch.float32, 13)
    before = p.clone()
    fp8q.adamw(fp8q.adamw_tensors([p], [g], [fp8q.adamw_state(p)]), step=1, lr=1e-2, eps=0.0, weight_decay=0.0)
    moved = g != 0
    d = (p - before)[moved].double()
    assert ((d + 1e-2 * g[moved].sign()).abs() <= 3 * R.U * before[moved].abs() + 20 * R.U * 1e-2).all()


def test_on_another_stream(fp8q):
    p, g = _tensor((100000,), torch.bfloat16, 14)
    st = _state(fp8q, p, 8, 15)
    want = _Want(p, g, st, 2)
    plan = fp8q.adamw_tensors([p], [g], [st])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8q.adamw(plan, step=2, **H)
    torch.cuda.current_stream().wait_stream(side)
    want.check(p, st)


def test_writes_nothing_around_the_tensors(fp8q):
    """Tensors inside larger arrays, their neighbours untouched."""
    for bits in (32, 8):
        for n in (5, 128, 1003):
            big = [torch.full((n + 512,), 3.0, device=DEV) for _ in range(4)]
            p, g = big[0][256: 256 + n], big[1][256: 256 + n]
            if bits == 32:
                st = fp8q.AdamwState(big[2][256: 256 + n], big[3][256: 256 + n], None, None)
            else:
                qs = [torch.full((n + 512,), 0x31, dtype=torch.uint8, device=DEV) for _ in range(2)]
                t = -(-n // 128)
                st = fp8q.AdamwState(qs[0][256: 256 + n], qs[1][256: 256 + n], big[2][1: 1 + t], big[3][1: 1 + t])
            fp8q.adamw(fp8q.adamw_tensors([p], [g], [st]), step=1, **H)
            for b in [big[0]] + (big[2:] if bits == 32 else []):
                assert (b[:256] == 3.0).all() and (b[256 + n:] == 3.0).all()
            if bits == 8:
                for q in qs:
                    assert (q[:256] == 0x31).all() and (q[256 + n:] == 0x31).all()
                for b in big[2:]:
                    assert b[0] == 3.0 and (b[1 + t:] == 3.0).all()
            assert (p != 3.0).all()


def test_refuses_scalars_elsewhere(fp8q):
    p = torch.zeros(8, device=DEV)
    plan = fp8q.adamw_tensors([p], [torch.zeros_like(p)], [fp8q.adamw_state(p)])
    for kw in (dict(step=torch.tensor(3), lr=1e-3), dict(step=1, lr=torch.tensor(1e-3)), dict(step=1, lr=1e-3, grad_scale=torch.ones(1)),
               dict(step=torch.tensor(3.0, device=DEV), lr=1e-3), dict(step=torch.ones(2, dtype=torch.int64, device=DEV), lr=1e-3)):
        with pytest.raises(ValueError, match="must be one"):
            fp8q.adamw(plan, **kw)
    for kw in (dict(step=0, lr=1e-3), dict(step=1, lr=-1.0), dict(step=1, lr=1e-3, beta1=1.0)):
        with pytest.raises(fp8q.Fp8qError):
            fp8q.adamw(plan, **kw)
    with pytest.raises(ValueError, match="overlap"):
        fp8q.adamw_tensors([p, p], [torch.zeros_like(p)] * 2, [fp8q.adamw_state(p), fp8q.adamw_state(p)])
    assert not p.any()


@pytest.mark.parametrize("coded", [False, True])
def test_more_elements_than_32_bits_count(fp8q, coded):
    """Behind 2^32 elements the random numbers start again, so what stands there steps like a tensor of its own."""
    rows, K = 40, 128
    small, sg = _tensor((rows, K), torch.bfloat16, 31)
    st = _state(fp8q, small, 8, 32)
    before, n = (1 << 32) // K, (1 << 32) + rows * K
    p = torch.zeros((before + rows, K), device=DEV)
    g = torch.zeros((before + rows, K), dtype=torch.bfloat16, device=DEV)
    big = fp8q.AdamwState(*(torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)),
                          *(torch.zeros(n // 128, device=DEV) for _ in range(2)))
    p[before:], g[before:] = small, sg
    for b, t in zip(big, st):
        b[-t.numel():] = t
    codes = [None, None]
    if coded:
        n16 = (before + rows + 15) // 16 * 16
        blocks = -(-(before + rows) // 128)
        codes = [fp8q.weight_codes(small),
                 fp8q.WeightCodes(torch.zeros((before + rows, K), dtype=torch.uint8, device=DEV),
                                  torch.zeros((blocks, 1), device=DEV),
                                  torch.zeros((K, n16), dtype=torch.uint8, device=DEV)[:, : before + rows],
                                  torch.zeros((1, blocks), device=DEV))]
    for one in ((small, sg, st, codes[0]), (p, g, big, codes[1])):
        fp8q.adamw(fp8q.adamw_tensors(*([v] for v in one)), step=3, seed=5, **H)
    assert torch.equal(p[before:], small) and not p[before - 1000: before].any()
    for b, t in zip(big, st):
        assert torch.equal(b[-t.numel():], t) and not b[-t.numel() - 1000: -t.numel()].any()
    if coded:
        a, b = codes
        assert torch.equal(b.q[before:], a.q) and torch.equal(b.s[-1], a.s[0])
        assert torch.equal(b.qt[:, before:], a.qt) and torch.equal(b.st[:, -1], a.st[:, 0])
