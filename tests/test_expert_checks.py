"""What the experts' weight gradients, their operands and the AdamW step refuse: the C entry points' status for each
kind of invalid argument and the tensor helpers' own checks (nothing is launched, so no GPU is needed)."""
import ctypes

import pytest
import torch

import fp8_fine_grained_x128_amd as f

FAKE = 1 << 20  # an aligned, never-dereferenced address


def _caller(fn, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return fn(*{**ok, **kw}.values())
    return call


@pytest.mark.parametrize("rows,G,want", [(0, 4, 0), (1, 1, 128), (1, 1024, 128), (128, 1, 128), (129, 1, 256), (4, 4, 512),
                                         (300, 2, 512), (1000, 8, 1920), (-1, 2, 0), (5, -1, 0)])
def test_padded_rows(rows, G, want):
    assert f.fp8q_grouped_padded_rows(rows, G) == want


def test_padded_rows_hold_every_division():
    """Against all ways to divide few rows among few groups (in whole chunks of 128 the worst is a group of 1 more)."""
    for G in (1, 2, 3, 5):
        for rows in list(range(0, 12)) + [127, 128, 129, 255, 256, 257, 384, 385, 386]:
            room = f.fp8q_grouped_padded_rows(rows, G) // 128
            most = 0
            for ones in range(0, min(G, rows) + 1):  # `ones` groups of 128 k + 1 rows, the rest in one group
                rest = rows - ones
                if rest < 0 or (ones == G and rest % 128):
                    continue
                most = max(most, ones + -(-rest // 128) if ones < G else ones + rest // 128)
            assert room >= most, (G, rows)


def test_grouped_quantize_act():
    c = _caller(f.fp8q_grouped_quantize_act, dict(x=FAKE, xt=1, rows=300, cols=256, ldx=256, off=FAKE, G=4, qt=FAKE,
                                                  ldqt=768, st=FAKE, ldst=256, mode=0))
    for kw in (dict(xt=2), dict(mode=2), dict(x=0), dict(off=0), dict(qt=0), dict(st=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-1), dict(cols=-1), dict(ldx=255), dict(G=0), dict(G=1025), dict(ldqt=752), dict(ldst=255),
               dict(ldqt=1 << 33)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(ldx=260), dict(off=FAKE + 2), dict(qt=FAKE + 8), dict(ldqt=776), dict(st=FAKE + 2)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    assert c(rows=128 * 65536, ldqt=1 << 30) == f.FP8Q_EUNSUPPORTED
    assert c(rows=1 << 31, ldqt=1 << 32) == f.FP8Q_EUNSUPPORTED
    assert c(rows=0, x=0, off=0, qt=0, st=0) == f.FP8Q_OK and c(cols=0, x=0, qt=0, st=0) == f.FP8Q_OK


def test_grouped_requant_transpose():
    c = _caller(f.fp8q_grouped_requant_transpose, dict(q=FAKE, rows=300, cols=256, ldq=256, s=FAKE, lds=300, off=FAKE, G=4,
                                                       qt=FAKE, ldqt=768, st=FAKE, ldst=256, mode=0))
    for kw in (dict(mode=2), dict(q=0), dict(s=0), dict(off=0), dict(qt=0), dict(st=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-1), dict(cols=-1), dict(ldq=255), dict(lds=299), dict(G=0), dict(ldqt=752), dict(ldst=255)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(q=FAKE + 8), dict(ldq=264), dict(s=FAKE + 2), dict(off=FAKE + 1), dict(qt=FAKE + 4), dict(ldqt=776)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    assert c(rows=0, q=0) == f.FP8Q_OK


def test_grouped_wgrad():
    rows, G, N, K = 300, 4, 256, 512
    need = f.fp8q_grouped_wgrad_workspace(rows, G, N, K)
    c = _caller(f.fp8q_grouped_wgrad, dict(
        a=FAKE, lda=768, sa=FAKE, ldsa=N, b=FAKE, ldb=768, sb=FAKE, ldsb=K, off=FAKE, G=G, rows=rows, N=N, K=K, dw=FAKE,
        dt=0, lddw=K, gs=N * K, acc=0, flags=0, ws=FAKE, wsb=need))
    for kw in (dict(dt=2), dict(flags=4), dict(a=0), dict(sa=0), dict(b=0), dict(sb=0), dict(off=0), dict(dw=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-1), dict(N=-1), dict(K=-1), dict(G=0), dict(G=1025), dict(lda=752), dict(ldb=752), dict(ldsa=255),
               dict(ldsb=511), dict(lddw=511), dict(gs=N * K - 1), dict(gs=-1), dict(wsb=-1), dict(lda=1 << 33)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(a=FAKE + 8), dict(lda=776), dict(b=FAKE + 8), dict(ldb=776), dict(sa=FAKE + 2), dict(sb=FAKE + 2),
               dict(dw=FAKE + 2), dict(off=FAKE + 2)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    assert c(dt=1, dw=FAKE + 1) == f.FP8Q_EALIGN
    for kw in (dict(dt=1, acc=1), dict(lda=1 << 24), dict(ldb=1 << 24), dict(rows=1 << 31, lda=1 << 32, ldb=1 << 32)):
        assert c(**kw) == f.FP8Q_EUNSUPPORTED, kw
    assert c(N=0) == f.FP8Q_OK and c(K=0) == f.FP8Q_OK
    assert c(rows=0, acc=1, a=0, b=0, off=0, ws=0) == f.FP8Q_OK
    if need:
        assert c(ws=0) == f.FP8Q_EINVAL and c(wsb=need - 1) == f.FP8Q_ESHAPE and c(ws=FAKE + 16) == f.FP8Q_EALIGN


@pytest.mark.parametrize("args", [(-1, 1, 1, 1), (1, 0, 1, 1), (1, 2000, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1), (0, 1, 5, 5),
                                  (5, 1, 0, 5), (1 << 31, 1, 5, 5), (1 << 25, 1, 5, 5)])
def test_no_workspace_for_sizes_that_are_refused(args):
    assert f.fp8q_grouped_wgrad_workspace(*args) == 0


def _adamw(tensor=None, config=None, **kw):
    t = dict(n=256 * 128, p=FAKE, g=FAKE, m=FAKE, v=FAKE, sm=FAKE, sv=FAKE, N=64, K=128, q=FAKE, s=FAKE, qt=FAKE, st=FAKE)
    c = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, lr_dev=None, step_dev=None,
             grad_scale=None, seed=0)
    a = dict(count=1, gt=0, bits=8, mode=0, config_given=True, tensors_given=True)
    t.update(tensor or {})
    c.update(config or {})
    a.update(kw)
    array = (f.fp8q_adamw_tensor * 1)(f.fp8q_adamw_tensor(**t))
    return f.fp8q_adamw(array if a["tensors_given"] else None, a["count"], a["gt"], a["bits"],
                        f.fp8q_adamw_config(**c) if a["config_given"] else None, a["mode"])


def test_adamw():
    assert ctypes.sizeof(f.fp8q_adamw_tensor) == 104 and ctypes.sizeof(f.fp8q_adamw_config) == 80
    for t in (dict(p=0), dict(g=0), dict(m=0), dict(v=0), dict(sm=0), dict(sv=0), dict(s=0), dict(q=0), dict(qt=0),
              dict(st=0), dict(q=0, s=0)):
        assert _adamw(t) == f.FP8Q_EINVAL, t
    for c in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
              dict(beta2=float("nan")), dict(eps=-1e-8), dict(weight_decay=-1.0), dict(step=0), dict(step=-3)):
        assert _adamw(config=c) == f.FP8Q_EINVAL, c
    for kw in (dict(gt=2), dict(bits=16), dict(bits=0), dict(mode=3), dict(config_given=False), dict(tensors_given=False)):
        assert _adamw(**kw) == f.FP8Q_EINVAL, kw
    for t in (dict(n=-1), dict(N=0), dict(K=0), dict(K=64), dict(N=65), dict(n=256 * 128 + 1), dict(K=384),
              dict(N=1 << 40, K=1 << 40), dict(N=-64)):
        assert _adamw(t) == f.FP8Q_ESHAPE, t
    assert _adamw(count=-1) == f.FP8Q_ESHAPE
    for t in (dict(p=FAKE + 4), dict(g=FAKE + 8), dict(m=FAKE + 8), dict(v=FAKE + 1), dict(sm=FAKE + 2), dict(sv=FAKE + 1),
              dict(q=FAKE + 8), dict(s=FAKE + 2), dict(qt=FAKE + 4), dict(st=FAKE + 2)):
        assert _adamw(t) == f.FP8Q_EALIGN, t
    for c in (dict(lr_dev=FAKE + 2), dict(step_dev=FAKE + 4), dict(grad_scale=FAKE + 1)):
        assert _adamw(config=c) == f.FP8Q_EALIGN, c
    assert _adamw(dict(n=(1 << 33) + 8, q=0, s=0, qt=0, st=0)) == f.FP8Q_EUNSUPPORTED
    assert _adamw(dict(n=1 << 31, N=1, K=128)) == f.FP8Q_EUNSUPPORTED  # 2^24 blocks
    assert _adamw(dict(n=0, p=0, g=0)) == f.FP8Q_OK and _adamw(count=0, tensors_given=False) == f.FP8Q_OK


# ------------------------------------------------------------------ helpers

def test_helpers_refuse_host_tensors_and_wrong_kinds():
    off = torch.tensor([0, 4], dtype=torch.int32)
    x = torch.zeros((4, 128))
    with pytest.raises(ValueError, match="HIP device"):
        f.grouped_quantize_act(x, off)
    with pytest.raises(ValueError, match="offsets"):
        f.grouped_quantize_act(x, off.long())
    with pytest.raises(ValueError, match="offsets"):
        f.grouped_quantize_act(x, off[:1])
    with pytest.raises(ValueError, match="offsets"):
        f.grouped_quantize_act(x, torch.zeros(8, dtype=torch.int32)[::2])
    with pytest.raises(ValueError, match="codes"):
        f.grouped_requant_transpose(x, x, off)
    q = torch.zeros((8, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        f.grouped_requant_transpose(q, torch.zeros((1, 4)), off)
    o = f.GroupedOperand(q, torch.zeros((1, 8)), 4)
    for bad, text in (((o, o._replace(rows=5)), "rows"), ((o._replace(rows=129), o._replace(rows=129)), "tokens"),
                      ((o._replace(s=torch.zeros((1, 7))), o), "scales"), ((o._replace(q=q.float()), o), "codes")):
        with pytest.raises(ValueError, match=text):
            f.grouped_wgrad(*bad, off)
    with pytest.raises(ValueError, match="accumulate"):
        f.grouped_wgrad(o, o, off, accumulate=True)
    with pytest.raises(ValueError, match="dw"):
        f.grouped_wgrad(o, o, off, dw=torch.zeros((1, 8, 9)))
    with pytest.raises(ValueError, match="HIP device"):
        f.grouped_wgrad(o, o, off)


def test_adamw_tensors_refuses():
    p = torch.zeros((2, 128))
    st = f.adamw_state(p)
    with pytest.raises(ValueError, match="no tensors"):
        f.adamw_tensors([], [], [])
    with pytest.raises(ValueError, match="1 params"):
        f.adamw_tensors([p], [], [st])
    for bad, text in (((p.double(), p, st), "parameter"), ((p.t(), p, st), "parameter"), ((p, p[:1], st), "gradient"),
                      ((p, p.half(), st), "HIP device"), ((p, p, st._replace(m=st.m[:5])), "m is"),
                      ((p, p, st._replace(sm=st.m)), "no scales"), ((p, p, f.adamw_state(p, 8)._replace(sv=None)), "scales"),
                      ((p, p.clone(), st), "HIP device")):
        with pytest.raises(ValueError, match=text):
            f.adamw_tensors(*([v] for v in bad))
    with pytest.raises(ValueError, match="bits"):
        f.adamw_state(p, 16)
    with pytest.raises(ValueError, match="multiple of 128"):
        f.weight_codes(torch.zeros((4, 100)))
    with pytest.raises(ValueError, match="HIP device"):
        f.weight_codes(p)


def test_overlap_check():
    from fp8_fine_grained_x128_amd.binding import _no_overlap

    def spans(written, read):
        return [(a, b, True) for a, b in written] + [(a, b, False) for a, b in read]

    _no_overlap("x", spans([(0, 128), (128, 256), (300, 300)], [(256, 300)]))
    _no_overlap("x", spans([(0, 128)], [(200, 300), (200, 300), (250, 400)]))  # gradients may be shared
    for w, r in (([(0, 64), (0, 64)], []), ([(0, 132), (128, 256)], []), ([(0, 64)], [(0, 64)]), ([(32, 64)], [(0, 128)]),
                 ([(0, 128)], [(32, 64)]), ([(40, 48), (16, 32), (24, 36)], []), ([(10, 20)], [(0, 100), (50, 60)])):
        with pytest.raises(ValueError, match="overlap"):
            _no_overlap("x", spans(w, r))
