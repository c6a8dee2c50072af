"""What the feed-forward operators refuse: the C entry points' status for each
kind of invalid argument (nothing is launched, so no GPU is needed), and the
tensor helpers' own checks."""
import os
import subprocess

import pytest
import torch

import fp8_fine_grained_x128_amd as f

FAKE = 1 << 20  # an aligned, never-dereferenced address
INF = float("inf")


def _caller(fn, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return fn(*{**ok, **kw}.values())
    return call


def test_layernorm():
    c = _caller(f.fp8q_layernorm, dict(
        x=FAKE, xt=1, rows=4, cols=256, ldx=256, gamma=FAKE, beta=0, wt=0, eps=1e-5, kind=0, y=FAKE, yt=0, ldy=256,
        q=FAKE, ldq=256, s=FAKE, lds=4, mode=0, mean=FAKE, rstd=FAKE))
    for kw in (dict(xt=2), dict(wt=7), dict(yt=2), dict(kind=2), dict(mode=2), dict(eps=-1.0), dict(eps=float("nan")),
               dict(x=0), dict(y=0, q=0, s=0), dict(q=0), dict(s=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-1), dict(cols=-1), dict(ldx=255), dict(ldy=255), dict(ldq=255), dict(lds=3), dict(ldx=1 << 33)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(ldx=260), dict(y=FAKE + 4), dict(ldy=258), dict(q=FAKE + 8), dict(ldq=264),
               dict(s=FAKE + 2), dict(gamma=FAKE + 4), dict(beta=FAKE + 8), dict(mean=FAKE + 1), dict(rstd=FAKE + 2)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    wide = f.NORM_MAX_COLS + 8
    assert c(cols=wide, ldx=wide, ldy=wide, q=0, s=0) == f.FP8Q_EUNSUPPORTED
    assert c(rows=0, x=0) == f.FP8Q_OK and c(cols=0, x=0, y=0, q=0, s=0) == f.FP8Q_OK


def test_layernorm_backward():
    need = f.fp8q_layernorm_backward_workspace(4, 256)
    assert need > 0 and f.fp8q_layernorm_backward_workspace(0, 256) == 0
    assert f.fp8q_layernorm_backward_workspace(4, f.NORM_MAX_COLS + 1) == 0
    c = _caller(f.fp8q_layernorm_backward, dict(
        dy=FAKE, lddy=256, x=FAKE, ldx=256, t=1, rows=4, cols=256, gamma=FAKE, wt=0, mean=FAKE, rstd=FAKE, kind=0,
        skip=FAKE, ldskip=256, dx=FAKE, lddx=256, dgamma=FAKE, dbeta=FAKE, acc=0, ws=FAKE, wsb=need))
    for kw in (dict(t=3), dict(wt=-1), dict(kind=5), dict(dy=0), dict(x=0), dict(mean=0), dict(rstd=0), dict(dx=0),
               dict(ws=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-2), dict(lddy=8), dict(ldx=0), dict(lddx=255), dict(ldskip=100), dict(wsb=need - 1),
               dict(wsb=-1)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(dy=FAKE + 2), dict(lddy=257), dict(x=FAKE + 8), dict(dx=FAKE + 4), dict(skip=FAKE + 2),
               dict(gamma=FAKE + 8), dict(dgamma=FAKE + 2), dict(ws=FAKE + 16), dict(rstd=FAKE + 2)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    wide = f.NORM_MAX_COLS + 8
    assert c(cols=wide, lddy=wide, ldx=wide, lddx=wide, ldskip=wide) == f.FP8Q_EUNSUPPORTED
    assert c(rows=0, acc=1) == f.FP8Q_OK and c(cols=0) == f.FP8Q_OK
    assert c(rows=0, dgamma=0, dbeta=0) == f.FP8Q_OK


def test_swiglu_quantize():
    c = _caller(f.fp8q_swiglu_quantize, dict(
        g=FAKE, u=FAKE, t=1, ldgu=256, rows=4, cols=256, qh=FAKE, ldqh=256, sh=FAKE, ldsh=4, qg=FAKE, qu=FAKE, ldq=256,
        sg=FAKE, su=FAKE, lds=4, mode=0))
    for kw in (dict(t=2), dict(mode=3), dict(g=0), dict(u=0), dict(qh=0), dict(sh=0), dict(qg=0), dict(su=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(rows=-1), dict(ldgu=128), dict(ldqh=255), dict(ldsh=3), dict(ldq=0), dict(lds=1)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(g=FAKE + 8), dict(u=FAKE + 2), dict(ldgu=257), dict(qh=FAKE + 4), dict(ldqh=264), dict(sh=FAKE + 1),
               dict(qu=FAKE + 8), dict(ldq=260), dict(sg=FAKE + 2)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    assert c(rows=0, g=0) == f.FP8Q_OK


IN = dict(qg=FAKE, qu=FAKE, ldq=256, sg=FAKE, su=FAKE, lds=4, dh=FAKE, t=1, lddh=256, rows=4, cols=256)
IN_BAD = [(dict(t=9), 1), (dict(qg=0), 1), (dict(dh=0), 1), (dict(su=0), 1), (dict(rows=-1), 2), (dict(ldq=255), 2),
          (dict(lds=3), 2), (dict(lddh=1), 2), (dict(qu=FAKE + 8), 3), (dict(ldq=264), 3), (dict(sg=FAKE + 2), 3),
          (dict(dh=FAKE + 4), 3), (dict(lddh=257), 3)]


def test_swiglu_backward():
    c = _caller(f.fp8q_swiglu_backward, dict(**IN, dg=FAKE, du=FAKE, ldd=256))
    for kw, status in IN_BAD + [(dict(dg=0), 1), (dict(ldd=255), 2), (dict(du=FAKE + 8), 3), (dict(ldd=260), 3)]:
        assert c(**kw) == status, kw
    assert c(cols=0) == f.FP8Q_OK


def test_swiglu_backward_quantize():
    c = _caller(f.fp8q_swiglu_backward_quantize, dict(
        **IN, qdg=FAKE, qdu=FAKE, ldqd=256, sdg=FAKE, sdu=FAKE, ldsd=4, qdgt=FAKE, qdut=FAKE, ldqt=16, sdgt=FAKE,
        sdut=FAKE, ldst=256, qht=FAKE, ldqht=16, sht=FAKE, ldsht=256, mode=0))
    more = [(dict(mode=2), 1), (dict(qdg=0), 1), (dict(sdut=0), 1), (dict(qht=0), 1), (dict(ldqd=255), 2),
            (dict(ldsd=3), 2), (dict(ldqt=3), 2), (dict(ldst=255), 2), (dict(ldqht=0), 2), (dict(ldsht=255), 2),
            (dict(qdut=FAKE + 8), 3), (dict(ldqt=24), 3), (dict(ldqht=8), 3), (dict(sht=FAKE + 2), 3)]
    for kw, status in IN_BAD + more:
        assert c(**kw) == status, kw
    assert c(rows=65536 * 128, lds=1 << 23, ldsd=1 << 23, ldqt=1 << 23, ldqht=1 << 23) == f.FP8Q_EUNSUPPORTED
    wide = dict(ldq=1 << 30, lddh=1 << 30, ldqd=1 << 30, ldst=1 << 30, ldsht=1 << 30)
    assert c(cols=1 << 30, **wide) == f.FP8Q_EUNSUPPORTED
    assert c(rows=0) == f.FP8Q_OK


def test_moe_decode():
    size = f.fp8q_moe_decode_workspace
    need = size(4, 256, 128, 8, 2)
    assert need > 0
    for bad in ((0, 256, 128, 8, 2), (65, 256, 128, 8, 2), (4, 200, 128, 8, 2), (4, 256, 100, 8, 2), (4, 256, 128, 0, 2),
                (4, 256, 128, 8, 0), (4, 256, 128, 1025, 2), (4, 256, 128, 64, 33)):
        assert size(*bad) == 0, bad
    c = _caller(f.fp8q_moe_decode, dict(
        x=FAKE, ldx=256, T=4, H=256, logits=FAKE, ldl=8, E=8, k=2, renorm=1, I=128, w=FAKE, ldw=256, ws=256 * 256,
        s=FAKE, lds=2, ss=4, d=FAKE, ldd=128, ds=256 * 128, sd=FAKE, ldsd=1, sds=2, y=FAKE, yt=1, ldy=256, work=FAKE,
        wb=need))
    for kw in (dict(yt=4), dict(x=0), dict(logits=0), dict(w=0), dict(s=0), dict(d=0), dict(sd=0), dict(y=0), dict(work=0)):
        assert c(**kw) == f.FP8Q_EINVAL, kw
    for kw in (dict(T=-1), dict(H=200), dict(I=0), dict(E=0), dict(k=0), dict(ldx=255), dict(ldl=7), dict(ldy=255),
               dict(ldw=128), dict(ws=256 * 256 - 16), dict(lds=1), dict(ss=3), dict(ldd=64), dict(ds=0), dict(sds=1),
               dict(wb=need - 1), dict(wb=-1)):
        assert c(**kw) == f.FP8Q_ESHAPE, kw
    for kw in (dict(T=65), dict(E=1025, ldl=1025), dict(k=33), dict(ldw=1 << 24, ws=1 << 40)):
        assert c(**kw) == f.FP8Q_EUNSUPPORTED, kw
    for kw in (dict(x=FAKE + 8), dict(ldx=257), dict(logits=FAKE + 2), dict(w=FAKE + 8), dict(ldw=264, ws=1 << 20),
               dict(ws=256 * 256 + 8), dict(s=FAKE + 1), dict(y=FAKE + 4), dict(ldy=257), dict(work=FAKE + 128)):
        assert c(**kw) == f.FP8Q_EALIGN, kw
    assert c(T=0, x=0, w=0) == f.FP8Q_OK


def test_helpers():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    v = torch.ones(256)
    with pytest.raises(ValueError, match="HIP device"):
        f.layernorm(x)
    with pytest.raises(ValueError, match="nothing to compute"):
        f.layernorm(x, quantize=False)
    with pytest.raises(ValueError, match="gamma"):
        f.layernorm(x, v[:255])
    with pytest.raises(ValueError, match="beta"):
        f.layernorm(x, v, v.bfloat16())
    r = torch.ones(4)
    with pytest.raises(ValueError, match="dy"):
        f.layernorm_backward(x.float(), x, v, r, r)
    with pytest.raises(ValueError, match="skip"):
        f.layernorm_backward(x, x, v, r, r, skip=x[:2])
    with pytest.raises(ValueError, match="mean"):
        f.layernorm_backward(x, x, v, None, r)
    with pytest.raises(ValueError, match="rstd"):
        f.layernorm_backward(x, x, v, r, r[:3])
    with pytest.raises(ValueError, match="accumulate"):
        f.layernorm_backward(x, x, v, r, r, accumulate=True)
    with pytest.raises(ValueError, match="dgamma"):
        f.layernorm_backward(x, x, v, r, r, dgamma=v.double())
    with pytest.raises(ValueError, match="u is"):
        f.swiglu_quantize(x, x.float())
    with pytest.raises(ValueError, match="strides"):
        f.swiglu_quantize(x, torch.zeros((4, 512), dtype=torch.bfloat16)[:, :256])
    with pytest.raises(ValueError, match="HIP device"):
        f.swiglu_quantize(x, x)
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 4))
    for bad in (f.SwigluCheckpoint(q, q[:, :128], s, s), f.SwigluCheckpoint(q, q, s.t(), s),
                f.SwigluCheckpoint(q, q.float(), s, s)):
        for call in (f.swiglu_backward, f.swiglu_backward_quantize):
            with pytest.raises(ValueError):
                call(bad, x)
    with pytest.raises(ValueError, match="HIP device"):
        f.swiglu_backward(f.SwigluCheckpoint(q, q, s, s), x)
    l = torch.zeros((4, 8))
    w, ws = torch.zeros((8, 256, 256), dtype=torch.uint8), torch.zeros((8, 2, 2))
    d, ds = torch.zeros((8, 256, 128), dtype=torch.uint8), torch.zeros((8, 2, 1))
    for args, text in (((x.float(), l, w, ws, d, ds), "bfloat16"), ((x, l.double(), w, ws, d, ds), "float32"),
                       ((x, l[:3], w, ws, d, ds), "logits"), ((x, l, w[:, :128], ws, d, ds), "w_gu"),
                       ((x, l, w, ws[:, :1], d, ds), "w_gu"), ((x, l, w, ws, d[:7], ds), "w_down"),
                       ((x, l, w, ws, d, ds.double()), "w_down"), ((x, l, w, ws, d[0], ds), "w_down"),
                       ((x, l, w.transpose(1, 2), ws, d, ds), "unit inner"), ((x, l, w, ws, d, ds), "HIP device")):
        with pytest.raises(ValueError, match=text):
            f.moe_decode(*args, 2)


def test_checks_under_host_sanitizers(tmp_path):
    """The argument checks on boundary values (negative, zero, odd, huge) with the address and undefined-behaviour
    sanitizers."""
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
    exe = str(tmp_path / "feed_forward_validate")
    subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1", "-std=c++17",
                    "-Wall", "-Werror", os.path.join(here, "feed_forward_validate.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
