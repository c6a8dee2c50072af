"""The feed-forward operators together: the example's training step against
the same step in fp32 with the dequantized weights, its decode step, and all
operators under HIP graph capture."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(fp8q):
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _weight(q, s):
    """fp32 values of codes [N][K] with 128x128 scales"""
    return q.contiguous().view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def _norm(x, gamma, beta):
    m = x.mean(1, keepdim=True) if beta is not None else 0.0
    y = (x - m) * ((x - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * gamma
    return y if beta is None else y + beta


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_training_step(example, rms):
    """E4M3 rounds a number by at most 2^-4 of itself, 2.6 % in the mean over a binade; a gradient here passes at most
    six roundings one after the other or side by side (dy, g, u, the gradient of the SwiGLU and the activations twice),
    6.4 % if they are independent.  Twice that is allowed."""
    say(f"feed-forward training step rms={rms}")
    M, H, I = 384, 512, 256
    b = example.make_block(H, I, rms=rms, seed=3)
    torch.manual_seed(0)
    x = torch.randn((M, H), device="cuda").to(torch.bfloat16)
    dy = (torch.randn((M, H), device="cuda") * 1e-3).to(torch.bfloat16)
    y, saved = example.forward(x, b)
    g = example.backward(dy, saved, b)

    leaves = [t.clone().requires_grad_() for t in (x.float(), b.gamma, _weight(b.w_gu, b.s_gu),
                                                   _weight(b.w_down, b.s_down))]
    beta = None if rms else b.beta.clone().requires_grad_()
    gu = _norm(leaves[0], leaves[1], beta) @ leaves[2].t()
    want = leaves[0] + (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ leaves[3].t()
    want.backward(dy.float())

    def off(a, w):
        return ((a.float() - w).norm() / w.norm()).item()

    assert off(y - x, want - x.float()) < 0.13
    for name, a, w in (("x", g.x - dy, leaves[0].grad - dy.float()), ("gamma", g.gamma, leaves[1].grad),
                       ("w_gu", g.w_gu, leaves[2].grad), ("w_down", g.w_down, leaves[3].grad)):
        e = off(a, w)
        say(f"  d{name}: {e:.4f}")
        assert e < 0.13, name
    assert (g.beta is None) == rms
    if not rms:
        assert off(g.beta, beta.grad) < 0.13


def test_decode_step(example, fp8q):
    say("feed-forward decode step")
    H, I, E, k = 512, 256, 16, 4
    b = example.make_block(H, I, experts=E, rms=True, seed=5)
    router = (torch.randn((E, H), device="cuda") * H ** -0.5).to(torch.bfloat16)
    x = torch.randn((3, H), device="cuda").to(torch.bfloat16)
    y = example.decode(x, router, b, k)
    n = fp8q.layernorm(x, b.gamma, kind=b.kind, quantize=False, out_dtype=torch.bfloat16).y
    logits = (n @ router.t()).float()
    want, err = R.moe(R.f64(n), R.f64(logits), b.w_gu, b.s_gu, b.w_down, b.s_down, k, True)
    # the layer's bf16 rounding, then the residual's
    err = err + R.bf16_half_ulp(np.abs(want) + err)
    R.assert_close(y, want + R.f64(x), err, "decode")


def test_graph_replays_match_eager(fp8q):
    """All feed-forward operators in one graph; four replays on new inputs, with eager work between them, equal the
    eager results bit for bit."""
    say("feed-forward operators under graph capture")
    M, N, T, E, H, I = 300, 640, 5, 24, 256, 128
    dev = "cuda"
    x, dy, g, u, dh = (torch.empty((M, N), dtype=torch.bfloat16, device=dev) for _ in range(5))
    gamma, beta = torch.empty(N, device=dev), torch.empty(N, device=dev)
    xt, logits = torch.empty((T, H), dtype=torch.bfloat16, device=dev), torch.empty((T, E), device=dev)
    xb, logits_b = torch.empty((40, H), dtype=torch.bfloat16, device=dev), torch.empty((40, E), device=dev)
    w = torch.randint(0, 0x7f, (E, 2 * I, H), dtype=torch.uint8, device=dev)
    d = torch.randint(0, 0x7f, (E, H, I), dtype=torch.uint8, device=dev)
    sw, sd = torch.rand((E, 2 * I // 128, H // 128), device=dev) * 1e-4, torch.rand((E, H // 128, 1), device=dev) * 1e-4
    dgamma, dbeta = torch.zeros(N, device=dev), torch.zeros(N, device=dev)

    def fill(seed):
        torch.manual_seed(seed)
        for t in (x, dy, g, u, dh, gamma, beta, xt, logits, xb, logits_b):
            t.copy_(torch.randn(t.shape, device=dev))
        logits[1] = -float("inf")
        dgamma.zero_()
        dbeta.zero_()

    def step():
        n = fp8q.layernorm(x, gamma, beta, out_dtype=torch.bfloat16)
        r = fp8q.layernorm(x, gamma, kind=fp8q.FP8Q_NORM_RMS, scale_mode=fp8q.FP8Q_SCALE_POW2)
        b1 = fp8q.layernorm_backward(dy, x, gamma, n.mean, n.rstd, skip=dh)
        b2 = fp8q.layernorm_backward(dy, x, gamma, None, r.rstd, kind=fp8q.FP8Q_NORM_RMS)
        fp8q.layernorm_backward(dy, x, gamma, n.mean, n.rstd, dgamma=dgamma, dbeta=dbeta, accumulate=True)
        qh, sh, kept = fp8q.swiglu_quantize(g, u)
        p = fp8q.swiglu_backward(kept, dh)
        o = fp8q.swiglu_backward_quantize(kept, dh)
        y = fp8q.moe_decode(xt, logits, w, sw, d, sd, 3)
        z = fp8q.moe_decode(xb, logits_b, w, sw, d, sd, 3, renormalize=False)
        return [*n, r.q, r.s, r.rstd, *b1, *b2[:2], qh, sh, *kept, *p, *o, y, z, dgamma.clone(), dbeta.clone()]

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    fill(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    torch.cuda.synchronize()
    for rep in range(4):
        fill(rep)
        want = [t.clone() for t in step()]
        fill(rep)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), (rep, i)


def test_calls_follow_the_current_stream(fp8q):
    """Work queued behind a long kernel on a side stream sees that kernel's results."""
    say("feed-forward operators on a side stream")
    x = torch.zeros((512, 1024), dtype=torch.bfloat16, device="cuda")
    src = torch.randn((512, 1024), device="cuda").to(torch.bfloat16)
    big = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    want = fp8q.layernorm(src, out_dtype=torch.bfloat16).y, fp8q.swiglu_quantize(src, src)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            big = big @ big * 1e-4
        x.copy_(src)
        got = fp8q.layernorm(x, out_dtype=torch.bfloat16).y, fp8q.swiglu_quantize(x, x)[0]
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
