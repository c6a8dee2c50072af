"""The experts' operators together: the example's training step against the same step in fp32, replayed from a graph,
and calls on several streams at once."""
import importlib.util
import itertools
import os

import numpy as np
import pytest
import torch

from tests import expert_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example(fp8q):
    spec = importlib.util.spec_from_file_location("expert_training", os.path.join(ROOT, "examples", "expert_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _weights(c):
    q = c.q.view(torch.float8_e4m3fn).float()
    return q * c.s.repeat_interleave(128, 1)[:, : q.shape[1]].repeat_interleave(128, 2)[:, :, : q.shape[2]]


def test_training_step(example, fp8q):
    """E4M3 rounds a number by 2.6 % of itself in the mean over a binade and a gradient here passes at most six
    roundings (dy, g, u, the gradient of the SwiGLU, and the activations twice): 6.4 % if they are independent.  Twice
    that is allowed.  The optimizer's step is then exact for the gradients it was given."""
    T, E, H, I = 300, 6, 256, 128
    e = example.make_experts(E, H, I, bits=8, seed=1)
    torch.manual_seed(2)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    chosen = torch.rand((T, E - 1), device=DEV).topk(2).indices  # the last expert has no rows
    rows, offsets = example.route(chosen, E)
    assert offsets.tolist()[-1] == 2 * T and offsets[-2] == offsets[-1]
    dy = (torch.randn((2 * T, H), device=DEV) * 1e-3).to(torch.bfloat16)
    y, saved = example.forward(x, rows, offsets, e)
    dx = example.backward(dy, saved, offsets, e)

    xr = x.float()[rows.long()].clone().requires_grad_()
    w_gu, w_down = _weights(e.c_gu).requires_grad_(), _weights(e.c_down).requires_grad_()
    off = offsets.tolist()
    out = []
    for g in range(E):
        gu = xr[off[g]: off[g + 1]] @ w_gu[g].t()
        out.append((torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ w_down[g].t())
    want = torch.cat(out)
    want.backward(dy.float())

    def far(a, w):
        return ((a.float() - w).norm() / w.norm()).item()

    for name, a, w in (("y", y, want), ("dx", dx, xr.grad), ("w_gu", e.g_gu, w_gu.grad), ("w_down", e.g_down, w_down.grad)):
        assert far(a, w) < 0.13, (name, far(a, w))
    assert not e.g_gu[-1].any() and not e.g_down[-1].any()

    before = [(p.double().cpu().numpy().reshape(-1), g.double().cpu().numpy().reshape(-1)) for p, g in
              ((e.w_gu, e.g_gu), (e.w_down, e.g_down))]
    fp8q.adamw(e.optimizer, step=1, lr=1e-2, seed=5)
    for (p, g), w, c in zip(before, (e.w_gu, e.w_down), (e.c_gu, e.c_down)):
        zero = np.zeros_like(p)
        p1, _, _, ep, _, _ = R.adamw(p, g, zero, zero, 1e-2, 0.9, 0.95, 1e-8, 0.1, 1)
        assert (np.abs(w.double().cpu().numpy().reshape(-1) - p1) <= ep).all()
        for k in range(E):
            q, s = fp8q.quantize_weight(w[k])
            qt, st = fp8q.transpose_weight(q, s)
            assert torch.equal(c.q[k], q) and torch.equal(c.s[k], s) and torch.equal(c.qt[k], qt) and torch.equal(c.st[k], st)


def test_gradients_add_up(example):
    """Two halves of the rows added one after the other are all rows, within the sums' rounding and what the tiles'
    other borders change (a chunk of other tokens has another scale: at most half an E4M3 step each, 2^-4)."""
    T, E, H, I = 256, 4, 256, 128
    e = example.make_experts(E, H, I, seed=3)
    torch.manual_seed(4)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    chosen = torch.rand((T, E), device=DEV).topk(1).indices
    grads = []
    for parts in ([slice(0, T)], [slice(0, 100), slice(100, T)]):
        for k, part in enumerate(parts):
            rows, offsets = example.route(chosen[part], E)
            y, saved = example.forward(x[part], rows, offsets, e)
            example.backward(torch.ones_like(y) * 1e-3, saved, offsets, e, accumulate=k > 0)
        grads.append((e.g_gu.clone(), e.g_down.clone()))
    for a, b in zip(*grads):
        assert (a - b).norm() <= 2 * 2.0 ** -4 * a.norm()


def test_captured_training_step(example, fp8q):
    """Forward, backward and the optimizer in one graph, replayed with eager work and other values between, against
    the same steps run eagerly, bit for bit."""
    T, E, H, I = 200, 4, 256, 128
    a, b = (example.make_experts(E, H, I, bits=8, seed=6) for _ in range(2))
    x = torch.zeros((T, H), device=DEV, dtype=torch.bfloat16)
    dy = torch.zeros((T, H), device=DEV, dtype=torch.bfloat16)
    rows = torch.zeros(T, device=DEV, dtype=torch.int32)
    offsets = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
    step = torch.zeros((), device=DEV, dtype=torch.int64)

    def run(e):
        y, saved = example.forward(x, rows, offsets, e)
        dx = example.backward(dy, saved, offsets, e)
        fp8q.adamw(e.optimizer, step=step, lr=1e-2, seed=9)
        return y, dx

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(a)
    for k in range(1, 5):
        torch.manual_seed(k)
        x.copy_(torch.randn((T, H), device=DEV))
        dy.copy_(torch.randn((T, H), device=DEV) * 1e-3)
        r, o = example.route(torch.randint(0, 1 + k % E, (T, 1), device=DEV), E)  # sizes change, experts without rows too
        rows.copy_(r)
        offsets.copy_(o)
        step.fill_(k)
        graph.replay()
        want = run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        for g, w in zip((a.w_gu, a.w_down, a.g_gu, a.g_down, *a.c_gu, *a.c_down), (b.w_gu, b.w_down, b.g_gu, b.g_down, *b.c_gu, *b.c_down)):
            assert torch.equal(g, w)


def test_captured_split_gradients_with_workspaces_of_their_own(fp8q):
    """Two graphs of split contractions and eager calls between them."""
    off = torch.tensor([0, 3000, 5000], dtype=torch.int32, device=DEV)
    torch.manual_seed(1)
    dy, x = torch.randn((5000, 128), device=DEV) * 1e-3, torch.randn((5000, 256), device=DEV)
    a, b = fp8q.grouped_quantize_act(dy, off), fp8q.grouped_quantize_act(x, off)
    assert fp8q.fp8q_grouped_wgrad_workspace(5000, 2, 128, 256) > 0
    want = fp8q.grouped_wgrad(a, b, off)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fp8q.grouped_wgrad(a, b, off))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        other = fp8q.grouped_wgrad(a, b, off, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        assert (other.float() - want).abs().max() <= 2.0 ** -8 * want.abs().max()


def test_workspace_of_exactly_the_bytes(fp8q):
    """The split writes nothing before or behind its workspace, whatever the groups' sizes."""
    rows, N, K = 6000, 130, 200
    for off in ([0, 6000, 6000, 6000], [0, 2000, 4000, 6000], [0, 640, 1281, 6000], [0, 1, 2, 3]):
        need = fp8q.fp8q_grouped_wgrad_workspace(rows, 3, N, K)
        assert need > 0
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        torch.manual_seed(2)
        a = fp8q.grouped_quantize_act(torch.randn((rows, N), device=DEV)[:, :N].contiguous() if N % 4 == 0 else
                                      torch.randn((rows, 132), device=DEV)[:, :N], o)
        b = fp8q.grouped_quantize_act(torch.randn((rows, K), device=DEV), o)
        want = fp8q.grouped_wgrad(a, b, o)
        buf = torch.full((need + 512,), 0x77, dtype=torch.uint8, device=DEV)
        base = (buf.data_ptr() + 255) // 256 * 256
        lead = base - buf.data_ptr()
        dw = torch.empty((3, N, K), device=DEV)
        st = fp8q.fp8q_grouped_wgrad(a.q.data_ptr(), a.q.shape[1], a.s.data_ptr(), N, b.q.data_ptr(), b.q.shape[1],
                                     b.s.data_ptr(), K, o.data_ptr(), 3, rows, N, K, dw.data_ptr(), 0, K, N * K, 0, 0, base,
                                     need, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(dw, want)
        assert (buf[:lead] == 0x77).all() and (buf[lead + need:] == 0x77).all()


@pytest.mark.parametrize("sizes", [[768] * 8, [641] * 8, [640] * 8, [641, 1, 1, 1, 4481, 1, 1, 1], [5000] + [1] * 7])
def test_most_slices_fit_the_workspace(fp8q, sizes):
    """Groups of one and a half slices, or just more or less, are cut into the most slices for their rows."""
    rows, G, N, K = sum(sizes), len(sizes), 70, 128
    need = fp8q.fp8q_grouped_wgrad_workspace(rows, G, N, K)
    assert need > 0
    o = torch.tensor([0, *itertools.accumulate(sizes)], dtype=torch.int32, device=DEV)
    torch.manual_seed(4)
    a = fp8q.grouped_quantize_act(torch.randn((rows, 72), device=DEV)[:, :N], o)
    b = fp8q.grouped_quantize_act(torch.randn((rows, K), device=DEV), o)
    dw = torch.empty((G, N, K), device=DEV)
    buf = torch.full((need + 512,), 0x77, dtype=torch.uint8, device=DEV)
    lead = -buf.data_ptr() % 256
    assert fp8q.fp8q_grouped_wgrad(a.q.data_ptr(), a.q.shape[1], a.s.data_ptr(), N, b.q.data_ptr(), b.q.shape[1],
                                   b.s.data_ptr(), K, o.data_ptr(), G, rows, N, K, dw.data_ptr(), 0, K, N * K, 0, 0,
                                   buf.data_ptr() + lead, need, torch.cuda.current_stream().cuda_stream) == 0
    assert (buf[:lead] == 0x77).all() and (buf[lead + need:] == 0x77).all()
    want, t = R.wgrad(*(v.cpu().numpy() for v in (a.q, a.s, b.q, b.s)), o.cpu().numpy())
    assert (np.abs(dw.cpu().numpy() - want) <= 1e-5 * t).all()


def test_two_streams_at_once(fp8q):
    """The same operands read by calls on two streams; each call has its own workspace and output."""
    off = torch.tensor([0, 1000, 2600, 4096], dtype=torch.int32, device=DEV)
    torch.manual_seed(3)
    x, dy = torch.randn((4096, 384), device=DEV).to(torch.bfloat16), torch.randn((4096, 256), device=DEV).to(torch.bfloat16)
    want = fp8q.grouped_wgrad(fp8q.grouped_quantize_act(dy, off), fp8q.grouped_quantize_act(x, off), off)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(fp8q.grouped_wgrad(fp8q.grouped_quantize_act(dy, off), fp8q.grouped_quantize_act(x, off), off))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
