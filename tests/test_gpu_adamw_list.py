"""A kept list of tensors whose parameters get other memory."""
import pytest
import torch

from tests.test_gpu_adamw import DEV, H, _tensor, _Want

pytestmark = pytest.mark.gpu


def test_replaced_parameter_is_refused(fp8q):
    p, g = _tensor((300,), torch.float32, 71)
    q, h = _tensor((4, 128), torch.float32, 72)
    p, q = torch.nn.Parameter(p), torch.nn.Parameter(q)
    sts = [fp8q.adamw_state(t) for t in (p, q)]
    plan = fp8q.adamw_tensors([p, q], [g, h], sts)
    fp8q.adamw(plan, step=1, **H)
    old, before = q.data, p.detach().clone()
    q.data = q.data.clone()
    with pytest.raises(ValueError, match="parameter 1 has other memory"):
        fp8q.adamw(plan, step=2, **H)
    torch.cuda.synchronize()
    assert torch.equal(p, before) and torch.equal(q, old)  # nothing ran
    fresh = fp8q.adamw_tensors([p, q], [g, h], sts)
    want = _Want(q.detach(), h, sts[1], 2)
    fp8q.adamw(fresh, step=2, **H)
    want.check(q.detach(), sts[1])
    q.data = old
    with pytest.raises(ValueError, match="parameter 1"):
        fp8q.adamw(fresh, step=3, **H)


def test_memory_given_up_is_not_written(fp8q):
    """A gradient and a moment whose tensors were given other memory: the step goes on in what the list was made of, which
    nobody else has got meanwhile."""
    n = 1 << 20
    p, g = torch.zeros(n, device=DEV), torch.ones(n, device=DEV)
    st = fp8q.adamw_state(p)
    plan = fp8q.adamw_tensors([p], [g], [st])
    for t in (g, st.m, st.v):
        t.data = torch.empty(0, device=DEV)
    others = [torch.full((n,), 5.0, device=DEV) for _ in range(8)]
    fp8q.adamw(plan, step=1, lr=1e-2, weight_decay=0.0)
    torch.cuda.synchronize()
    assert all((o == 5.0).all() for o in others)
    assert ((p + 1e-2).abs() <= 1e-7).all()


def test_backward_through_changed_weights_is_refused(fp8q):
    """As after any change in place: a graph that kept a parameter, or its codes, does not go on with other values."""
    w = torch.nn.Parameter(torch.randn((16, 128), device=DEV))
    c, st = fp8q.weight_codes(w.detach()), fp8q.adamw_state(w)
    plan = fp8q.adamw_tensors([w], [torch.ones((16, 128), device=DEV)], [st], [c])

    class ByCodes(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            ctx.save_for_backward(c.q, c.st)
            return x * 2

        @staticmethod
        def backward(ctx, dy):
            return dy * ctx.saved_tensors[0].float().mean()

    x = torch.randn((4, 128), device=DEV, requires_grad=True)
    for graph in (lambda: (x @ w.t()).sum(), lambda: ByCodes.apply(x).sum()):
        graph().backward()
        loss = graph()
        fp8q.adamw(plan, step=1, **H)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        graph().backward()


def test_inference_tensors(fp8q):
    """They have no version counter; the step takes them."""
    with torch.inference_mode():
        p = torch.ones((2, 128), device=DEV)
        st, c = fp8q.adamw_state(p), fp8q.weight_codes(p)
        plan = fp8q.adamw_tensors([p], [torch.ones_like(p)], [st], [c])
        fp8q.adamw(plan, step=1, lr=0.5, weight_decay=0.5)
    assert (p < 0.5).all()
    fp8q.adamw(plan, step=2, lr=0.5)
