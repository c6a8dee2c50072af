"""A mixture-of-experts feed-forward layer in FP8: one training step, from the
routed tokens to the experts' new weights.

    python examples/expert_training.py [tokens experts hidden inner]

Forward: the tokens' rows are gathered expert by expert in FP8, gate|up GEMM,
SwiGLU, down GEMM per expert.  Backward: the gradient of the rows through the
transposed codes, and every expert's weight gradients over its own rows (their
operands in 128-token tiles that do not cross experts).  The optimizer step then
writes the new weights' codes, which the next step's GEMMs read: the fp32
master weights are read and written by nothing else.
"""
from __future__ import annotations

import os
import sys
from typing import NamedTuple, Tuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_x128_amd as fp8q  # noqa: E402


class Experts(NamedTuple):
    w_gu: torch.Tensor                  # fp32 [experts][2*inner][hidden], gate rows first
    w_down: torch.Tensor                # fp32 [experts][hidden][inner]
    c_gu: fp8q.WeightCodes
    c_down: fp8q.WeightCodes
    g_gu: torch.Tensor                  # gradients of the master weights
    g_down: torch.Tensor
    optimizer: fp8q.AdamwTensors


class Saved(NamedTuple):
    qx: torch.Tensor
    sx: torch.Tensor
    qh: torch.Tensor
    sh: torch.Tensor
    kept: fp8q.SwigluCheckpoint


def make_experts(experts: int, hidden: int, inner: int, bits: int = 8, seed: int = 0) -> Experts:
    g = torch.Generator(device="cuda").manual_seed(seed)
    weights = [torch.randn(s, generator=g, device="cuda") * 0.02
               for s in ((experts, 2 * inner, hidden), (experts, hidden, inner))]
    codes = [fp8q.weight_codes(w) for w in weights]
    grads = [torch.zeros_like(w) for w in weights]
    optimizer = fp8q.adamw_tensors(weights, grads, [fp8q.adamw_state(w, bits) for w in weights], codes)
    return Experts(*weights, *codes, *grads, optimizer)


def route(experts: torch.Tensor, count: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """(token of every row, first row of every expert) for the expert of each pair [tokens][top_k]."""
    flat = experts.reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(count + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.bincount(flat, minlength=count).cumsum(0)
    return (order // experts.shape[1]).to(torch.int32), offsets


def forward(x: torch.Tensor, rows: torch.Tensor, offsets: torch.Tensor, e: Experts):
    """x [tokens][hidden] bf16 -> (the rows' outputs bf16, grouped by expert, what backward() needs)."""
    inner = e.w_down.shape[2]
    qx, sx = fp8q.gather_quantize_act(x, rows)
    gu = fp8q.grouped_gemm(qx, sx, e.c_gu.q, e.c_gu.s, offsets)
    qh, sh, kept = fp8q.swiglu_quantize(gu[:, :inner], gu[:, inner:])
    return fp8q.grouped_gemm(qh, sh, e.c_down.q, e.c_down.s, offsets), Saved(qx, sx, qh, sh, kept)


def backward(dy: torch.Tensor, s: Saved, offsets: torch.Tensor, e: Experts, accumulate: bool = False) -> torch.Tensor:
    """The rows' gradient; the weights' gradients are written (or added) to e.g_gu and e.g_down."""
    def wgrad(grad, qx, sx, dw):
        fp8q.grouped_wgrad(fp8q.grouped_quantize_act(grad, offsets), fp8q.grouped_requant_transpose(qx, sx, offsets), offsets,
                           dw=dw, accumulate=accumulate)

    dh = fp8q.grouped_gemm(*fp8q.quantize_act(dy), e.c_down.qt, e.c_down.st, offsets)
    wgrad(dy, s.qh, s.sh, e.g_down)
    dg, du = fp8q.swiglu_backward(s.kept, dh)
    dgu = dg.as_strided((dg.shape[0], 2 * dg.shape[1]), (dg.stride(0), 1))  # the halves lie side by side
    wgrad(dgu, s.qx, s.sx, e.g_gu)
    return fp8q.grouped_gemm(*fp8q.quantize_act(dgu), e.c_gu.qt, e.c_gu.st, offsets)


def train_step(x: torch.Tensor, experts: torch.Tensor, dy_of, e: Experts, step: int, lr: float = 1e-3):
    """One step; dy_of(y) gives the gradient of the rows' outputs.  Returns (y, rows' gradient)."""
    rows, offsets = route(experts, e.w_gu.shape[0])
    y, saved = forward(x, rows, offsets, e)
    dx = backward(dy_of(y), saved, offsets, e)
    fp8q.adamw(e.optimizer, step=step, lr=lr, seed=step)
    return y, dx


def main() -> None:
    tokens, experts, hidden, inner = (int(a) for a in sys.argv[1:5]) if len(sys.argv) > 4 else (1024, 8, 1024, 512)
    e = make_experts(experts, hidden, inner)
    torch.manual_seed(0)
    x = torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16)
    chosen = torch.rand((tokens, experts), device="cuda").topk(2).indices
    target = torch.randn((2 * tokens, hidden), device="cuda") * 0.1
    for step in range(1, 6):
        y, _ = train_step(x, chosen, lambda y: ((y.float() - target) / y.numel()).to(torch.bfloat16), e, step)
        print(f"step {step}: mean square {float((y.float() - target).square().mean()):.6f}")


if __name__ == "__main__":
    main()
