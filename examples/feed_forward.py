"""A feed-forward block in FP8: one training step, and a decode step of its
mixture-of-experts form.

    python examples/feed_forward.py [tokens hidden inner]

Training (dense): norm -> gate|up GEMM -> SwiGLU -> down GEMM, plus the
residual.  Between forward and backward only FP8 is kept of the block: the
normalized activations (the operand of the first GEMM) and the SwiGLU's inputs;
the SwiGLU's output is recomputed.  x itself belongs to the residual stream.
Serving: the same block with 16 experts, a few tokens at a time.
"""
from __future__ import annotations

import os
import sys
from typing import NamedTuple, Optional

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_x128_amd as fp8q  # noqa: E402


class Block(NamedTuple):
    gamma: torch.Tensor                # [hidden]
    beta: Optional[torch.Tensor]       # [hidden]; None: RMS norm
    w_gu: torch.Tensor                 # codes [2*inner][hidden], gate rows first
    s_gu: torch.Tensor                 # [2*inner/128][hidden/128]
    w_down: torch.Tensor               # codes [hidden][inner]
    s_down: torch.Tensor               # [hidden/128][inner/128]

    @property
    def kind(self) -> int:
        return fp8q.FP8Q_NORM_RMS if self.beta is None else fp8q.FP8Q_NORM_LAYER


class Saved(NamedTuple):
    x: torch.Tensor
    n: fp8q.LayernormOut
    kept: fp8q.SwigluCheckpoint


class Gradients(NamedTuple):
    x: torch.Tensor
    gamma: torch.Tensor
    beta: Optional[torch.Tensor]
    w_gu: torch.Tensor
    w_down: torch.Tensor


def forward(x: torch.Tensor, b: Block):
    """x [tokens][hidden] bf16 -> (x + block(x), what backward() needs)."""
    inner = b.w_down.shape[1]
    n = fp8q.layernorm(x, b.gamma, b.beta, kind=b.kind)
    gu = fp8q.gemm(n.q, n.s, b.w_gu, b.s_gu)
    qh, sh, kept = fp8q.swiglu_quantize(gu[:, :inner], gu[:, inner:])
    y = fp8q.gemm(qh, sh, b.w_down, b.s_down)
    return x + y, Saved(x, n, kept)


def backward(dy: torch.Tensor, saved: Saved, b: Block) -> Gradients:
    """Every GEMM of the backward pass runs on FP8 operands; weights' gradients are fp32."""
    q, s = fp8q.quantize_act(dy)
    qt, st = fp8q.quantize_act(dy, fp8q.FP8Q_TILE_128x1)
    dh = fp8q.dgrad(q, s, *fp8q.transpose_weight(b.w_down, b.s_down))
    g = fp8q.swiglu_backward_quantize(saved.kept, dh)
    dw_down = fp8q.gemm(qt, st, g.qht, g.sht, bscale=fp8q.FP8Q_BSCALE_ROW, out_dtype=torch.float32)
    q, s, qt, st = g.gate_up()
    dn = fp8q.dgrad(q, s, *fp8q.transpose_weight(b.w_gu, b.s_gu))
    qx, sx = fp8q.requant_transpose(saved.n.q, saved.n.s)
    dw_gu = fp8q.gemm(qt, st, qx, sx, bscale=fp8q.FP8Q_BSCALE_ROW, out_dtype=torch.float32)
    dx, dgamma, dbeta = fp8q.layernorm_backward(dn, saved.x, b.gamma, saved.n.mean, saved.n.rstd, skip=dy, kind=b.kind)
    return Gradients(dx, dgamma, dbeta, dw_gu, dw_down)


def decode(x: torch.Tensor, router: torch.Tensor, b: Block, top_k: int) -> torch.Tensor:
    """A decode step of the block with experts: b.w_gu [experts][2*inner][hidden] and so on, router [experts][hidden]
    bf16; the gate stays in higher precision.  x + experts(norm(x))."""
    n = fp8q.layernorm(x, b.gamma, b.beta, kind=b.kind, quantize=False, out_dtype=torch.bfloat16).y
    logits = (n @ router.t()).float()
    return x + fp8q.moe_decode(n, logits, b.w_gu, b.s_gu, b.w_down, b.s_down, top_k)


def make_block(hidden: int, inner: int, experts: int = 0, rms: bool = False, seed: int = 0) -> Block:
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def weight(rows, cols):
        w = torch.randn((rows, cols), generator=gen, device="cuda") * cols ** -0.5
        return fp8q.quantize_weight(w.to(torch.bfloat16))

    def weights(rows, cols):
        if not experts:
            return weight(rows, cols)
        return tuple(torch.stack(t) for t in zip(*(weight(rows, cols) for _ in range(experts))))

    gamma = 1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")
    beta = None if rms else 0.1 * torch.randn(hidden, generator=gen, device="cuda")
    return Block(gamma, beta, *weights(2 * inner, hidden), *weights(hidden, inner))


def main(tokens: int = 4096, hidden: int = 7168, inner: int = 2048) -> None:
    b = make_block(hidden, inner)
    x = torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16)
    target = torch.randn_like(x)
    y, saved = forward(x, b)
    loss = (y.float() - target.float()).square().mean()
    g = backward(((2.0 / y.numel()) * (y.float() - target.float())).to(torch.bfloat16), saved, b)
    kept = sum(t.numel() * t.element_size() for t in (saved.n.q, saved.n.s, *saved.kept))
    print(f"training: loss {loss.item():.4f}, |dx| {g.x.float().norm().item():.3e}, "
          f"|dW_gate_up| {g.w_gu.norm().item():.3e}, |dW_down| {g.w_down.norm().item():.3e}; "
          f"{kept / 2**20:.0f} MiB kept for {tokens} tokens")
    e = make_block(hidden, inner, experts=16, rms=True, seed=1)
    router = (torch.randn((16, hidden), device="cuda") * hidden ** -0.5).to(torch.bfloat16)
    y = decode(x[:4], router, e, top_k=4)
    print(f"decode: 4 tokens through 4 of 16 experts, |y| {y.float().norm().item():.3e}")


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
