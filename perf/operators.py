"""Measured cases of the operators around the FP8 GEMMs of a feed-forward block.

Three families, each with its smallest calls, ordinary ones and large ones:

``norm`` / ``norm_grad``      layer norm (or RMS norm) into 1x128 FP8 codes, and its backward pass with the
                              reduction of the weights' gradients over the rows;
``swiglu`` / ``swiglu_grad``  SwiGLU into FP8 codes with its inputs kept as 8-bit checkpoints, and the backward
                              pass from those checkpoints;
``moe``                       a mixture-of-experts layer for the few tokens of a decode step.

Widths 7168 and 2048, 64 experts and 8192 rows are those of the repository's own workloads.  E4M3 codes are
returned as float8 tensors (the numbers that multiply the scales beside them).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-5
MOE_MAX_TOKENS = 64


def listed():
    return [
        # one token's hidden state before the first GEMM of a decode step: latency only
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 7168, "type": "bf16", "kind": "layer", "y": False},
        # a training step's tokens: codes for the GEMM, values for the router beside it
        {"name": "norm_train", "op": "norm", "rows": 8192, "cols": 7168, "type": "bf16", "kind": "rms", "y": True},
        # odd sizes in fp32: a ragged last tile, rows that do not fill a work-group
        {"name": "norm_ragged", "op": "norm", "rows": 1001, "cols": 1000, "type": "f32", "kind": "layer", "y": True},
        # the same training step backward, added to the gradient that goes round the block
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "cols": 7168, "type": "bf16", "kind": "layer",
         "skip": True},
        # odd sizes in fp32, no skip
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 777, "cols": 1001, "type": "f32", "kind": "layer",
         "skip": False},
        # a few tokens of serving: no checkpoint
        {"name": "swiglu_serve", "op": "swiglu", "rows": 7, "cols": 2048, "type": "bf16", "checkpoint": False},
        # a training step's tokens, inputs kept in 8 bits
        {"name": "swiglu_train", "op": "swiglu", "rows": 8192, "cols": 7168, "type": "bf16", "checkpoint": True},
        # the same step backward: every FP8 operand of the four backward GEMMs in one call
        {"name": "swiglu_grad_train", "op": "swiglu_grad", "rows": 8192, "cols": 7168, "type": "bf16",
         "quantize": True},
        # backward of a ragged batch into plain gradients, fp32
        {"name": "swiglu_grad_ragged", "op": "swiglu_grad", "rows": 1000, "cols": 1111, "type": "f32",
         "quantize": False},
        # one token through 8 of 64 experts: the decode step that streams 8 experts' weights
        {"name": "moe_token", "op": "moe", "tokens": 1, "experts": 64, "top_k": 8, "hidden": 7168, "inner": 2048,
         "padded": 0, "renormalize": True},
        # a decode batch, two slots of it empty: nearly every expert is active
        {"name": "moe_batch", "op": "moe", "tokens": 64, "experts": 64, "top_k": 8, "hidden": 7168, "inner": 2048,
         "padded": 2, "renormalize": True},
        # a small model's layer, five tokens, one of them an empty slot: latency
        {"name": "moe_small", "op": "moe", "tokens": 5, "experts": 16, "top_k": 2, "hidden": 512, "inner": 384,
         "padded": 1, "renormalize": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "swiglu", "swiglu_grad", "moe"])
    if op == "moe":
        experts = rng.choice([8, 16, 24, 40, 64])
        return {"op": op, "tokens": _log_int(rng, 1, MOE_MAX_TOKENS), "experts": experts,
                "top_k": rng.randint(1, 8), "hidden": 128 * _log_int(rng, 2, 56), "inner": 128 * _log_int(rng, 1, 16),
                "padded": rng.choice([0, 0, 1]), "renormalize": rng.random() < 0.5}
    cols = _log_int(rng, 64, 7168)
    rows = _log_int(rng, 1, min(32768, 8192 * 7168 // cols))
    c = {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("norm", "norm_grad"):
        c["kind"] = rng.choice(["layer", "rms"])
    if op == "norm":
        c["y"] = rng.random() < 0.5
    elif op == "norm_grad":
        c["skip"] = rng.random() < 0.5
    elif op == "swiglu":
        c["checkpoint"] = rng.random() < 0.75
    else:
        c["quantize"] = rng.random() < 0.6
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows16(rows, cols, dtype):
    """[rows][cols] whose row stride is a multiple of 16 bytes, as the library's operands have it."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _normal(g, rows, cols, dtype, std=1.0):
    t = _rows16(rows, cols, dtype)
    t.copy_(torch.randn((rows, cols), generator=g, device="cuda") * std)
    return t


def _tiles(x, axis):
    """x in float32 padded with zeros to whole 128-groups along `axis`, that axis split into (groups, 128)."""
    x = x.float()
    n = x.shape[axis]
    pad = -n % 128
    if pad:
        shape = list(x.shape)
        shape[axis] = pad
        x = torch.cat([x, x.new_zeros(shape)], dim=axis)
    return x.unflatten(axis, (-1, 128))


def _quantize_1x128(x):
    """(codes [rows][cols] float8, scales [groups][rows])"""
    rows, cols = x.shape
    t = _tiles(x, 1)
    s = t.abs().amax(dim=2) / E4M3_MAX
    d = torch.where(s > 0, s, torch.ones_like(s))[:, :, None]
    q = (t / d).clamp(-E4M3_MAX, E4M3_MAX).reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q, s.t().contiguous()


def _quantize_128x1(x):
    """(codes [cols][rows] float8, scales [groups][cols])"""
    rows, cols = x.shape
    t = _tiles(x, 0)
    s = t.abs().amax(dim=1) / E4M3_MAX
    d = torch.where(s > 0, s, torch.ones_like(s))[:, None, :]
    q = (t / d).clamp(-E4M3_MAX, E4M3_MAX).reshape(-1, cols)[:rows].t().contiguous().to(torch.float8_e4m3fn)
    return q, s


def _dequantize_1x128(q, s):
    """float32 values of uint8 codes [rows][cols] with scales [groups][rows]"""
    return q.view(torch.float8_e4m3fn).float() * s.t().repeat_interleave(128, dim=1)[:, : q.shape[1]]


def _codes(q):
    """float8 codes as the uint8 operand with a 16-byte row stride"""
    out = _rows16(q.shape[0], q.shape[1], torch.uint8)
    out.copy_(q.view(torch.uint8))
    return out


def _type(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def _weights(g, experts, rows, cols):
    """Codes [experts][rows][cols] of normally distributed weights of deviation 0.02, with 128x128 scales."""
    q = torch.empty((experts, rows, cols), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        v = torch.randn((rows, cols), generator=g, device="cuda").mul_(E4M3_MAX / 4.5).clamp_(-E4M3_MAX, E4M3_MAX)
        q[e] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.rand((experts, rows // 128, cols // 128), generator=g, device="cuda") * 0.2 + 0.9
    return q, s * (0.02 * 4.5 / E4M3_MAX)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "moe":
        T, E, H, I = case["tokens"], case["experts"], case["hidden"], case["inner"]
        st["x"] = _normal(g, T, H, torch.bfloat16)
        st["logits"] = torch.randn((T, E), generator=g, device="cuda")
        if case["padded"] and T > case["padded"]:  # empty slots of the batch: every expert masked
            st["logits"][T - case["padded"]:] = -math.inf
        st["w_gu"], st["s_gu"] = _weights(g, E, 2 * I, H)
        st["w_down"], st["s_down"] = _weights(g, E, H, I)
        return st
    rows, cols, dt = case["rows"], case["cols"], _type(case)
    if case["op"] in ("norm", "norm_grad"):
        x = _rows16(rows, cols, dt)
        # a residual stream: an offset, and a few channels far larger than the others
        v = torch.randn((rows, cols), generator=g, device="cuda") + 0.25
        v[:, torch.randint(0, cols, (max(1, cols // 1024),), generator=g, device="cuda")] *= 20.0
        x.copy_(v)
        st["x"] = x
        st["gamma"] = torch.randn((cols,), generator=g, device="cuda") * 0.1 + 1.0
        st["beta"] = torch.randn((cols,), generator=g, device="cuda") * 0.1 if case["kind"] == "layer" else None
        if case["op"] == "norm_grad":
            xf = x.double()
            mu = xf.mean(dim=1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(xf[:, :1])
            st["mean"] = mu[:, 0].float() if case["kind"] == "layer" else None
            st["rstd"] = ((xf - mu).square().mean(dim=1) + EPS).rsqrt().float()
            st["dy"] = _normal(g, rows, cols, dt, 1e-3)
            st["skip"] = _normal(g, rows, cols, dt, 1e-3) if case["skip"] else None
        return st
    gate, up = _normal(g, rows, cols, dt), _normal(g, rows, cols, dt)
    if case["op"] == "swiglu":
        st["g"], st["u"] = gate, up
        return st
    for name, v in (("g", gate), ("u", up)):
        q, s = _quantize_1x128(v)
        st["q" + name], st["s" + name] = _codes(q), s
    st["dh"] = _normal(g, rows, cols, dt, 1e-3)
    return st


# ------------------------------------------------------------------ one pass

def _f8(q):
    return q.view(torch.float8_e4m3fn)


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import fp8_fine_grained_x128_amd as fp8q
    op = st["op"]
    if op == "moe":
        return fp8q.moe_decode(st["x"], st["logits"], st["w_gu"], st["s_gu"], st["w_down"], st["s_down"],
                               st["top_k"], renormalize=st["renormalize"])
    if op == "norm":
        kind = fp8q.FP8Q_NORM_LAYER if st["kind"] == "layer" else fp8q.FP8Q_NORM_RMS
        o = fp8q.layernorm(st["x"], st["gamma"], st["beta"], eps=EPS, kind=kind,
                           out_dtype=st["x"].dtype if st["y"] else None)
        return {"q": _f8(o.q), "s": o.s, "y": o.y, "mean": o.mean, "rstd": o.rstd}
    if op == "norm_grad":
        kind = fp8q.FP8Q_NORM_LAYER if st["kind"] == "layer" else fp8q.FP8Q_NORM_RMS
        dx, dgamma, dbeta = fp8q.layernorm_backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"],
                                                    skip=st["skip"], kind=kind)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "swiglu":
        qh, sh, kept = fp8q.swiglu_quantize(st["g"], st["u"], checkpoint=st["checkpoint"])
        out = {"qh": _f8(qh), "sh": sh}
        if st["checkpoint"]:
            out.update(qg=_f8(kept.qg), qu=_f8(kept.qu), sg=kept.sg, su=kept.su)
        return out
    kept = fp8q.SwigluCheckpoint(st["qg"], st["qu"], st["sg"], st["su"])
    if st["quantize"]:
        o = fp8q.swiglu_backward_quantize(kept, st["dh"])
        return {"dg": _f8(o.qdg), "sdg": o.sdg, "du": _f8(o.qdu), "sdu": o.sdu, "dgt": _f8(o.qdgt), "sdgt": o.sdgt,
                "dut": _f8(o.qdut), "sdut": o.sdut, "ht": _f8(o.qht), "sht": o.sht}
    dg, du = fp8q.swiglu_backward(kept, st["dh"])
    return {"dg": dg, "du": du}


def _run_plain(st):
    op = st["op"]
    if op == "moe":
        return _moe_plain(st)
    if op == "norm":
        x = st["x"].float()
        layer = st["kind"] == "layer"
        mu = x.mean(dim=1, keepdim=True)
        d = x - mu if layer else x
        r = 1.0 / torch.sqrt(d.square().mean(dim=1, keepdim=True) + EPS)
        y = d * r * st["gamma"]
        if layer:
            y = y + st["beta"]
        q, s = _quantize_1x128(y)
        return {"q": q, "s": s, "y": y.to(st["x"].dtype) if st["y"] else None, "mean": mu[:, 0] if layer else None,
                "rstd": r[:, 0]}
    if op == "norm_grad":
        x, dy, r = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
        layer = st["kind"] == "layer"
        xh = (x - st["mean"][:, None]) * r if layer else x * r
        w = dy * st["gamma"]
        dx = w - xh * (w * xh).mean(dim=1, keepdim=True)
        if layer:
            dx = dx - w.mean(dim=1, keepdim=True)
        dx = dx * r
        if st["skip"] is not None:
            dx = dx + st["skip"].float()
        return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xh).sum(dim=0), "dbeta": dy.sum(dim=0) if layer else None}
    if op == "swiglu":
        g, u = st["g"].float(), st["u"].float()
        qh, sh = _quantize_1x128(g / (1.0 + torch.exp(-g)) * u)
        out = {"qh": qh, "sh": sh}
        if st["checkpoint"]:
            out["qg"], out["sg"] = _quantize_1x128(g)
            out["qu"], out["su"] = _quantize_1x128(u)
        return out
    g, u = _dequantize_1x128(st["qg"], st["sg"]), _dequantize_1x128(st["qu"], st["su"])
    dh = st["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    du = dh * g * sig
    dg = dh * u * sig * (1.0 + g * (1.0 - sig))
    if not st["quantize"]:
        return {"dg": dg.to(st["dh"].dtype), "du": du.to(st["dh"].dtype)}
    out = {}
    out["dg"], out["sdg"] = _quantize_1x128(dg)
    out["du"], out["sdu"] = _quantize_1x128(du)
    out["dgt"], out["sdgt"] = _quantize_128x1(dg)
    out["dut"], out["sdut"] = _quantize_128x1(du)
    out["ht"], out["sht"] = _quantize_128x1(g * sig * u)
    return out


def _dequantize_blocks(q, s):
    """float32 weights of codes [..][rows][cols] with scales [..][rows/128][cols/128]"""
    t = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    return (t * s[..., :, None, :, None]).flatten(-4, -3).flatten(-2, -1)


def _moe_plain(st):
    x, logits, k, inner = st["x"].float(), st["logits"], st["top_k"], st["inner"]
    T, E = logits.shape
    value, order = torch.sort(logits, dim=1, descending=True, stable=True)
    value, order = value[:, :k], order[:, :k]
    live = value > -math.inf
    top = torch.where(live[:, :1], value[:, :1], torch.zeros_like(value[:, :1]))
    p = torch.exp(value - top)
    total = p.sum(dim=1, keepdim=True) if st["renormalize"] else torch.exp(logits - top).sum(dim=1, keepdim=True)
    p = torch.where(live, p / total, torch.zeros_like(p))
    if T * k <= E:  # the chosen experts' weights, one product for each pair of token and expert
        w = _dequantize_blocks(st["w_gu"][order.reshape(-1)], st["s_gu"][order.reshape(-1)])
        a = (w * x.repeat_interleave(k, dim=0)[:, None, :]).sum(dim=2)
        h = a[:, :inner] / (1.0 + torch.exp(-a[:, :inner])) * a[:, inner:]
        w = _dequantize_blocks(st["w_down"][order.reshape(-1)], st["s_down"][order.reshape(-1)])
        y = (w * h[:, None, :]).sum(dim=2).reshape(T, k, -1)
        return (y * p[:, :, None]).sum(dim=1).to(torch.bfloat16)
    # every expert on every token, weighted with zero where it is not chosen
    a = torch.matmul(_dequantize_blocks(st["w_gu"], st["s_gu"]), x.t().contiguous())
    h = (a[:, :inner] / (1.0 + torch.exp(-a[:, :inner])) * a[:, inner:]).contiguous()
    y = torch.matmul(_dequantize_blocks(st["w_down"], st["s_down"]), h)
    weight = torch.zeros((T, E), device=x.device).scatter_(1, order, p)
    return (y * weight.t()[:, None, :]).sum(dim=0).t().contiguous().to(torch.bfloat16)


# ------------------------------------------------------------------ 64 bits

def _e4m3_64(v):
    """Nearest E4M3 value of float64 numbers: 4 significant bits, ties to even, subnormal step 2^-9, at most 448."""
    a = v.abs().clamp(max=E4M3_MAX)
    e = torch.frexp(a).exponent.to(torch.float64) - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), v)


def _exact_rows(v):
    """1x128 codes' values and scales of float64 numbers"""
    rows, cols = v.shape
    groups = -(-cols // 128)
    t = v.new_zeros((rows, groups * 128))
    t[:, :cols] = v
    t = t.view(rows, groups, 128)
    s = t.abs().amax(dim=2) / E4M3_MAX
    q = _e4m3_64(torch.nan_to_num(t / s[:, :, None], nan=0.0))
    return q.view(rows, -1)[:, :cols].contiguous(), s.t().contiguous()


def _exact_columns(v):
    return _exact_rows(v.t().contiguous())


def _values_64(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().t().repeat_interleave(128, dim=1)[:, : q.shape[1]]


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "moe":
        return _moe_exact(st)
    if op == "norm":
        x = st["x"].double()
        layer = st["kind"] == "layer"
        mu = x.sum(dim=1, keepdim=True) / x.shape[1] if layer else torch.zeros_like(x[:, :1])
        var = (x - mu).pow(2).sum(dim=1, keepdim=True) / x.shape[1]
        r = (var + EPS).pow(-0.5)
        y = (x - mu) * r * st["gamma"].double() + (st["beta"].double() if layer else 0.0)
        q, s = _exact_rows(y)
        return {"q": q, "s": s, "y": y if st["y"] else None, "mean": mu[:, 0] if layer else None, "rstd": r[:, 0]}
    if op == "norm_grad":
        x, dy, r = st["x"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        layer = st["kind"] == "layer"
        n = x.shape[1]
        xh = (x - (st["mean"].double()[:, None] if layer else 0.0)) * r
        w = dy * st["gamma"].double()
        dx = r / n * (n * w - xh * (w * xh).sum(dim=1, keepdim=True)
                      - (w.sum(dim=1, keepdim=True) if layer else 0.0))
        if st["skip"] is not None:
            dx = dx + st["skip"].double()
        return {"dx": dx, "dgamma": (dy * xh).sum(dim=0), "dbeta": dy.sum(dim=0) if layer else None}
    if op == "swiglu":
        g, u = st["g"].double(), st["u"].double()
        out = {}
        out["qh"], out["sh"] = _exact_rows(g * torch.sigmoid(g) * u)
        if st["checkpoint"]:
            out["qg"], out["sg"] = _exact_rows(g)
            out["qu"], out["su"] = _exact_rows(u)
        return out
    g, u, dh = _values_64(st["qg"], st["sg"]), _values_64(st["qu"], st["su"]), st["dh"].double()
    sig = torch.sigmoid(g)
    du = dh * (g * sig)
    dg = dh * u * (sig + g * sig * (1.0 - sig))
    if not st["quantize"]:
        return {"dg": dg, "du": du}
    out = {}
    out["dg"], out["sdg"] = _exact_rows(dg)
    out["du"], out["sdu"] = _exact_rows(du)
    out["dgt"], out["sdgt"] = _exact_columns(dg)
    out["dut"], out["sdut"] = _exact_columns(du)
    out["ht"], out["sht"] = _exact_columns(g * sig * u)
    return out


def _moe_exact(st):
    x, k, inner = st["x"].double(), st["top_k"], st["inner"]
    logits = st["logits"].double().cpu()
    T, E = logits.shape
    y = torch.zeros((T, st["hidden"]), dtype=torch.float64, device="cuda")
    rows = logits.tolist()
    chosen = [[] for _ in range(E)]
    for t, row in enumerate(rows):
        ids = [e for e in sorted(range(E), key=lambda e: (-row[e], e))[:k] if row[e] > -math.inf]
        if not ids:
            continue
        top = row[ids[0]]
        total = math.fsum(math.exp(row[e] - top) for e in (ids if st["renormalize"] else range(E)))
        for e in ids:
            chosen[e].append((t, math.exp(row[e] - top) / total))

    def weight(q, s):
        return (q.view(torch.float8_e4m3fn).double()
                * s.double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1))

    for e in range(E):
        if not chosen[e]:
            continue
        at = torch.tensor([t for t, _ in chosen[e]], device="cuda")
        p = torch.tensor([v for _, v in chosen[e]], dtype=torch.float64, device="cuda")
        a = weight(st["w_gu"][e], st["s_gu"][e]) @ x[at].t().contiguous()
        h = torch.sigmoid(a[:inner]) * a[:inner] * a[inner:]
        y[at] += p[:, None] * (weight(st["w_down"][e], st["s_down"][e]) @ h).t()
    return y


# ------------------------------------------------------------------ work

def work(case):
    """Bytes each input is read and each output written once; operations counted once each (a product and a sum are two)."""
    if case["op"] == "moe":
        T, E, k, H, I = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "inner"))
        live = T - (case["padded"] if T > case["padded"] else 0)
        k = min(k, E)
        active = E * (1.0 - (1.0 - k / E) ** live)  # expected number of experts that some token chooses
        weights = 3 * H * I * (1 + 4 / 16384.0)
        return {"bytes": active * weights + T * (4 * H + 4 * E), "flops": 6.0 * H * I * live * k}
    n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
    e = 2 if case["type"] == "bf16" else 4
    codes = n + 4 * rows * (-(-cols // 128))        # 1x128 codes with their scales
    columns = n + 4 * cols * (-(-rows // 128))      # 128x1
    layer = 1 if case.get("kind") == "layer" else 0
    if case["op"] == "norm":
        return {"bytes": e * n * (2 if case["y"] else 1) + codes + 4 * cols * (1 + layer) + 4 * rows * (1 + layer),
                "flops": (8 + 2 * layer) * n}
    if case["op"] == "norm_grad":
        return {"bytes": e * n * (4 if case["skip"] else 3) + 4 * cols * (2 + layer) + 4 * rows * (1 + layer),
                "flops": (11 + 3 * layer) * n}
    if case["op"] == "swiglu":
        return {"bytes": 2 * e * n + codes * (3 if case["checkpoint"] else 1),
                "flops": (10 if case["checkpoint"] else 6) * n}
    if case["quantize"]:
        return {"bytes": 2 * codes + e * n + 2 * codes + 3 * columns, "flops": 24 * n}
    return {"bytes": 2 * codes + e * n + 2 * e * n, "flops": 14 * n}
