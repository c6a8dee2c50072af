"""Measured cases of the experts' backward products and of the optimizer step that takes their gradients.

Three families, each with its smallest calls, ordinary ones and large ones:

``columns``  the operands of the weight gradients: rows grouped by expert, quantized (or requantized from the cached
             1x128 codes) per 128 tokens of one expert, transposed, each expert padded to whole tiles;
``wgrad``    the weight gradient of every expert, contracted over that expert's own tokens;
``adamw``    one AdamW step over many tensors: master weights and gradients, moments in 32 or in 8 bits, and the FP8
             codes of the new weights (and of their transposes) for the next step's GEMMs.

Widths 7168, 4096 and 2048, 64 experts, 32768 rows and Zipf(1.1) expert sizes are those of the repository's own
workloads.  E4M3 codes are returned as float8 tensors (the numbers that multiply the scales beside them).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 3e-4
SEED = 20250


def listed():
    return [
        # the down projections' incoming gradient of a training step, 64 experts of very different sizes
        {"name": "columns_train", "op": "columns", "rows": 32768, "cols": 2048, "experts": 64, "source": "bf16"},
        # the cached FP8 inputs of the same step, converted for the same products
        {"name": "columns_cached", "op": "columns", "rows": 32768, "cols": 7168, "experts": 64, "source": "codes"},
        # a small ragged batch in fp32, experts without tokens among them: latency
        {"name": "columns_small", "op": "columns", "rows": 333, "cols": 1000, "experts": 160, "source": "f32"},
        # weight gradients of 64 experts: about 512 tokens for each, so the gradients themselves are most of the bytes
        {"name": "wgrad_train", "op": "wgrad", "rows": 32768, "experts": 64, "N": 2048, "K": 7168, "type": "f32",
         "accumulate": False},
        # few large experts, added to the gradients of the micro-batch before: the product is most of the time
        {"name": "wgrad_tokens", "op": "wgrad", "rows": 16384, "experts": 4, "N": 4096, "K": 7168, "type": "f32",
         "accumulate": True},
        # a small model's layer: few output tiles, many tokens for each
        {"name": "wgrad_long", "op": "wgrad", "rows": 8192, "experts": 4, "N": 384, "K": 512, "type": "f32",
         "accumulate": False},
        # odd widths and a small batch, bf16 gradients
        {"name": "wgrad_ragged", "op": "wgrad", "rows": 1000, "experts": 16, "N": 333, "K": 1111, "type": "bf16",
         "accumulate": False},
        # norm weights and biases: many small vectors, latency
        {"name": "adamw_vectors", "op": "adamw", "experts": 0, "N": 0, "K": 0, "vectors": 60, "longest": 7168,
         "type": "f32", "bits": 32, "transposed": False},
        # a dense projection and its block's vectors: fp32 moments, codes for the forward and the backward GEMM
        {"name": "adamw_dense", "op": "adamw", "experts": 1, "N": 4096, "K": 7168, "vectors": 4, "longest": 7168,
         "type": "f32", "bits": 32, "transposed": True},
        # experts with 8-bit moments: the largest arrays of a mixture-of-experts model
        {"name": "adamw_experts", "op": "adamw", "experts": 16, "N": 2048, "K": 7168, "vectors": 0, "longest": 0,
         "type": "f32", "bits": 8, "transposed": True},
        # tensors of odd sizes, bf16 gradients, 8-bit moments, no codes
        {"name": "adamw_ragged", "op": "adamw", "experts": 0, "N": 0, "K": 0, "vectors": 13, "longest": 1500001,
         "type": "bf16", "bits": 8, "transposed": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["columns", "wgrad", "wgrad", "adamw", "adamw"])
    if op == "columns":
        cols = _log_int(rng, 64, 7168)
        return {"op": op, "rows": _log_int(rng, 1, 32768), "cols": cols, "experts": _log_int(rng, 1, 256),
                "source": rng.choice(["bf16", "f32", "codes"])}
    if op == "wgrad":
        experts, n, k = _log_int(rng, 1, 64), _log_int(rng, 64, 4096), _log_int(rng, 64, 7168)
        if rng.random() < 0.5:  # widths as models have them
            n, k = 64 * -(-n // 64), 64 * -(-k // 64)
        rows = min(_log_int(rng, 16, 32768), 32768 * 2048 * 7168 // (n * k))
        experts = max(1, min(experts, 64 * 2048 * 7168 // (n * k)))
        kind = rng.choice(["f32", "f32", "bf16"])
        return {"op": op, "rows": rows, "experts": experts, "N": n, "K": k, "type": kind,
                "accumulate": kind == "f32" and rng.random() < 0.4}
    bits, kind = rng.choice([8, 32]), rng.choice(["f32", "bf16"])
    if rng.random() < 0.6:
        n, k = _log_int(rng, 16, 4096), 128 * _log_int(rng, 1, 56)
        experts = max(1, min(_log_int(rng, 1, 32), 16 * 2048 * 7168 // (n * k)))
        return {"op": op, "experts": experts, "N": n, "K": k, "vectors": rng.choice([0, 3, 8]), "longest": 7168,
                "type": kind, "bits": bits, "transposed": rng.random() < 0.5}
    return {"op": op, "experts": 0, "N": 0, "K": 0, "vectors": _log_int(rng, 1, 200), "longest": _log_int(rng, 16, 500000),
            "type": kind, "bits": bits, "transposed": False}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _counts(rows, experts, seed):
    """Zipf(1.1) expert sizes by largest remainder, dealt to the experts by a permutation of the seed."""
    weight = torch.arange(1, experts + 1, dtype=torch.float64).pow(-1.1)
    share = weight / weight.sum() * rows
    counts = share.floor().long()
    order = torch.argsort(share - counts, descending=True, stable=True)
    counts[order[: rows - int(counts.sum())]] += 1
    g = torch.Generator()
    g.manual_seed(seed)
    return counts[torch.randperm(experts, generator=g)].tolist()


def _padded(rows, experts):
    """Tokens that the padded layout has room for, whatever the experts' sizes are."""
    return (rows + 127 * min(experts, rows)) // 128 * 128


def _rows16(rows, cols, dtype):
    """[rows][cols] whose row stride is a multiple of 16 bytes, as the library's operands have it."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _layout(counts):
    """Places of the experts' tokens in the padded layout: (place of each row, tokens of whole tiles)"""
    place, at = [], 0
    for n in counts:
        place.append(torch.arange(at, at + n))
        at += -(-n // 128) * 128
    return torch.cat(place), at


def _flat_layout(case):
    """Sizes of the tensors, and their starts in the flat arrays (multiples of 128 elements)."""
    sizes = [case["experts"] * case["N"] * case["K"]] if case["experts"] else []
    for i in range(case["vectors"]):  # the longest first, then a range of shorter ones
        sizes.append(max(1, case["longest"] >> (i % 5)) if i else case["longest"])
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // 128) * 128
    return sizes, starts, at


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _random_codes(g, rows, cols):
    v = torch.randn((rows, cols), generator=g, device="cuda").mul_(E4M3_MAX / 4.5).clamp_(-E4M3_MAX, E4M3_MAX)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(st, g)
    counts = _counts(case["rows"], case["experts"], seed)
    place, used = _layout(counts)
    ends = torch.tensor([0] + counts).cumsum(0)
    st.update(counts=counts, used=used, place=place.cuda(), offsets=ends.to(torch.int32).cuda())
    rows = case["rows"]
    if case["op"] == "columns":
        cols = case["cols"]
        if case["source"] == "codes":
            st["x"] = _rows16(rows, cols, torch.uint8)
            st["x"].copy_(_random_codes(g, rows, cols))
            st["sx"] = torch.rand((-(-cols // 128), rows), generator=g, device="cuda") * 0.01 + 0.005
        else:
            st["x"] = _rows16(rows, cols, _type(case["source"]))
            st["x"].copy_(torch.randn((rows, cols), generator=g, device="cuda") * 1e-3)
        return st
    cap = _padded(rows, case["experts"])
    live = torch.zeros(cap, dtype=torch.bool, device="cuda")
    live[st["place"]] = True
    for name, width, scale in (("dy", case["N"], 1e-5), ("x", case["K"], 1e-2)):
        q = _random_codes(g, width, cap)
        q.masked_fill_(~live[None, :], 0)
        st["q" + name] = q
        st["s" + name] = (torch.rand((cap // 128, width), generator=g, device="cuda") + 0.5) * scale
    if case["accumulate"]:
        st["dw"] = torch.randn((case["experts"], case["N"], case["K"]), generator=g, device="cuda") * 1e-2
    return st


def _prepare_adamw(st, g):
    sizes, starts, n = _flat_layout(st)
    st.update(sizes=sizes, starts=starts, step=1000)
    spread = torch.empty(n // 128, 1, device="cuda").uniform_(-2.0, 2.0, generator=g).exp_().mul_(1e-4)
    live = torch.zeros(n, device="cuda")
    for size, start in zip(sizes, starts):
        live[start: start + size] = 1.0

    def rand(scale):
        v = torch.randn((n // 128, 128), generator=g, device="cuda")
        return v.mul_(scale).view(-1).mul_(live)

    st["p"] = rand(0.02)
    st["g"] = rand(spread).to(_type(st["type"]))
    m, r = rand(0.4 * spread), rand(spread).abs_().add_(0.3 * spread.expand(-1, 128).reshape(-1) * live)
    if st["bits"] == 32:
        st["m"], st["v"] = m, r.square()
    else:
        for name, v in (("m", m), ("v", r)):
            t = v.view(-1, 128)
            s = t.abs().amax(dim=1) / E4M3_MAX
            d = torch.where(s > 0, s, torch.ones_like(s))[:, None]
            st[name] = (t / d).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
            st["s" + name] = s
    if st["experts"]:
        E, N, K = st["experts"], st["N"], st["K"]
        st["q"] = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
        st["s"] = torch.zeros((E, -(-N // 128), K // 128), device="cuda")
        if st["transposed"]:
            st["qt"] = torch.zeros((E, K, -(-N // 16) * 16), dtype=torch.uint8, device="cuda")[:, :, :N]
            st["st"] = torch.zeros((E, K // 128, -(-N // 128)), device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def _f8(q):
    return q.view(torch.float8_e4m3fn)


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import fp8_fine_grained_x128_amd as fp8q
    if st["op"] == "columns":
        if st["source"] == "codes":
            o = fp8q.grouped_requant_transpose(st["x"], st["sx"], st["offsets"])
        else:
            o = fp8q.grouped_quantize_act(st["x"], st["offsets"])
        return {"q": o.q.view(torch.float8_e4m3fn)[:, : st["used"]], "s": o.s[: st["used"] // 128]}
    if st["op"] == "wgrad":
        dy = fp8q.GroupedOperand(st["qdy"], st["sdy"], st["rows"])
        x = fp8q.GroupedOperand(st["qx"], st["sx"], st["rows"])
        return fp8q.grouped_wgrad(dy, x, st["offsets"], out_dtype=_type(st["type"]), dw=st.get("dw"),
                                  accumulate=st["accumulate"])
    if "plan" not in st:
        params, grads, states, codes = [], [], [], []
        for i, (size, start) in enumerate(zip(st["sizes"], st["starts"])):
            at = slice(start, start + size)
            shape = (st["experts"], st["N"], st["K"]) if st["experts"] and i == 0 else (size,)
            params.append(st["p"][at].view(shape))
            grads.append(st["g"][at].view(shape))
            if st["bits"] == 32:
                states.append(fp8q.AdamwState(st["m"][at], st["v"][at], None, None))
            else:
                tiles = slice(start // 128, start // 128 + -(-size // 128))
                states.append(fp8q.AdamwState(st["m"][at], st["v"][at], st["sm"][tiles], st["sv"][tiles]))
            codes.append(fp8q.WeightCodes(st["q"], st["s"], st.get("qt"), st.get("st")) if len(shape) == 3 else None)
        st["plan"] = fp8q.adamw_tensors(params, grads, states, codes)
    st["step"] += 1
    fp8q.adamw(st["plan"], step=st["step"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, seed=SEED)
    return _adamw_outputs(st)


def _adamw_outputs(st):
    out = {"p": st["p"]}
    if st["bits"] == 32:
        out.update(m=st["m"], v=st["v"])
    else:
        out.update(m=_f8(st["m"]), v=_f8(st["v"]), sm=st["sm"], sv=st["sv"])
    if st["experts"]:
        out.update(q=_f8(st["q"]), s=st["s"])
        if st["transposed"]:
            out.update(qt=_f8(st["qt"]), st=st["st"])
    return out


def _run_plain(st):
    if st["op"] == "columns":
        return _columns_plain(st)
    if st["op"] == "wgrad":
        return _wgrad_plain(st)
    return _adamw_plain(st)


def _columns_plain(st):
    x = st["x"]
    if st["source"] == "codes":
        x = x.contiguous().view(torch.float8_e4m3fn).float()
        x = x * st["sx"].t().repeat_interleave(128, dim=1)[:, : x.shape[1]]
    x = x.float()
    t = x.new_zeros((st["used"], x.shape[1]))
    t[st["place"]] = x
    t = t.view(-1, 128, x.shape[1])
    s = t.abs().amax(dim=1) / E4M3_MAX
    d = torch.where(s > 0, s, torch.ones_like(s))[:, None, :]
    q = (t / d).clamp(-E4M3_MAX, E4M3_MAX).view(-1, x.shape[1]).t().contiguous().to(torch.float8_e4m3fn)
    return {"q": q, "s": s}


def _values(q, s, used):
    """float32 values [used tokens][width] of transposed codes"""
    t = q[:, :used].contiguous().view(torch.float8_e4m3fn).float().t().contiguous()
    return t * s[: used // 128].repeat_interleave(128, dim=0)


def _wgrad_plain(st):
    dy, x = _values(st["qdy"], st["sdy"], st["used"]), _values(st["qx"], st["sx"], st["used"])
    out, at = torch.empty((st["experts"], st["N"], st["K"]), device=x.device), 0
    for e, n in enumerate(st["counts"]):  # a library product for each expert
        to = at + -(-n // 128) * 128
        torch.mm(dy[at:to].t(), x[at:to], out=out[e])
        at = to
    if st["accumulate"]:
        return st["dw"].add_(out)
    return out.to(_type(st["type"]))


def _mix(x):
    """32 bits from 32 bits: two rounds of xor-shift and multiplication (int64 arithmetic modulo 2^32)"""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_16(st, device):
    """Two 16-bit numbers for each element of the flat arrays, from the seed, the tensor's place in the list, the step
    and the element's index in its tensor"""
    starts = torch.tensor(st["starts"], device=device)
    lengths = torch.tensor(st["starts"][1:] + [st["p"].numel()], device=device) - starts
    key = _mix((_mix((SEED + torch.arange(len(starts), device=device) * 0x9E3779B9) & 0xFFFFFFFF) + st["step"]) & 0xFFFFFFFF)
    n = st["p"].numel()
    index = torch.arange(n, device=device) - starts.repeat_interleave(lengths, output_size=n)
    h = _mix(index ^ key.repeat_interleave(lengths, output_size=n))
    return h & 0xFFFF, h >> 16


def _round_e4m3(v, bits):
    """(values on the E4M3 grid, scales) of tiles of 128; the neighbour above with a probability of v's way to it"""
    t = v.view(-1, 128)
    s = t.abs().amax(dim=1) / E4M3_MAX
    y = t.abs() / torch.where(s > 0, s, torch.ones_like(s))[:, None]
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y).exponent - 1).clamp(min=-6) - 3)
    u = (bits.view(-1, 128).float() + 0.5) / 65536.0
    y = (torch.floor(y / step + u) * step).clamp(max=E4M3_MAX)
    return torch.copysign(y, t).view(-1), s


def _quantize_blocks(w):
    """128x128 codes of [E][N][K] weights: (float8 codes, scales)"""
    E, N, K = w.shape
    rows = -(-N // 128)
    t = w
    if N % 128:
        t = w.new_zeros((E, rows * 128, K))
        t[:, :N] = w
    t = t.view(E, rows, 128, K // 128, 128)
    s = t.abs().amax(dim=(2, 4)) / E4M3_MAX
    d = torch.where(s > 0, s, torch.ones_like(s))[:, :, None, :, None]
    q = (t / d).clamp(-E4M3_MAX, E4M3_MAX).view(E, rows * 128, K)[:, :N].to(torch.float8_e4m3fn)
    return q, s


def _adamw_plain(st):
    st["step"] += 1
    p, g = st["p"], st["g"].float()
    bc1, bc2 = 1.0 - BETA1 ** st["step"], 1.0 - BETA2 ** st["step"]
    if st["bits"] == 32:
        m = st["m"].mul_(BETA1).add_(g, alpha=1.0 - BETA1)
        v = st["v"].mul_(BETA2).add_(g * g, alpha=1.0 - BETA2)
        root = torch.sqrt(v)
    else:
        m, r = ((st[n].view(torch.float8_e4m3fn).float().view(-1, 128) * st["s" + n][:, None]).view(-1) for n in ("m", "v"))
        m = m * BETA1 + g * (1.0 - BETA1)
        root = torch.sqrt(r * r * BETA2 + g * g * (1.0 - BETA2))
        low, high = _random_16(st, p.device)
        code, st["sm"][:] = _round_e4m3(m, low)
        st["m"].copy_(code.to(torch.float8_e4m3fn).view(torch.uint8))
        code, st["sv"][:] = _round_e4m3(root, high)
        code = torch.where(root > 0, code.clamp(min=2.0 ** -9), code)
        st["v"].copy_(code.to(torch.float8_e4m3fn).view(torch.uint8))
    p.mul_(1.0 - LR * DECAY).addcdiv_(m, root / math.sqrt(bc2) + EPS, value=-LR / bc1)
    if st["experts"]:
        E, N, K = st["experts"], st["N"], st["K"]
        q, s = _quantize_blocks(p[: E * N * K].view(E, N, K))
        st["q"].copy_(q.view(torch.uint8))
        st["s"].copy_(s)
        if st["transposed"]:
            st["qt"].copy_(q.view(torch.uint8).transpose(1, 2))
            st["st"].copy_(s.transpose(1, 2))
    return _adamw_outputs(st)


# ------------------------------------------------------------------ 64 bits

def _e4m3_64(v):
    """Nearest E4M3 value of float64 numbers: 4 significant bits, ties to even, subnormal step 2^-9, at most 448."""
    a = v.abs().clamp(max=E4M3_MAX)
    e = torch.frexp(a).exponent.to(torch.float64) - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), v)


def _tiles_64(v):
    """Values on the E4M3 grid and scales of float64 [tiles][128]"""
    s = v.abs().max(dim=1).values / E4M3_MAX
    return _e4m3_64(torch.nan_to_num(v / s[:, None], nan=0.0)), s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "columns":
        x = st["x"].double() if case["source"] != "codes" else st["x"].contiguous().view(torch.float8_e4m3fn).double()
        cols = x.shape[1]
        if case["source"] == "codes":
            for j in range(st["sx"].shape[0]):
                x[:, 128 * j: 128 * j + 128] *= st["sx"][j].double()[:, None]
        q = torch.zeros((cols, st["used"]), dtype=torch.float64, device="cuda")
        s = torch.zeros((st["used"] // 128, cols), dtype=torch.float64, device="cuda")
        row = chunk = 0
        for n in st["counts"]:
            for first in range(0, n, 128):
                part = torch.zeros((cols, 128), dtype=torch.float64, device="cuda")
                part[:, : min(128, n - first)] = x[row + first: row + min(first + 128, n)].t()
                q[:, 128 * chunk: 128 * chunk + 128], s[chunk] = _tiles_64(part)
                chunk += 1
            row += n
        return {"q": q, "s": s}
    if case["op"] == "wgrad":
        sides = []
        for name in ("dy", "x"):
            v = st["q" + name].view(torch.float8_e4m3fn).double()[:, : st["used"]]
            for c in range(st["used"] // 128):
                v[:, 128 * c: 128 * c + 128] *= st["s" + name][c].double()[:, None]
            sides.append(v)
        out = torch.zeros((case["experts"], case["N"], case["K"]), dtype=torch.float64, device="cuda")
        at = 0
        for e, n in enumerate(st["counts"]):
            to = at + 128 * math.ceil(n / 128)
            out[e] = sides[0][:, at:to] @ sides[1][:, at:to].t().contiguous()
            at = to
        return out + st["dw"].double() if case["accumulate"] else out
    return _adamw_exact(case, st)


def _hash_64(x):
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B), (16, 1)):
        x = ((x ^ (x >> shift)) * factor) % (1 << 32)
    return x


def _stochastic_64(v, u):
    """E4M3 values of float64 [tiles][128]: k or k + 1 steps, k + 1 where the rest and u make a whole step"""
    s = v.abs().max(dim=1).values / E4M3_MAX
    y = torch.nan_to_num(v.abs() / s[:, None], nan=0.0)
    e = torch.frexp(y).exponent.to(torch.float64) - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    k = torch.floor(y / step)
    k = k + ((y / step - k) + u >= 1.0).double()
    return torch.sign(v) * torch.minimum(k * step, torch.full_like(y, E4M3_MAX)), s


def _adamw_exact(case, st):
    t = st["step"] + 1
    out = {"p": st["p"].double()}
    names = ("m", "v") if case["bits"] == 32 else ("m", "v", "sm", "sv")
    for name in names:
        out[name] = torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
    for i, (size, start) in enumerate(zip(st["sizes"], st["starts"])):
        n = 128 * math.ceil(size / 128)
        at, tiles = slice(start, start + n), slice(start // 128, (start + n) // 128)
        g = st["g"][at].double()
        if case["bits"] == 32:
            m0, v0 = st["m"][at].double(), st["v"][at].double()
        else:
            m0, r0 = ((st[k][at].view(torch.float8_e4m3fn).double().view(-1, 128) * st["s" + k][tiles].double()[:, None])
                      .view(-1) for k in ("m", "v"))
            v0 = r0.pow(2)
        m = BETA1 * m0 + (1.0 - BETA1) * g
        v = BETA2 * v0 + (1.0 - BETA2) * g.pow(2)
        p = out["p"][at]
        p -= LR * DECAY * p
        p -= LR * (m / (1.0 - BETA1 ** t)) / ((v / (1.0 - BETA2 ** t)).pow(0.5) + EPS)
        if case["bits"] == 32:
            out["m"][at], out["v"][at] = m, v
            continue
        key = _hash_64((_hash_64((SEED + i * 0x9E3779B9) % (1 << 32)) + t) % (1 << 32))
        h = _hash_64(torch.arange(n, device="cuda") ^ key)
        q, s = _stochastic_64(m.view(-1, 128), ((h % 65536).double() + 0.5).div(65536.0).view(-1, 128))
        out["m"][at], out["sm"][tiles] = q.view(-1), s
        r = v.pow(0.5)
        q, s = _stochastic_64(r.view(-1, 128), ((h // 65536).double() + 0.5).div(65536.0).view(-1, 128))
        out["v"][at], out["sv"][tiles] = torch.where(r > 0.0, q.view(-1).clamp(min=2.0 ** -9), q.view(-1)), s
    if case["experts"]:
        E, N, K = case["experts"], case["N"], case["K"]
        w = out["p"][: E * N * K].view(E, N, K)
        out["q"] = torch.zeros_like(w)
        out["s"] = torch.zeros(st["s"].shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            for i in range(out["s"].shape[1]):
                band = w[e, 128 * i: 128 * i + 128].unflatten(1, (-1, 128))
                s = band.abs().amax(dim=(0, 2)) / E4M3_MAX
                q = _e4m3_64(torch.nan_to_num(band / s[None, :, None], nan=0.0))
                out["q"][e, 128 * i: 128 * i + 128], out["s"][e, i] = q.flatten(1), s
        if case["transposed"]:
            out["qt"], out["st"] = out["q"].transpose(1, 2), out["s"].transpose(1, 2)
    return out


# ------------------------------------------------------------------ work

def work(case):
    """Bytes each input is read and each output written once; operations counted once each (a product and a sum are two)."""
    if case["op"] == "columns":
        n, tiles = case["rows"] * case["cols"], -(-case["rows"] // 128)
        source = {"bf16": 2 * n, "f32": 4 * n, "codes": n + 4 * case["rows"] * -(-case["cols"] // 128)}[case["source"]]
        return {"bytes": source + n + 4 * tiles * case["cols"], "flops": 3.0 * n}
    if case["op"] == "wgrad":
        rows, E, N, K = (case[k] for k in ("rows", "experts", "N", "K"))
        out = (4 if case["type"] == "f32" else 2) * E * N * K * (2 if case["accumulate"] else 1)
        return {"bytes": out + (rows + 4 * -(-rows // 128)) * (N + K), "flops": 2.0 * rows * N * K}
    n = sum(_flat_layout(case)[0])
    weights = case["experts"] * case["N"] * case["K"]
    moments = 16.0 * n if case["bits"] == 32 else 4.0 * n + 16.0 * n / 128
    return {"bytes": 8.0 * n + (4 if case["type"] == "f32" else 2) * n + moments
            + weights * (2 if case["transposed"] else 1), "flops": (14.0 if case["bits"] == 32 else 26.0) * n + 3.0 * weights}
