"""Operands and weight gradients of rows grouped by expert against the oracle's quantizers and 64-bit sums."""
import numpy as np
import pytest
import torch

from tests import expert_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _x(rows, cols, dtype, seed, scale=1.0):
    """Row stride a multiple of 16 bytes, values over several binades, some zeros."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-3, 3, (1, cols))) * scale
    v[rng.random((rows, cols)) < 0.02] = 0.0
    per = 16 // dtype.itemsize
    buf = torch.zeros((rows, -(-max(cols, 1) // per) * per), dtype=dtype, device=DEV)
    buf[:, :cols] = torch.from_numpy(v).to(DEV)
    return buf[:, :cols]


OFFSETS = {  # rows, offsets: sizes around a chunk, empty groups first, last and between
    "one": (1, [0, 1]),
    "chunk": (128, [0, 128]),
    "around": (515, [0, 127, 255, 384, 515]),
    "empty": (300, [0, 0, 0, 129, 129, 130, 300, 300]),
    "inside": (400, [17, 60, 60, 333]),  # rows before and behind the groups
    "none": (50, [0, 0, 0]),
}


def _many(G, rows, seed):
    rng = np.random.default_rng(seed)
    return rows, np.concatenate([[0], np.sort(rng.integers(0, rows + 1, G - 1)), [rows]]).tolist()


OFFSETS["many"] = _many(200, 3000, 5)
OFFSETS["most"] = _many(1024, 2000, 6)
OFFSETS["wild"] = (300, [-5, 100, 40, 90, 1 << 30, 200, -(1 << 31)])


def _offsets(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def _check_operand(o, parts, cols, off):
    """parts: per group (codes [n][cols], scales [chunks][cols]) of the oracle"""
    q, s = o.q.cpu().numpy(), o.s.cpu().numpy()
    first = R.first_chunks(off)
    assert q.shape[1] % 128 == 0 and q.shape[1] >= 128 * first[-1] and s.shape == (q.shape[1] // 128, cols)
    for g, (qo, so) in enumerate(parts):
        n, at = qo.shape[0], 128 * first[g]
        assert np.array_equal(q[:, at: at + n], qo.T), f"codes of group {g}"
        assert not q[:, at + n: 128 * first[g + 1]].any(), f"padding of group {g}"
        assert np.array_equal(s[first[g]: first[g + 1]], so), f"scales of group {g}"


@pytest.mark.parametrize("name", list(OFFSETS))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [1, 130, 256])
def test_quantized_columns(fp8q, oracle, name, dtype, cols):
    rows, raw = OFFSETS[name]
    x = _x(rows, cols, dtype, 1)
    o = fp8q.grouped_quantize_act(x, _offsets(raw))
    off = R.clamped(raw, rows)
    xs = x.float().cpu().numpy()
    parts = [oracle.quantize_act_128x1(np.ascontiguousarray(xs[a:b])) if b > a
             else (np.zeros((0, cols), np.uint8), np.zeros((0, cols), np.float32)) for a, b in zip(off, off[1:])]
    _check_operand(o, parts, cols, off)


@pytest.mark.parametrize("name", list(OFFSETS))
@pytest.mark.parametrize("cols", [128, 300])
def test_requantized_columns(fp8q, oracle, name, cols):
    rows, raw = OFFSETS[name]
    q, s = fp8q.quantize_act(_x(rows, cols, torch.bfloat16, 2))
    o = fp8q.grouped_requant_transpose(q, s, _offsets(raw))
    off = R.clamped(raw, rows)
    qn, sn = q.cpu().numpy(), s.cpu().numpy()
    parts = [oracle.requant_1x128_to_128x1(np.ascontiguousarray(qn[a:b]), np.ascontiguousarray(sn[:, a:b].T)) if b > a
             else (np.zeros((0, cols), np.uint8), np.zeros((0, cols), np.float32)) for a, b in zip(off, off[1:])]
    _check_operand(o, parts, cols, off)


@pytest.mark.parametrize("aligned", [[0, 128, 512, 640], [0, 0, 640]])
def test_aligned_groups_are_the_plain_layout(fp8q, aligned):
    x = _x(640, 200, torch.bfloat16, 3)
    for mode in (fp8q.FP8Q_SCALE_FP32, fp8q.FP8Q_SCALE_POW2):
        o = fp8q.grouped_quantize_act(x, _offsets(aligned), scale_mode=mode)
        q, s = fp8q.quantize_act(x, fp8q.FP8Q_TILE_128x1, scale_mode=mode)
        assert torch.equal(o.q[:, :640], q) and torch.equal(o.s[:5], s)


def test_power_of_two_scales_per_group(fp8q):
    rows, raw = OFFSETS["around"]
    x = _x(rows, 130, torch.float32, 4)
    o = fp8q.grouped_quantize_act(x, _offsets(raw), scale_mode=fp8q.FP8Q_SCALE_POW2)
    first = R.first_chunks(np.array(raw))
    for g, (a, b) in enumerate(zip(raw, raw[1:])):
        q, s = fp8q.quantize_act(x[a:b], fp8q.FP8Q_TILE_128x1, scale_mode=fp8q.FP8Q_SCALE_POW2)
        assert torch.equal(o.q[:, 128 * first[g]: 128 * first[g] + b - a], q)
        assert torch.equal(o.s[first[g]: first[g + 1]], s)


def test_columns_write_nothing_else(fp8q):
    """Columns past the last chunk, scales past it and what stands around the arrays keep their values."""
    rows, cols, raw = 300, 130, [0, 129, 129, 200]
    x = _x(rows, cols, torch.bfloat16, 5)
    ld = fp8q.fp8q_grouped_padded_rows(rows, 3) + 16
    q = torch.full((cols + 2, ld), 0x5A, dtype=torch.uint8, device=DEV)
    s = torch.full((ld // 128 + 3, cols + 5), 7.0, dtype=torch.float32, device=DEV)
    assert fp8q.fp8q_grouped_quantize_act(x.data_ptr(), 1, rows, cols, x.stride(0), _offsets(raw).data_ptr(), 3,
                                          q[1:].data_ptr(), ld, s[1:].data_ptr(), cols + 5, 0,
                                          torch.cuda.current_stream().cuda_stream) == 0
    qn, sn = q.cpu(), s.cpu()
    assert (qn[0] == 0x5A).all() and (qn[cols + 1] == 0x5A).all() and (qn[1: cols + 1, 384:] == 0x5A).all()
    assert (sn[0] == 7.0).all() and (sn[4:] == 7.0).all() and (sn[1:4, cols:] == 7.0).all()
    assert (qn[1: cols + 1, 129: 256] == 0).all()
    assert (sn[1:4, :cols] != 7.0).all()  # written; a chunk of one row has a zero scale where its value is zero


def test_columns_past_32_bits(fp8q):
    """Inputs and codes of more than 2^31 elements: the last group's last columns, against its rows alone."""
    rows, cols, at = 70001, 32768, 69003
    offs, tail = _offsets([0, at, rows]), slice(cols - 130, cols)
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[at:] = _x(rows - at, cols, torch.bfloat16, 24)
    first = 128 * -(-at // 128)
    o = fp8q.grouped_quantize_act(x, offs)
    q, s = fp8q.quantize_act(x[at:], fp8q.FP8Q_TILE_128x1)
    assert torch.equal(o.q[tail, first: first + rows - at], q[tail]) and not o.q[tail, at - 500: first].any()
    assert torch.equal(o.s[first // 128:, tail][: s.shape[0]], s[:, tail])
    q, s = fp8q.quantize_act(x)
    o = fp8q.grouped_requant_transpose(q, s, offs)
    q, s = fp8q.requant_transpose(q[at:], s[:, at:].contiguous())
    assert torch.equal(o.q[tail, first: first + rows - at], q[tail]) and not o.q[tail, at - 500: first].any()
    assert torch.equal(o.s[first // 128:, tail][: s.shape[0]], s[:, tail])


# ------------------------------------------------------------------ the product

def _operand(fp8q, rows, off, width, seed, scale):
    """Codes over the whole range, NaN codes and NaN scales where nothing may be read."""
    rng = np.random.default_rng(seed)
    first = R.first_chunks(off)
    cap = fp8q.fp8q_grouped_padded_rows(rows, len(off) - 1)
    q = np.full((width, cap), 0x7F, dtype=np.uint8)
    s = np.full((cap // 128, width), np.nan, dtype=np.float32)
    for g in range(len(off) - 1):
        at, end, n = 128 * first[g], 128 * first[g + 1], off[g + 1] - off[g]
        c = rng.integers(0, 256, (width, end - at)).astype(np.uint8)
        c[(c & 0x7F) == 0x7F] = 0
        c[:, n:] = 0
        q[:, at:end] = c
    s[: first[-1]] = rng.uniform(0.5, 2.0, (first[-1], width)).astype(np.float32) * np.float32(scale)
    return fp8q.GroupedOperand(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), rows), q, s


def _check_dw(got, dw, t, dtype, tol=1e-5):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    bound = tol * t
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(dw) + tol * t)
    bad = np.abs(got - dw) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.max(np.abs(got - dw) / np.maximum(bound, 1e-300))))


@pytest.mark.parametrize("name", list(OFFSETS))
@pytest.mark.parametrize("N,K", [(1, 1), (64, 200), (333, 130)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad(fp8q, name, N, K, dtype):
    rows, raw = OFFSETS[name]
    if len(raw) > 500 and N * K > 20000:
        N = 40
    off = R.clamped(raw, rows)
    dy, qa, sa = _operand(fp8q, rows, off, N, 7, 1e-3)
    x, qb, sb = _operand(fp8q, rows, off, K, 8, 0.1)
    dw, t = R.wgrad(qa, sa, qb, sb, off)
    got = fp8q.grouped_wgrad(dy, x, _offsets(raw), out_dtype=dtype)
    assert got.shape == (len(off) - 1, N, K)
    _check_dw(got, dw, t, dtype)
    assert torch.equal(got, fp8q.grouped_wgrad(dy, x, _offsets(raw), out_dtype=dtype))


@pytest.mark.parametrize("G,rows,N,K", [(2, 5000, 128, 128), (3, 2000, 520, 260), (1, 4096, 256, 300),
                                        (40, 1500, 300, 520), (5, 700, 1040, 770)])
def test_wgrad_shapes(fp8q, G, rows, N, K):
    """Long contractions of few tiles, and tiles enough to fill the GPU."""
    rows, raw = _many(G, rows, G)
    off = R.clamped(raw, rows)
    dy, qa, sa = _operand(fp8q, rows, off, N, 9, 1e-3)
    x, qb, sb = _operand(fp8q, rows, off, K, 10, 0.1)
    start = np.random.default_rng(11).standard_normal((G, N, K)).astype(np.float32)
    dw, t = R.wgrad(qa, sa, qb, sb, off)
    offs = _offsets(raw)
    _check_dw(fp8q.grouped_wgrad(dy, x, offs), dw, t, torch.float32)
    acc = torch.from_numpy(start).to(DEV)
    out = fp8q.grouped_wgrad(dy, x, offs, dw=acc, accumulate=True)
    assert out is acc
    _check_dw(acc, dw + start, t + np.abs(start), torch.float32)
    _check_dw(fp8q.grouped_wgrad(dy, x, offs, out_dtype=torch.bfloat16), dw, t, torch.bfloat16)


@pytest.mark.parametrize("G,rows,N,K", [(4, 300, 2000, 4076), (4, 300, 2000, 4075), (3, 9000, 333, 130),
                                        (6, 40000, 640, 520), (300, 900, 140, 130), (20, 2500, 700, 520)])
def test_wgrad_cuts(fp8q, G, rows, N, K):
    """Large tiles past both ends of the gradient; groups in slices, several a work-group; more groups than are taken
    by size; groups by size."""
    rows, raw = _many(G, rows, G)
    off = R.clamped(raw, rows)
    dy, qa, sa = _operand(fp8q, rows, off, N, 21, 1e-3)
    x, qb, sb = _operand(fp8q, rows, off, K, 22, 0.1)
    dw, t = R.wgrad(qa, sa, qb, sb, off)
    offs = _offsets(raw)
    one = fp8q.grouped_wgrad(dy, x, offs)
    _check_dw(one, dw, t, torch.float32)
    assert torch.equal(fp8q.grouped_wgrad(dy, x, offs, dw=one.clone(), accumulate=True), one + one)
    _check_dw(fp8q.grouped_wgrad(dy, x, offs, out_dtype=torch.bfloat16), dw, t, torch.bfloat16)


def test_wgrad_strided_output(fp8q):
    """Row and group strides of odd lengths; what lies between the rows stays."""
    rows, raw = OFFSETS["empty"]
    off = R.clamped(raw, rows)
    G, N, K = len(raw) - 1, 70, 131
    dy, qa, sa = _operand(fp8q, rows, off, N, 12, 1e-3)
    x, qb, sb = _operand(fp8q, rows, off, K, 13, 0.1)
    dw, t = R.wgrad(qa, sa, qb, sb, off)
    for ld, dtype in ((137, torch.float32), (136, torch.float32), (137, torch.bfloat16), (136, torch.bfloat16)):
        buf = torch.full((G, N + 1, ld), 9.0, dtype=dtype, device=DEV)
        out = buf[:, :N, :K]
        fp8q.grouped_wgrad(dy, x, _offsets(raw), dw=out)
        _check_dw(out, dw, t, dtype)
        assert (buf[:, N] == 9.0).all() and (buf[:, :, K:] == 9.0).all()


@pytest.mark.parametrize("flags", [1, 2, 3])
def test_wgrad_datapaths(fp8q, flags):
    rows, raw = OFFSETS["around"]
    x = _x(rows, 300, torch.bfloat16, 14)
    dy = _x(rows, 140, torch.bfloat16, 15, 1e-3)
    offs = _offsets(raw)
    a = fp8q.grouped_quantize_act(dy, offs, scale_mode=fp8q.FP8Q_SCALE_POW2)
    b = fp8q.grouped_quantize_act(x, offs, scale_mode=fp8q.FP8Q_SCALE_POW2)
    dw, t = R.wgrad(*(v.cpu().numpy() for v in (a.q, a.s, b.q, b.s)), np.array(raw))
    for dtype in (torch.float32, torch.bfloat16):
        _check_dw(fp8q.grouped_wgrad(a, b, offs, out_dtype=dtype, flags=flags), dw, t, dtype,
                  tol=1e-5 + (2.0 ** -10 if flags & 1 else 0.0))


def test_wgrad_of_the_longest_rows(fp8q):
    """Offsets inside an operand past 32 bits: as many tokens as the product takes, few of them not zero."""
    rows, N, K, raw = (1 << 24) - 256, 256, 20, [0, 12345, (1 << 24) - 256]
    cap = fp8q.fp8q_grouped_padded_rows(rows, 2)
    first = R.first_chunks(np.array(raw))
    assert cap == 128 * first[-1] == (1 << 24) - 128
    q = [torch.zeros((n, cap), dtype=torch.uint8, device=DEV) for n in (N, K)]
    s = [torch.ones((cap // 128, n), dtype=torch.float32, device=DEV) for n in (N, K)]
    want = torch.zeros((2, N, K))
    one = 0x38  # 1.0
    for g, n, k, at, scale in ((0, 0, 0, 5, 2.0), (0, 255, 19, 12344, 3.0), (1, 255, 0, 128 * first[1], 5.0),
                               (1, 127, 7, 128 * (first[2] - 1), 7.0), (1, 255, 19, 128 * first[2] - 130, 11.0)):
        q[0][n, at], q[1][k, at] = one, one
        s[0][at // 128, n] = scale
        want[g, n, k] += scale
    dy, x = (fp8q.GroupedOperand(a, b, rows) for a, b in zip(q, s))
    assert torch.equal(fp8q.grouped_wgrad(dy, x, _offsets(raw)).cpu(), want)


def test_wgrad_refuses_strided_codes_of_one_channel(fp8q):
    offs = _offsets([0, 200])
    one, other = (fp8q.grouped_quantize_act(_x(200, n, torch.bfloat16, 23), offs) for n in (1, 40))
    apart = fp8q.GroupedOperand(torch.zeros((1, 2 * one.q.shape[1]), dtype=torch.uint8, device=DEV)[:, ::2], one.s, 200)
    for dy, x in ((apart, other), (other, apart)):
        with pytest.raises(ValueError, match="unit column stride"):
            fp8q.grouped_wgrad(dy, x, offs)
    assert fp8q.grouped_wgrad(one, other, offs).shape == (1, 1, 40)


def test_wgrad_of_no_rows(fp8q):
    o = fp8q.grouped_quantize_act(torch.empty((0, 64), device=DEV), _offsets([0, 0, 0]))
    assert o.q.shape == (64, 0) and o.s.shape == (0, 64)
    got = fp8q.grouped_wgrad(o, o, _offsets([0, 0, 0]))
    assert got.shape == (2, 64, 64) and not got.any()
    acc = torch.ones((2, 64, 64), device=DEV)
    fp8q.grouped_wgrad(o, o, _offsets([0, 0, 0]), dw=acc, accumulate=True)
    assert (acc == 1).all()


def test_wgrad_matches_the_plain_gemm_of_one_group(fp8q):
    """One group of whole chunks is the Wgrad GEMM, bit for bit where neither splits the contraction."""
    x, dy = _x(512, 384, torch.bfloat16, 16), _x(512, 256, torch.bfloat16, 17, 1e-3)
    offs = _offsets([0, 512])
    a, b = fp8q.grouped_quantize_act(dy, offs), fp8q.grouped_quantize_act(x, offs)
    qa, sa = fp8q.quantize_act(dy, fp8q.FP8Q_TILE_128x1)
    qb, sb = fp8q.quantize_act(x, fp8q.FP8Q_TILE_128x1)
    want = fp8q.gemm(qa, sa, qb, sb, bscale=fp8q.FP8Q_BSCALE_ROW, out_dtype=torch.float32, split_k=False)
    got = fp8q.grouped_wgrad(a, b, offs)[0]
    t = (fp8q.gemm(qa & 0x7F, sa, qb & 0x7F, sb, bscale=fp8q.FP8Q_BSCALE_ROW, out_dtype=torch.float32))
    assert ((got - want).abs() <= 2e-6 * t).all()


def test_gradient_of_the_grouped_product_by_differences(fp8q):
    """d/dW of sum(dY * (X W^T)) for dequantized operands, against differences of that sum in 64 bits (it is linear in
    W, so a difference has no error but rounding)."""
    rows, raw, N, K = 200, [0, 70, 70, 200], 24, 40
    offs = _offsets(raw)
    a = fp8q.grouped_quantize_act(_x(rows, N, torch.float32, 18, 1e-2), offs)
    b = fp8q.grouped_quantize_act(_x(rows, K, torch.float32, 19), offs)
    got = fp8q.grouped_wgrad(a, b, offs).double().cpu().numpy()
    first = R.first_chunks(np.array(raw))
    qa, sa, qb, sb = (v.cpu().numpy() for v in (a.q, a.s, b.q, b.s))
    w = np.random.default_rng(20).standard_normal((3, N, K))

    def loss(w):
        total = 0.0
        for g in range(3):
            for c in range(first[g], first[g + 1]):
                dy = e = R.e4m3(qa[:, 128 * c: 128 * c + 128]) * sa[c][:, None]
                x = R.e4m3(qb[:, 128 * c: 128 * c + 128]) * sb[c][:, None]
                total += float((e.T * (x.T @ w[g].T)).sum())
        return total

    _, t = R.wgrad(qa, sa, qb, sb, np.array(raw))
    for g, n, k in ((0, 0, 0), (0, 23, 39), (1, 5, 5), (2, 7, 11), (2, 23, 0)):
        up, down = w.copy(), w.copy()
        up[g, n, k] += 1.0
        down[g, n, k] -= 1.0
        diff = (loss(up) - loss(down)) / 2
        assert abs(got[g, n, k] - diff) <= 1e-5 * t[g, n, k] + 1e-9
