"""The weight gradients of groups on every datapath, in every way that they are cut and stored."""
import numpy as np
import pytest
import torch

from tests import expert_ref as R
from tests.test_gpu_grouped_wgrad import DEV, _check_dw, _many, _offsets, _operand

pytestmark = pytest.mark.gpu

CASES = {  # groups, rows, N, K
    "large": (4, 300, 2000, 4096),        # 256x256 tiles in whole rows of 16 bytes, two jobs a work-group
    "large, last": (4, 300, 2000, 4040),  # the same, the last columns' tiles element by element
    "slices": (3, 9000, 336, 136),        # 128x128 tiles of groups in slices, and the join
    "small": (20, 2500, 704, 520),        # 128x128 tiles, more jobs than fit at once
}


def _cut(fp8q, name):
    """The case is cut as its name says (the rules at the kernel's plan, for this device)."""
    G, rows, N, K = CASES[name]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-N // 256) * -(-K // 256)
    rounds = -(-tiles * G // cus)
    large = 2 * tiles >= cus and 100 * G * N * K >= 75 * rounds * cus * 65536
    assert large == name.startswith("large")
    assert (fp8q.fp8q_grouped_wgrad_workspace(rows, G, N, K) > 0) == (name == "slices")
    if large:
        assert rounds > 1


def _pow2_operand(fp8q, rows, off, width, seed, exponents):
    o, q, s = _operand(fp8q, rows, off, width, seed, 1.0)
    live = np.isfinite(s)
    s[live] = 2.0 ** np.random.default_rng(seed).integers(*exponents, live.sum())
    return o._replace(s=torch.from_numpy(s).to(DEV)), q, s


@pytest.mark.parametrize("name", list(CASES))
def test_datapaths(fp8q, name):
    _cut(fp8q, name)
    G, rows, N, K = CASES[name]
    rows, raw = _many(G, rows, G)
    off = R.clamped(raw, rows)
    dy, qa, sa = _pow2_operand(fp8q, rows, off, N, 81, (-14, -6))
    x, qb, sb = _pow2_operand(fp8q, rows, off, K, 82, (-6, 2))
    dw, t = R.wgrad(qa, sa, qb, sb, off)
    start = (np.random.default_rng(83).standard_normal((G, N, K)) * np.abs(dw).mean()).astype(np.float32)
    offs = _offsets(raw)
    for flags in range(4):
        print(f"flags {flags}", flush=True)
        tol = 1e-5 + (2.0 ** -10 if flags & fp8q.FP8Q_GEMM_MMA_FP8 else 0.0)
        one = fp8q.grouped_wgrad(dy, x, offs, flags=flags)
        _check_dw(one, dw, t, torch.float32, tol)
        acc = torch.from_numpy(start).to(DEV)
        assert fp8q.grouped_wgrad(dy, x, offs, dw=acc, accumulate=True, flags=flags) is acc
        assert torch.equal(acc, torch.from_numpy(start).to(DEV) + one)  # the sum is rounded once
        half = fp8q.grouped_wgrad(dy, x, offs, out_dtype=torch.bfloat16, flags=flags)
        assert torch.equal(half, one.to(torch.bfloat16))
        for dtype, want in ((torch.float32, one), (torch.bfloat16, half)):
            assert torch.equal(fp8q.grouped_wgrad(dy, x, offs, out_dtype=dtype, flags=flags), want)


@pytest.mark.parametrize("flags", range(4))
@pytest.mark.parametrize("dtype,add", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
def test_large_tiles_write_nothing_around(fp8q, flags, dtype, add):
    """Rows of a larger array, whole rows of 16 bytes: what lies between and behind them stays."""
    G, rows, N, K = CASES["large"]
    rows, raw = _many(G, rows, G)
    off = R.clamped(raw, rows)
    dy, x = (_pow2_operand(fp8q, rows, off, n, 84, (-6, 2))[0] for n in (N, K))
    want = fp8q.grouped_wgrad(dy, x, _offsets(raw), out_dtype=dtype, flags=flags)
    buf = torch.full((G, N + 1, K + 8), 9.0, dtype=dtype, device=DEV)
    out = buf[:, :N, :K]
    if add:
        out.zero_()
    fp8q.grouped_wgrad(dy, x, _offsets(raw), dw=out, accumulate=add, flags=flags)
    assert torch.equal(out, want)
    assert (buf[:, N] == 9.0).all() and (buf[:, :, K:] == 9.0).all()


def test_one_group_is_the_plain_gemm_bit_for_bit(fp8q):
    """One group of whole chunks that neither call splits: the same chunks in the same order."""
    rows, N, K = 512, 2048, 4096
    assert fp8q.fp8q_grouped_wgrad_workspace(rows, 1, N, K) == 0 and fp8q.fp8q_gemm_splitk_workspace(N, K, rows) == 0
    torch.manual_seed(85)
    dy, x = torch.randn((rows, N), device=DEV) * 1e-3, torch.randn((rows, K), device=DEV)
    for mode, all_flags in ((fp8q.FP8Q_SCALE_FP32, (0, 1)), (fp8q.FP8Q_SCALE_POW2, (2, 3))):
        a, b = (fp8q.grouped_quantize_act(v, _offsets([0, rows]), scale_mode=mode) for v in (dy, x))
        for flags in all_flags:
            want = fp8q.gemm(a.q, a.s, b.q, b.s, bscale=fp8q.FP8Q_BSCALE_ROW, out_dtype=torch.float32, split_k=False,
                             flags=flags)
            assert torch.equal(fp8q.grouped_wgrad(a, b, _offsets([0, rows]), flags=flags)[0], want)
