"""The mixture-of-experts layer for few tokens against a 64-bit reference:
one token to the most, one expert to many, every token on one expert, ties,
masked experts and empty slots, NaN and infinite logits, padded strides."""
import numpy as np
import pytest
import torch

from tests import ffn_ref as R
from tests.parity import say

pytestmark = pytest.mark.gpu


def _codes(rng, E, N, K, ldw=None):
    """codes [E][N][K] (row stride ldw, 0x7f between the rows) and scales [E][N/128][K/128] with a wider row stride"""
    ldw = ldw or K
    v = torch.from_numpy(np.clip(rng.standard_normal((E, N, K)) * 100, -448, 448)).float().to(torch.float8_e4m3fn)
    w = torch.full((E, N, ldw), 0x7f, dtype=torch.uint8, device="cuda")
    w[:, :, :K] = v.view(torch.uint8).cuda()
    s = torch.full((E, N // 128, K // 128 + 3), float("nan"), device="cuda")
    s[:, :, : K // 128] = torch.from_numpy(rng.uniform(0.5, 2.0, (E, N // 128, K // 128)) * 1e-3).float().cuda()
    return w[:, :, :K], s[:, :, : K // 128]


def _layer(seed, T, E, H, I, pad=0):
    rng = np.random.default_rng(seed)
    x = R.place(rng.standard_normal((T, H)), torch.bfloat16, pad)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    w_gu, s_gu = _codes(rng, E, 2 * I, H, H + 16 * pad)
    w_down, s_down = _codes(rng, E, H, I, I + 16 * pad)
    return x, logits, w_gu, s_gu, w_down, s_down


def _check(fp8q, layer, top_k, renormalize, out_dtype=torch.float32):
    x, logits, w_gu, s_gu, w_down, s_down = layer
    T, E = logits.shape
    lt = torch.full((T, E + 5), float("nan"), device="cuda")[:, :E]
    lt.copy_(torch.from_numpy(logits))
    y = fp8q.moe_decode(x, lt, w_gu, s_gu, w_down, s_down, top_k, renormalize=renormalize, out_dtype=out_dtype)
    want, err = R.moe(R.f64(x), logits.astype(np.float64), w_gu, s_gu, w_down, s_down, top_k, renormalize)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(R.f64(y)), nan)
    R.assert_close(torch.where(torch.from_numpy(nan).cuda(), 0, y), np.where(nan, 0, want), err, "y")
    again = fp8q.moe_decode(x, lt, w_gu, s_gu, w_down, s_down, top_k, renormalize=renormalize, out_dtype=out_dtype)
    assert torch.equal(y.view(torch.uint8), again.view(torch.uint8)), "not the same bits twice"
    return y


@pytest.mark.parametrize("T,E,top_k,H,I", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 512, 384), (2, 16, 4, 384, 256), (3, 5, 7, 128, 640),
    (7, 24, 3, 1024, 128), (15, 9, 2, 256, 256), (16, 64, 6, 256, 128), (17, 12, 4, 384, 128), (31, 300, 8, 256, 128),
    (33, 65, 32, 128, 128), (48, 16, 2, 640, 256), (64, 8, 8, 256, 384), (64, 256, 8, 128, 128), (5, 1000, 3, 128, 128)])
def test_against_reference(fp8q, T, E, top_k, H, I):
    say(f"moe T={T} E={E} k={top_k} H={H} I={I}")
    layer = _layer(T + E, T, E, H, I, pad=(T + E) % 3)
    _check(fp8q, layer, top_k, renormalize=bool((T + top_k) % 2))


@pytest.mark.parametrize("T,top_k", [(19, 14), (32, 8), (33, 20), (64, 8), (64, 17)])
def test_enough_work_for_the_wide_variants(fp8q, T, top_k):
    """64 experts of 1024/512 are two work-groups of eight row tiles for every compute unit."""
    say(f"moe wide T={T} k={top_k}")
    _check(fp8q, _layer(T + top_k, T, 64, 1024, 512, pad=T % 2), top_k, T % 2 == 0)


@pytest.mark.parametrize("T", [17, 32, 33, 48, 49, 64])
def test_full_and_partial_token_groups(fp8q, T):
    """Every token on each of the experts: two to four groups of 16, the last one full or not."""
    say(f"moe groups T={T}")
    for E in (2, 6):
        _check(fp8q, _layer(T, T, E, 384, 256), E, True)
    layer = _layer(T, T, 12, 256, 384)  # one expert for all, the others few tokens each
    layer[1][:, 5] = 60.0
    _check(fp8q, layer, 3, False)


@pytest.mark.parametrize("T", [1, 16, 64])
def test_bf16_output(fp8q, T):
    say(f"moe bf16 T={T}")
    _check(fp8q, _layer(T, T, 32, 512, 256), 4, True, torch.bfloat16)


@pytest.mark.parametrize("T", [1, 20, 64])
def test_every_token_on_the_same_experts(fp8q, T):
    say(f"moe one pair of experts for all {T} tokens")
    layer = _layer(T, T, 16, 256, 256)
    layer[1][:, 3] = 50.0
    layer[1][:, 11] = 49.0
    _check(fp8q, layer, 2, True)


@pytest.mark.parametrize("T", [2, 8, 9, 40])
def test_an_experts_nan_reaches_only_its_tokens(fp8q, T):
    say(f"moe NaN weights T={T}")
    x, logits, w_gu, s_gu, w_down, s_down = _layer(T, T, 8, 256, 256)
    logits[:, 2:4] = -np.inf
    logits[0, 2:4] = 5.0
    lt = torch.from_numpy(logits).cuda()
    clean = fp8q.moe_decode(x, lt, w_gu, s_gu, w_down, s_down, 2)
    w_gu[2, 7, 3] = 0x7f
    w_down[2, 5, 9] = 0xff
    s_down[3, 1, 1] = float("inf")
    y = fp8q.moe_decode(x, lt, w_gu, s_gu, w_down, s_down, 2)
    assert bool(torch.isnan(y[0]).any())
    assert torch.equal(y[1:], clean[1:])


def test_ties_masks_and_empty_rows(fp8q):
    """Equal logits (all of them, and around the last place), -0 beside 0, masked experts, fewer candidates than
    top_k, rows of -inf, the lowest finite values."""
    say("moe ties and masks")
    T, E = 12, 80
    layer = _layer(4, T, E, 256, 128)
    l = layer[1]
    low = np.finfo(np.float32).min
    l[0] = 0.25
    l[1] = np.where(np.arange(E) % 2 == 0, -0.0, 0.0)
    l[2] = np.round(l[2])
    l[3, :] = -np.inf
    l[4, :] = -np.inf
    l[4, [70, 5]] = [1.0, 2.0]
    l[5, ::2] = -np.inf
    l[6] = low
    l[7] = low
    l[7, 79] = -np.inf
    l[7, 64] = 3.0
    l[8] = -np.inf
    l[8, 79] = low
    l[9] = np.repeat([1.0, 2.0, 3.0, 4.0], 20)
    l[10] *= 1e30
    y = _check(fp8q, layer, 4, True)
    assert not y[3].any() and bool(y[4].any())
    _check(fp8q, layer, 4, False)


def test_nan_and_infinite_logits_stay_in_their_rows(fp8q):
    say("moe non-finite logits")
    layer = _layer(6, 6, 70, 256, 128)
    l = layer[1]
    l[1, 68] = np.nan
    l[3, 0] = np.inf
    l[4, 9] = -np.inf
    y = _check(fp8q, layer, 3, True)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all()) and bool(torch.isfinite(y[0]).all())


def test_nan_activations_stay_in_their_rows(fp8q):
    say("moe NaN activations")
    layer = _layer(7, 20, 8, 256, 128)
    clean = _check(fp8q, layer, 2, True)
    layer[0][13, 100] = float("nan")
    lt = torch.from_numpy(layer[1]).cuda()
    y = fp8q.moe_decode(layer[0], lt, *layer[2:], 2, out_dtype=torch.float32)
    assert bool(torch.isnan(y[13]).all())
    keep = [t for t in range(20) if t != 13]
    assert torch.equal(y[keep], clean[keep])


def test_no_tokens_and_side_stream(fp8q):
    say("moe: no tokens, another stream")
    layer = _layer(9, 4, 8, 256, 128)
    lt = torch.from_numpy(layer[1]).cuda()
    y = fp8q.moe_decode(layer[0], lt, *layer[2:], 2)
    assert fp8q.moe_decode(layer[0][:0], lt[:0], *layer[2:], 2).shape == (0, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = fp8q.moe_decode(layer[0], lt, *layer[2:], 2)
    side.synchronize()
    assert torch.equal(y, z)


def test_expert_stride_past_32_bits(fp8q):
    """Experts whose codes lie beyond 2^32 bytes."""
    say("moe: far experts")
    rng = np.random.default_rng(11)
    x, logits, w_gu, s_gu, w_down, s_down = _layer(11, 3, 3, 256, 128)
    far = torch.zeros(2 * (3 << 30) + 256 * 256, dtype=torch.uint8, device="cuda").as_strided((3, 256, 256), (3 << 30, 256, 1))
    far.copy_(w_gu)
    lt = torch.from_numpy(logits).cuda()
    a = fp8q.moe_decode(x, lt, w_gu, s_gu, w_down, s_down, 2)
    b = fp8q.moe_decode(x, lt, far, s_gu, w_down, s_down, 2)
    assert torch.equal(a, b)
