"""Statuses and workspace sizes of the feed-forward operators at the edges of
what they take (nothing is launched, so no GPU is needed)."""
import fp8_fine_grained_x128_amd as f

FAKE = 1 << 20  # an aligned, never-dereferenced address


def test_too_wide_a_norm_is_unsupported_whatever_its_workspace():
    """No workspace holds the sums of a norm that is not implemented (its size is 0): the status names the width."""
    wide = f.NORM_MAX_COLS + 8
    assert f.fp8q_layernorm_backward_workspace(4, wide) == 0
    for ws, size in ((0, 0), (FAKE, 0), (FAKE, 1 << 30)):
        assert f.fp8q_layernorm_backward(FAKE, wide, FAKE, wide, 1, 4, wide, FAKE, 0, FAKE, FAKE, 0, None, 0, FAKE, wide, FAKE,
                                         FAKE, 0, ws, size) == f.FP8Q_EUNSUPPORTED


def test_moe_sizes_follow_the_experts_that_a_token_can_take():
    """A top_k beyond the number of experts takes all of them and needs no more memory than that."""
    size = f.fp8q_moe_decode_workspace
    for tokens, experts in ((1, 1), (3, 5), (64, 8)):
        need = size(tokens, 256, 128, experts, experts)
        assert need > 0
        for top_k in (experts + 1, 32):
            assert size(tokens, 256, 128, experts, top_k) == need
    call = dict(x=FAKE, ldx=256, T=3, H=256, logits=FAKE, ldl=5, E=5, k=7, renorm=1, I=128, w=FAKE, ldw=256, ws=256 * 256,
                s=FAKE, lds=2, ss=4, d=FAKE, ldd=128, ds=256 * 128, sd=FAKE, ldsd=1, sds=2, y=FAKE, yt=1, ldy=256,
                work=FAKE, wb=size(3, 256, 128, 5, 5) - 1)
    assert f.fp8q_moe_decode(*call.values()) == f.FP8Q_ESHAPE
