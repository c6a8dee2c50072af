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
