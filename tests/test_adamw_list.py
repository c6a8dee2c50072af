"""The list of tensors that an AdamW step keeps: parameters whose memory was replaced are refused (no GPU needed)."""
import pytest
import torch

from fp8_fine_grained_x128_amd import binding


@pytest.mark.parametrize("one_call", [True, False])
def test_parameters_that_moved(monkeypatch, one_call):
    if not one_call:
        monkeypatch.setattr(binding, "_same_addresses", None)
    params = [torch.nn.Parameter(torch.zeros(100 + i)) for i in range(5)] + [torch.zeros(0)]
    args = (params, [p.data_ptr() for p in params], list(range(6)))
    binding._not_moved(*args)
    with torch.no_grad():
        params[2].add_(1)  # in place
    binding._not_moved(*args)
    kept = params[3].data
    params[3].data = torch.zeros(103)
    with pytest.raises(ValueError, match="parameter 3 has other memory"):
        binding._not_moved(*args)
    params[3].data = kept
    binding._not_moved(*args)
    params[1].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="parameter 1 has other memory"):
        binding._not_moved(*args)


def test_a_list_keeps_the_memory():
    """Memory that a tensor of the list gives up is not reused while the list is there."""
    p, g = torch.zeros(256, 128), torch.zeros(256, 128)
    st = binding.AdamwState(*(torch.zeros(256 * 128, dtype=torch.uint8) for _ in range(2)),
                            *(torch.zeros(256) for _ in range(2)))
    c = binding.WeightCodes(torch.zeros(256, 128, dtype=torch.uint8), torch.zeros(2, 1), None, None)
    held = ((p, g), (g, g), (st, binding.AdamwState(g, g, None, None)), (c, None))
    tensors = [p, g, *st, c.q, c.s]
    kept = binding.AdamwTensors(held, None, 0, 8, p.device)
    addresses = {t.data_ptr() for t in tensors}
    assert addresses <= {s.data_ptr() for s in kept.memory}
    for t in tensors:
        t.data = torch.empty(0, dtype=t.dtype)
    later = [torch.empty(n, dtype=torch.uint8) for n in (4 * 256 * 128, 256 * 128, 1024, 8) for _ in range(50)]
    assert not addresses & {t.data_ptr() for t in later}
