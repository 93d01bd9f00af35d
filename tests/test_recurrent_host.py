"""The recurrent layer's parts that run without a GPU."""
import pytest
import torch

from depthwise_convolution_grouped_amd import recurrent


@pytest.mark.parametrize("lengths", [None, [5, 0, 1, 3], [-4, 6, 8, 2 ** 31 - 1]])
@pytest.mark.parametrize("taps", [1, 2, 4, 9])
def test_last_inputs(lengths, taps):
    """Whatever the lengths, every row read lies inside u; they count clamped to [0, L]."""
    B, L, D = 4, 5, 3
    u = torch.randn(B, L, D, generator=torch.Generator().manual_seed(taps))
    got = recurrent.last_inputs(u, taps, None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    assert got.shape == (B, taps - 1, D)
    for b in range(B):
        n = L if lengths is None else min(max(lengths[b], 0), L)
        want = torch.cat([torch.zeros(taps - 1, D), u[b, :n]])[n:]
        assert torch.equal(got[b], want)
