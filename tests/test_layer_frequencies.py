"""A DeltaLayer that turns by position takes its frequencies along to another device, whole and in float64. CPU only."""
import copy

import pytest

torch = pytest.importorskip("torch")

from fft_block_toeplitz_amd.layers import DeltaLayer  # noqa: E402


def want():
    return 10.0 ** (-2.0 / 8 * torch.arange(4, dtype=torch.float64))


def test_frequencies_follow_the_layer():
    layer = DeltaLayer(4, 2, 8, 8, 4, base=10.0, device="cpu")
    assert torch.equal(layer.frequencies, want())
    assert layer.to("meta").frequencies.device.type == "meta"
    made = DeltaLayer(4, 2, 8, 8, 4, base=10.0, device="meta")
    for t in (made.to_empty(device="cpu"), copy.deepcopy(made).to(torch.bfloat16), made.half().float()):
        assert torch.equal(t.frequencies, want())
    assert "frequencies" not in made.state_dict()


def test_layers_that_do_not_turn_move_too():
    layer = DeltaLayer(4, 2, 8, 8, 4, device="cpu").to("meta").to_empty(device="cpu").double()
    assert layer.frequencies is None and layer.into.weight.dtype is torch.float64
