"""The decoder layers that bench.py times compute real numbers."""
import types

import pytest

pytestmark = pytest.mark.gpu


def test_timed_decoder_layers_stay_finite(monkeypatch):
    """Four layers (an unnormalised stream through them is infinite in the third)."""
    import torch

    import bench
    from ternary_weight_02_b200 import bonsai as bz
    monkeypatch.setattr(bench, "LAYERS", 4)
    dev = torch.device("cuda", torch.cuda.current_device())
    stack, _, _ = bench.build_stack(2, bench.base_planes(2, dev, bz, torch), dev, torch)
    out = bench.measure_decode_layers(2, stack, bz, torch, torch.cuda.Stream(), dev, types.SimpleNamespace(context=700, steps=3),
                                      6534.5)
    for part in ("step", "attention"):
        assert out[part]["us"] > 0
        for name, rms in out[part]["rms"].items():
            assert 0 < rms < 1000, (part, name, rms)


def test_values_that_are_not_finite_are_refused():
    import torch

    import bench
    assert bench.finite_rms(torch, "x", torch.full((4,), 3.0)) == 3.0
    for bad in (float("nan"), float("inf")):
        with pytest.raises(FloatingPointError):
            bench.finite_rms(torch, "x", torch.tensor([1.0, bad]))
