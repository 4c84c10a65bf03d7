"""What the binding takes for the library's entry points and for tensors, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_05_gb300 import build
    build.build()
    import newton_schulz_05_gb300 as m
    return m.load()


def test_entry_points_that_are_missing_or_not_known_are_refused(lib):
    from newton_schulz_05_gb300 import layers
    binding = layers._b()
    real = {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in layers._ENTRY_POINTS}
    first = {n: real[n] for n in layers._ENTRY_POINTS[:7]}
    try:
        for n in real:
            with pytest.raises(ValueError):
                binding.bind({m: p for m, p in real.items() if m != n})
            with pytest.raises(ValueError):
                binding.bind(dict(real, **{n: 0}))
        for bad in ({}, dict(real, muon_dropuot=real["muon_dropout"]), dict(first, muon_gated_scna=real["muon_gated_scan"])):
            with pytest.raises(ValueError):
                binding.bind(bad)
        with pytest.raises((TypeError, ValueError)):
            binding.bind(None)
        binding.bind(first)      # those over sequences keep what they are bound to
    finally:
        binding.bind(real)


def test_what_is_no_tensor_is_refused_as_such():
    from newton_schulz_05_gb300 import layers
    x = torch.zeros(3, 2, 8)
    for call in (lambda: layers.layer_norm(x, [1.0] * 8), lambda: layers.dropout_add_layer_norm(x, x, None, 0.5, p=0.1, seed=1),
                 lambda: layers.norm_rotate_heads(x, x, [1.0] * 8), lambda: layers.norm_rotate_heads(x, cos=1, sin=1),
                 lambda: layers.gated_scan(x, x, state=0.0), lambda: layers.policy_loss(x, x, x, token_mask=True)):
        with pytest.raises(TypeError, match="must be a tensor"):
            call()
