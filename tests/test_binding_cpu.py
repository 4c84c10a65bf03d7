"""What the binding takes for the library's entry points, without a GPU."""
import ctypes

import pytest


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
