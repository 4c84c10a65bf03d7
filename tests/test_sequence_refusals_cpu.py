"""What the operators over sequences refuse at the ends of their ranges, without a GPU."""
import pytest

INVALID = -1


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_05_gb300 import build
    build.build()
    import newton_schulz_05_gb300 as m
    return m.load()


def test_scale_is_refused_where_its_change_of_base_overflows(lib):
    # for no tokens, so that nothing is launched where it is not refused
    def forward(scale):
        return lib.muon_token_log_probs(0, 8, 0, None, 8, None, scale, None, None, None)

    def backward(scale):
        return lib.muon_token_log_probs_backward(0, 8, 0, None, None, 8, None, None, scale, None, None)

    for call in (forward, backward):
        assert call(2.0 ** 127) == 0
        for scale in (2.0 ** 127 * 1.001, 3e38):
            assert call(scale) == INVALID
