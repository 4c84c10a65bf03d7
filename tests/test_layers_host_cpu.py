"""Host side of the training operators without a GPU: offsets of dropout calls
under recomputation."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint


@pytest.mark.parametrize("reentrant", [True, False])
def test_counter_refuses_to_move_in_a_recomputed_forward_pass(reentrant):
    from newton_schulz_05_gb300.layers import RandomCounter
    rng = RandomCounter(3)

    def inside(x):
        rng.take(x.numel())
        return (x * x).sin()

    x = torch.randn(16, requires_grad=True)
    y = checkpoint(inside, x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="recompute"):
        y.sum().backward()
    assert rng.offset == 2
    # the offset taken outside and passed in is the way
    seen = []

    def outside(x, at):
        seen.append(at)
        return (x * x).sin()

    checkpoint(outside, x, rng.take(x.numel()), use_reentrant=reentrant).sum().backward()
    assert seen == [2, 2] and rng.take(8) == 4
