"""The example that trains a gated feed-forward layer and serves it in 4 bits."""
import pytest

pytestmark = pytest.mark.gpu


def test_training_falls_and_four_bits_follow():
    from examples import feed_forward
    losses, error = feed_forward.main()
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert losses[-1] < 0.9 * losses[0]
    # A code is off by at most half a step, uniformly: 1 / sqrt(12) of a step of
    # a fifteenth of the group's range.  64 normal weights span about 4.7 of
    # their deviations, so a weight is off by 0.09 deviations, and so is each of
    # the two products of the block; with the down projection 0.09 * sqrt(3) =
    # 0.16 of the result.  Twice that is a failure.
    assert error < 0.32
