"""The example layer: router, experts, their gradients and the 4-bit experts
together."""
import pytest

pytestmark = pytest.mark.gpu


def test_moe_layer_trains_and_serves():
    from examples import moe_layer

    losses, off = moe_layer.main(steps=12)
    assert all(v == v for v in losses) and losses[-1] < losses[0]
    # rounding to e2m1 blocks moves an operand by about 0.12 (relative): gate and
    # up products by 0.17 each, their product by 0.24, and with the roundings of
    # the SwiGLU outputs and of the down-projection 0.30
    assert 0.05 < off < 0.35
