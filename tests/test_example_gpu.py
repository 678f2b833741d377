"""The example layer: decode steps reproduce one pass, and the gradient follows a difference (needs a GB300)."""
import pytest

from examples.gated_layer import GatedLayer, serve, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from state_space_model_ssm_gb300 import build
    build.build()
    return GatedLayer(256)


def test_serving_steps_reproduce_one_pass(layer):
    # The same operators on the same rows; the recurrence's sums in another order can move a bf16 rounding
    # (2^-9 relative) of y and with it a code (1/127 of the row's largest): well below 1e-2 of the norm.
    assert serve(layer, 200, 5) <= 1e-2


def test_training_gradient_follows_a_difference(layer):
    # central difference with step 1e-2: the loss is smooth on that scale (third-order term ~1e-4 relative),
    # and fp32 rounding of the layer ~1e-6 relative of the loss, over 2e-2, below 1e-3 of the slope
    slope, difference = train(layer, 300)
    assert abs(slope - difference) <= 1e-2 * (abs(slope) + 1.0)
