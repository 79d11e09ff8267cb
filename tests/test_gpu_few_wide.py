"""The few-token layer's experts' kernel that makes its own picks, in slices of 128 columns of mlp: a decode step of a wide
layer. Checked as the other shapes are."""
import pytest

import test_gpu_few as tf
from test_few_plan import _slices

pytestmark = pytest.mark.gpu

# at most 8 tokens and 64 picks; workgroups for each compute unit once, and for more than three of 64 columns; last slices
# of 64 columns; k = E; emb past a whole number of 128
SHAPES = [(4, 192, 576, 64, 8), (8, 128, 1216, 64, 8), (1, 64, 9280, 2, 2), (3, 1088, 832, 24, 8), (8, 64, 2304, 256, 8),
          (2, 320, 896, 32, 32)]


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_layer_with_its_router(T, emb, mlp, E, k, bias):
    assert T <= 8 and T * k <= 64 and round(_slices(T, emb, mlp, E, k), 2) == -(-mlp // 128)
    tf.test_layer_with_its_router(T, emb, mlp, E, k, bias)


@pytest.mark.parametrize("T,emb,mlp,E,k", SHAPES)
def test_given_routing_gives_the_same_bits_and_mx_weights_their_values(T, emb, mlp, E, k):
    tf.test_given_routing_gives_the_same_bits_and_mx_weights_their_values(T, emb, mlp, E, k)
