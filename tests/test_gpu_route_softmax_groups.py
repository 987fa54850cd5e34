"""The grouped softmax router at group sizes that are no power of two (a lane's experts, and whether a group's
score comes by shuffles or through shared memory, go by them), at spreads and biases that leave many rows to
float64, and with experts left out: against the float64 oracle, with the tolerances of the other tests."""
import pytest
import torch

from test_gpu_route_softmax import TYPES, bias_of, check, logits_of

pytestmark = pytest.mark.gpu
GROUPS = [(248, 8, 4, 8), (124, 4, 2, 8), (60, 1, 1, 8), (31, 1, 1, 8), (20, 4, 2, 4), (40, 8, 4, 6), (112, 16, 8, 8),
          (120, 8, 4, 8), (72, 8, 4, 8), (56, 8, 4, 6), (57, 3, 2, 6), (93, 3, 2, 8), (250, 2, 1, 8), (500, 20, 8, 8),
          (930, 30, 10, 8), (100, 4, 2, 30), (100, 4, 2, 33), (960, 32, 5, 9), (1022, 73, 20, 40), (62, 2, 1, 31)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,G,SG,k", GROUPS)
@pytest.mark.parametrize("two", [False, True])
def test_group_sizes(dtype, E, G, SG, k, two):
    x = logits_of(60, E, dtype, E + k)
    check(x, k, G, SG, two)
    check(x, k, G, SG, two, renorm=False, scale=2.5, bias=bias_of(E, E))
    check(x, k, G, SG, two, bias=torch.zeros(E))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spread", [4.0, 6.0, 8.0, 20.0])
@pytest.mark.parametrize("two", [False, True])
def test_peaked_rows(dtype, spread, two):
    """A trained router's: most rows' choices are closer than FP32 scores of the largest one tell."""
    for E, G, SG, k in ((256, 8, 4, 8), (64, 8, 3, 6), (153, 3, 2, 11)):
        x = logits_of(500, E, dtype, E, spread)
        check(x, k, G, SG, two, bias=torch.zeros(E))
        check(x, k, G, SG, two, renorm=False, bias=bias_of(E, 3))
        check(x, k, G, SG, two, renorm=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("two", [False, True])
def test_experts_left_out_of_many_rows(dtype, two):
    x, bias = logits_of(700, 256, dtype, 8), bias_of(256, 8)
    bias[3] = float("-inf")
    check(x, 8, 8, 4, two, bias=bias)
    bias[32:64] = float("-inf")                # a whole group
    check(x, 8, 8, 4, two, bias=bias)
