"""The router where infinities meet the largest numbers, against the plain implementation of test_gpu_router.py."""
import pytest
import torch

from test_gpu_router import LARGEST, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [7, 4100])          # a wave and a quarter wave per token
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinity_ties_with_the_largest_number_in_a_groups_worth(tokens, score):
    """+inf counts as the largest fp32 number, in the worth of a group as in the rank of an expert: the lower group
    and the lower expert win."""
    x = torch.randn(tokens, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[0, 3], x[0, 60] = LARGEST, float("inf")
    x[1, 3], x[1, 60] = float("inf"), LARGEST
    x[2, 20:] = float("inf")
    x[2, 9] = LARGEST
    x[3] = float("inf")
    x[3, 15], x[3, 40] = LARGEST, float("-inf")
    x[4, ::5] = float("inf")
    x[4, 1::5] = LARGEST
    rows = slice(0, 7)
    for groups, kept in ((8, 1), (8, 3), (4, 2), (2, 1)):
        for top in (1, 2):
            check_forward(x, 5, None, score, groups, kept, top, rows=rows)
    idx, _ = check_forward(x, 1, None, score, 8, 1, 1, rows=rows)
    assert idx[:2, 0].tolist() == [3, 3]
