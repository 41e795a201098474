"""Routing where f32 sums or their bounds do not tell: against the definition in 64 bits, of test_gpu_route.py."""
import pytest

from test_gpu_route import check, env  # noqa: F401

pytestmark = pytest.mark.gpu
LOWEST = -3.4028234663852886e38      # the lowest f32, which masks are made of


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("e,groups,top,k,free", [(8, 4, 2, 4, 2), (8, 4, 3, 6, 2), (8, 4, 2, 4, 0), (6, 2, 1, 3, 1), (12, 4, 2, 5, 4), (64, 8, 4, 20, 16), (256, 8, 4, 32, 40),
                                                 (1000, 10, 3, 32, 100), (96, 48, 20, 32, 6)])
def test_groups_of_lowest_biases(env, e, groups, top, k, free, best, score):  # noqa: F811
    # the two best of a group may both have the lowest f32: a sum that f32 does not hold, and no empty group
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(e + top)
    logits = torch.randn(50, e, generator=g, device="cuda") * 2
    logits[1, : e // groups] = -float("inf")          # a group without anything to choose, before those of lowest biases
    logits[2, e // 2:] = float("nan")
    for low in (LOWEST, -1.8e38, -1.0e9):
        bias = torch.full((e,), low, device="cuda")   # free 0: the same low one for all
        bias[:free] = 0.05 * torch.randn(free, generator=g, device="cuda")
        check(env, logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=best)
        check(env, logits, k, score=score, bias=bias.flip(0), groups=groups, top_groups=top, group_best=best)


def test_the_last_group_of_lowest_biases(env):  # noqa: F811
    torch, _ = env
    bias = torch.full((8,), LOWEST, device="cuda")
    bias[:2] = 0.0
    ids, _ = check(env, torch.zeros(3, 8, device="cuda"), 4, score="sigmoid", bias=bias, groups=4, top_groups=2, group_best=2)
    assert ids.tolist() == [[0, 1, 2, 3]] * 3
