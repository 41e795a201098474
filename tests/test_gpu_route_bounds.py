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


def test_sums_of_two_at_the_worst_roundings(env):  # noqa: F811
    """Scores + 63.5 lie in [64, 65), 2^-17 apart in f32, and the sums of two are 2^-16 apart.  Group 0's scores are just above the
    middle of two places and group 1's just below it, so that scores some 1e-7 off are rounded apart by four halves of
    2^-17; the places are chosen for the sums, ties of 2^-16, to be rounded apart as well: 2^-15 in favour of group 1 where group 0
    has the larger sum."""
    torch, _ = env
    t, step = 1 << 16, 2.0 ** -17
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda n: torch.randint(0, n, (t,), generator=g, device="cuda")   # noqa: E731
    a0, a1 = 8000 + 2 * draw(4000), 8001 + 4 * draw(2000)                 # even, odd
    a0 += (1 - a0 - a1) % 4                                               # (a sum of 4 i + 1)
    b0 = 8001 + 2 * draw(2000)
    b0 = torch.minimum(b0, a0 + a1)
    b1 = a0 + a1 - b0
    sides = torch.tensor([1.0, 1.0, -1.0, -1.0], device="cuda", dtype=torch.float64)
    middle = 0.5 + (torch.stack([a0, a1, b0, b1], 1).double() + 0.5) * step
    off = 1e-9 + 3e-8 * torch.rand(t, 4, generator=g, device="cuda", dtype=torch.float64)
    s = middle + sides * off
    logits = torch.log(s / (1 - s)).float()
    exact = 1 / (1 + torch.exp(-logits.double()))
    sums = exact[:, :2].sum(1) - exact[:, 2:].sum(1)
    assert bool((sums.abs() < 4e-7).all()) and bool(((a0 + a1) % 4 == 1).all()) and bool((b1 % 2 == 0).all())
    check(env, logits, 2, score="sigmoid", bias=torch.full((4,), 63.5, device="cuda"), groups=2, top_groups=1, group_best=2)


def times(torch, *calls):
    """The least time of each call, in turn, as nodes of a graph: the host's part does not count."""
    graphs, best = [], [float("inf")] * len(calls)
    for call in calls:
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                call()
    for _ in range(20):
        for i, graph in enumerate(graphs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    return best


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("masked", ["one", "half", "groups"])
@pytest.mark.parametrize("low", [-1.0e4, -1.0e9, LOWEST])
def test_a_finite_mask_costs_no_time(env, score, masked, low):  # noqa: F811
    # (ranking all tokens in 64 bits takes 20 times as long)
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(4)
    t, e = 16384, 256
    logits, bias = torch.randn(t, e, generator=g, device="cuda") * 2, 0.05 * torch.randn(e, generator=g, device="cuda")
    with_mask = bias.clone()
    with_mask[{"one": slice(7, 8), "half": slice(0, e, 2), "groups": slice(32, 160)}[masked]] = low
    for kw in ({}, {"groups": 8, "top_groups": 4, "group_best": 2}):
        check(env, logits[:512], 8, score=score, bias=with_mask, **kw)
        ids, weights = loom.loom_route_tokens(logits, 8)
        call = lambda b: loom.loom_route_tokens(logits, 8, score=score, bias=b, ids=ids, weights=weights, **kw)   # noqa: E731, B023
        plain, other = times(torch, lambda: call(bias), lambda: call(with_mask))    # noqa: B023
        assert other <= 2 * plain, (kw, other, plain)
