"""Routing to experts and its gradient on the GPU against the definitions in 64 bits.  The experts are
compared for equality: their order is that of the real numbers, which 64 bits tell apart here.

Tolerance of a weight, u = 2^-24.  A softmax score is exp(l - m) / sum: the difference l - m is rounded, which
moves the exponential by |l - m| u at most, the exponential is within 2 ulp (4 u) of its argument's, the sum of positive
terms that are each as near takes 10 further roundings (5 by lane, 5 across lanes; 37 with 32 experts
a lane), the quotient one, its own renormalisation the same once more with 5 roundings.  With D the largest |l - m| that
counts (104: beyond it a term is below 2^-149): relative error <= (2 D + 2 * 4 + 37 + 5 + 6) u <= (2 D + 64) u.
A sigmoid is within 4 + 2 u of its value and its renormalisation within 8 + 5 + 3 more: the same bound holds.
Below 2^-126 a score may be lost altogether.
Gradients: dl = s (1 - s) h or s (h - common), h = g or (g - sum(g s) / S) / S; each factor carries the bound above and each
sum is bounded by the sum of its terms' sizes: |error| <= 3 (2 D + 64) u s (|h| + sum |h| s) + the output's rounding, with |h| taken
over as (|g| + sum |g| s / S) / S where renormalised."""
import math

import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def clean(torch, l):
    l = l.double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -INF), l)
    return l.clamp(max=float(torch.finfo(torch.float32).max))


def scores(torch, l, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    e = torch.exp(l - m)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def definition(torch, logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_best=1, renormalise=True, factor=1.0):
    """(ids, weights) in 64 bits."""
    l = clean(torch, logits)
    t, e = l.shape
    choose = scores(torch, l, score)
    ranked_by = choose
    if bias is not None:
        b = clean(torch, bias)
        choose = choose + b
        ranked_by = choose if float(b[b > -INF].max()) > float(b[b > -INF].min()) else torch.where(b > -INF, l, torch.full_like(l, -INF))
    else:
        ranked_by = l           # (the order of the scores, and of those that 64 bits do not tell from zero)
    choose, ranked_by = (torch.where(l == -INF, torch.full_like(choose, -INF), q) for q in (choose, ranked_by))
    top_groups = groups if top_groups is None else top_groups
    if top_groups < groups:
        of = (choose if group_best == 2 else ranked_by).view(t, groups, e // groups)
        best = torch.sort(of, dim=2, descending=True)[0][:, :, :group_best]
        total = torch.where(best == -INF, torch.zeros_like(best), best).sum(2)
        total = torch.where(best[:, :, 0] == -INF, torch.full_like(total, -INF), total)
        kept = torch.sort(total, dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros_like(total, dtype=torch.bool).scatter_(1, kept, True)
        of = ranked_by.view(t, groups, e // groups)
        ranked_by = torch.where(keep[:, :, None], of, torch.full_like(of, -INF)).reshape(t, e)
    ranked, ids = torch.sort(ranked_by, dim=1, descending=True, stable=True)
    ids, there = ids[:, :top_k], ranked[:, :top_k] > -INF
    chosen = torch.where(there, l.gather(1, ids), torch.full_like(ranked[:, :top_k], -INF))
    if renormalise:
        # log scores relative to the largest: nothing is lost far below zero
        log = chosen if score == "softmax" else torch.where(chosen < -30, chosen, torch.nn.functional.logsigmoid(chosen))
        top = log.amax(1, keepdim=True)
        w = torch.where(there, torch.exp(log - torch.where(top == -INF, torch.zeros_like(top), top)), torch.zeros_like(log))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.where(there, scores(torch, l, score).gather(1, ids), torch.zeros_like(chosen))
    return torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32), w * factor


def bound(torch, logits):
    l = clean(torch, logits)
    low = torch.where(l == -INF, torch.full_like(l, INF), l).amin(1)
    spread = torch.where(torch.isfinite(low), l.amax(1) - low, torch.zeros_like(low)).clamp(0, 104)
    return (2 * spread + 64)[:, None] * 2.0 ** -24


def check(env, logits, top_k, **kw):
    torch, loom = env
    ids, weights = loom.loom_route_tokens(logits, top_k, **kw)
    want_ids, want = definition(torch, logits, top_k, **kw)
    assert torch.equal(ids, want_ids), (ids != want_ids).nonzero()[:3].tolist()
    err = (weights.double() - want).abs()
    assert bool((err <= bound(torch, logits) * want.abs() + 2.0 ** -126).all()), float(err.max())
    return ids, weights


KINDS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


@pytest.mark.parametrize("score,renormalise", KINDS)
@pytest.mark.parametrize("t,e,k,dtype", [(1, 1, 1, "float32"), (3, 2, 2, "bfloat16"), (5, 7, 3, "float32"), (17, 32, 8, "float16"), (1, 64, 8, "float32"), (100, 60, 4, "bfloat16"),
                                         (33, 65, 32, "float32"), (700, 256, 8, "float32"), (64, 255, 12, "float16"), (20, 512, 10, "bfloat16"), (9, 1000, 32, "float32"),
                                         (3, 1024, 1, "float32"), (5000, 128, 6, "bfloat16")])
def test_sizes(env, t, e, k, dtype, score, renormalise):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(e + t)
    logits = (torch.randn(t, e, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    bias = 0.1 * torch.randn(e, generator=g, device="cuda")
    check(env, logits, k, score=score, renormalise=renormalise, factor=2.5)
    check(env, logits, k, score=score, renormalise=renormalise, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,top,best,k", [(256, 8, 4, 2, 8), (256, 8, 3, 1, 6), (160, 8, 3, 1, 6), (60, 4, 2, 2, 4), (96, 32, 5, 2, 10), (64, 64, 9, 2, 9), (12, 3, 1, 2, 8),
                                                 (1000, 10, 7, 2, 20), (1024, 4, 3, 2, 32), (30, 2, 2, 2, 5), (35, 5, 2, 1, 3), (768, 3, 2, 2, 8), (1020, 510, 200, 2, 8)])
def test_groups(env, e, groups, top, best, k, score):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(e * groups)
    logits = torch.randn(90, e, generator=g, device="cuda") * 2
    for bias in (None, 0.2 * torch.randn(e, generator=g, device="cuda")):
        ids, _ = check(env, logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=best)
        of = torch.where(ids >= 0, ids // (e // groups), ids)
        assert all(len(set(row) - {-1}) <= top for row in of.tolist())


def test_ties_go_to_the_lower_index(env):
    torch, _ = env
    for dtype in (torch.float32, torch.bfloat16):
        same = torch.full((3, 200), 0.25, dtype=dtype, device="cuda")
        for kw in ({}, {"bias": torch.zeros(200, device="cuda")}, {"score": "sigmoid", "bias": torch.full((200,), 0.5, device="cuda")}):
            ids, weights = check(env, same, 7, **kw)
            assert torch.equal(ids, torch.arange(7, device="cuda", dtype=torch.int32).expand(3, 7))
        check(env, same, 7, groups=10, top_groups=3, group_best=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    coarse = torch.randint(-3, 4, (400, 96), generator=g, device="cuda").to(torch.bfloat16)
    for score in ("softmax", "sigmoid"):
        check(env, coarse, 10, score=score)
        check(env, coarse, 10, score=score, bias=torch.zeros(96, device="cuda"))
        check(env, coarse, 10, score=score, bias=torch.randint(0, 2, (96,), generator=g, device="cuda") * 0.25)
        check(env, coarse, 10, score=score, groups=8, top_groups=3, group_best=1)
    # (sums of two scores that tie are sums of the same two numbers, in either order)
    check(env, coarse, 10, score="sigmoid", groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("e", [20, 256, 1000])
def test_both_zeros_are_one_logit(env, e):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(e)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        zeros = torch.where(torch.rand(64, e, generator=g, device="cuda") < 0.5, -0.0, 0.0).to(dtype)
        for kw in ({}, {"score": "sigmoid"}, {"bias": torch.full((e,), 0.5, device="cuda")}, {"groups": 5 if e % 5 == 0 else 4, "top_groups": 2}):
            check(env, zeros, 9, **kw)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("e,groups,top", [(2, 2, 1), (4, 2, 1), (6, 3, 2), (8, 8, 3), (8, 4, 2), (8, 2, 1), (9, 3, 1), (10, 5, 2), (10, 2, 1), (12, 6, 2), (15, 5, 3), (16, 16, 5)])
def test_ties_among_a_few_experts_in_groups(env, e, groups, top, best):
    """Few experts, most groups alike at the cut: every warp lists those that 64 bits are to tell apart, at once."""
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(e + groups)
    logits = torch.randint(0, 3, (2000, e), generator=g, device="cuda").float()
    k = min(e, max(1, e // groups * top - 1))
    for bias in (None, torch.randint(0, 2, (e,), generator=g, device="cuda") * 0.25):
        counts = torch.zeros(e, dtype=torch.int32, device="cuda")
        kw = dict(score="sigmoid", bias=bias, groups=groups, top_groups=top, group_best=best)
        ids, _ = check(env, logits, k, **kw)
        again, _ = loom.loom_route_tokens(logits, k, counts=counts, **kw)
        assert torch.equal(ids, again)
        assert torch.equal(counts.long(), torch.bincount(ids[ids >= 0].long(), minlength=e))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k", [(40, 6), (256, 8), (1024, 16)])
def test_choices_that_32_bits_do_not_tell_apart(env, score, e, k):
    # the bias undoes the scores' differences but for its own rounding
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(e)
    row = torch.randn(1, e, generator=g, device="cuda")
    bias = (0.75 - scores(torch, row.double(), score)[0]).float()
    logits = torch.cat([row, row.flip(1), row])
    check(env, logits, k, score=score, bias=bias)
    check(env, logits, k, score=score, bias=bias, groups=8, top_groups=3, group_best=2)
    check(env, logits, k, score=score, bias=bias, groups=4, top_groups=1, group_best=1)


def test_logits_that_are_not_finite(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(64, 40, generator=g, device="cuda")
    logits[0] = -INF                                    # nothing to choose
    logits[1] = float("nan")
    logits[2, 3:] = -INF                                # three to choose
    logits[3, ::2] = float("nan")
    logits[4, 5], logits[4, 9] = INF, INF
    logits[5] = torch.finfo(torch.float32).min          # a mask's lowest value
    logits[6, :30] = torch.finfo(torch.float32).min
    logits[7] = -200.0 - torch.arange(40, device="cuda")         # scores that underflow
    logits[8, 1:] = -1000.0
    bias = 0.1 * torch.randn(40, generator=g, device="cuda")
    bias[11], bias[12] = -INF, float("nan")
    for score, renormalise in KINDS:
        for b in (None, bias):
            ids, weights = check(env, logits, 6, score=score, renormalise=renormalise, bias=b)
            assert bool((ids[:2] == -1).all()) and not bool(weights[:2].any()) and bool((ids[2, 3:] == -1).all())
            if b is not None:
                assert not bool(((ids == 11) | (ids == 12)).any())
            check(env, logits, 6, score=score, renormalise=renormalise, bias=b, groups=8, top_groups=2, group_best=2)
    out = torch.zeros(40, dtype=torch.int32, device="cuda")
    ids, _ = loom.loom_route_tokens(logits, 6, counts=out)
    assert torch.equal(out.long(), torch.bincount(ids[ids >= 0].long(), minlength=40))


def test_counts_strides_and_outputs(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(3000, 130, generator=g, device="cuda").to(torch.bfloat16)
    logits = wide[:, 1:129]
    counts = torch.full((128,), 5, dtype=torch.int32, device="cuda")
    ids, weights = torch.full((3000, 8), -9, dtype=torch.int32, device="cuda"), torch.empty(3000, 8, device="cuda")
    out = loom.loom_route_tokens(logits, 8, counts=counts, ids=ids, weights=weights)
    assert out[0] is ids and out[1] is weights
    want = loom.loom_route_tokens(logits.contiguous(), 8)
    assert torch.equal(ids, want[0]) and torch.equal(weights, want[1])
    assert torch.equal(counts.long() - 5, torch.bincount(ids.view(-1).long(), minlength=128))
    assert loom.loom_route_tokens(logits[:0], 8)[0].shape == (0, 8)
    # two tokens further apart than 2^31 elements
    far = torch.empty((1 << 31) + 200, dtype=torch.bfloat16, device="cuda").as_strided((2, 128), ((1 << 31) + 8, 1))
    far.copy_(logits[:2])
    assert torch.equal(loom.loom_route_tokens(far, 8)[0], ids[:2])
    d = torch.randn(2, 8, generator=g, device="cuda")
    assert torch.equal(loom.loom_route_tokens_backward(d, far, ids[:2].clone()), loom.loom_route_tokens_backward(d, logits[:2].contiguous(), ids[:2].clone()))


def test_biases_that_settle_the_choice(env):
    # +infinity counts as the largest f32, whose sums f32 does not hold
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(40, 64, generator=g, device="cuda")
    bias = 0.1 * torch.randn(64, generator=g, device="cuda")
    bias[[3, 9, 10, 33]] = INF
    bias[[20, 21]] = 3.0e38
    bias[[50, 51]] = -3.0e38
    for score in ("softmax", "sigmoid"):
        check(env, logits, 6, score=score, bias=bias)
        for groups, top in ((8, 3), (8, 1), (4, 2)):
            for best in (1, 2):
                check(env, logits, 6, score=score, bias=bias, groups=groups, top_groups=top, group_best=best)


# ---- gradient ---------------------------------------------------------------------------------
def gradient(torch, dw, logits, ids, score, renormalise, factor):
    """(dlogits, the size that bounds its error) in 64 bits."""
    l = clean(torch, logits)
    there = (ids >= 0) & (ids < l.shape[1])
    at = torch.where(there, ids.long(), torch.zeros_like(ids, dtype=torch.int64))
    lc = l.gather(1, at)
    there &= lc > -INF
    zero = torch.zeros_like(lc)
    g = torch.where(there, dw.double() * factor, zero)
    full, size = torch.zeros_like(l), torch.zeros_like(l)
    if renormalise:
        log = lc if score == "softmax" else torch.where(lc < -30, lc, torch.nn.functional.logsigmoid(lc))
        log = torch.where(there, log, torch.full_like(log, -INF))
        top = log.amax(1, keepdim=True)
        w = torch.where(there, torch.exp(log - torch.where(top == -INF, zero[:, :1], top)), zero)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        h, mag = g - (g * w).sum(1, keepdim=True), g.abs() + (g.abs() * w).sum(1, keepdim=True)
        part = w if score == "softmax" else w / (1 + torch.exp(lc))
        full.scatter_add_(1, at, torch.where(there, part * h, zero))
        size.scatter_add_(1, at, torch.where(there, part * mag, zero))
        return full, size
    s = scores(torch, l, score)
    sc = torch.where(there, s.gather(1, at), zero)
    if score == "sigmoid":
        part = torch.where(there, sc / (1 + torch.exp(lc)), zero)
        return full.scatter_add_(1, at, part * g), size.scatter_add_(1, at, part * g.abs())
    full.scatter_add_(1, at, sc * g)
    size.scatter_add_(1, at, sc * g.abs())
    return full - s * (g * sc).sum(1, keepdim=True), size + s * (g.abs() * sc).sum(1, keepdim=True)


def check_gradient(env, dw, logits, ids, score, renormalise, factor=1.0, **kw):
    torch, loom = env
    got = loom.loom_route_tokens_backward(dw, logits, ids, score=score, renormalise=renormalise, factor=factor, **kw)
    want, size = gradient(torch, dw, logits, ids, score, renormalise, factor)
    tol = 3 * bound(torch, logits) * size + 2.0 ** -126
    if got.dtype != torch.float32:
        tol = tol * 1.01 + want.abs() * torch.finfo(got.dtype).eps / 2 + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), (err > tol).nonzero()[:3].tolist())
    return got


@pytest.mark.parametrize("score,renormalise", KINDS)
@pytest.mark.parametrize("t,e,k,dtype", [(1, 1, 1, "float32"), (3, 2, 2, "bfloat16"), (5, 7, 3, "float32"), (17, 32, 8, "float16"), (1, 64, 8, "float32"), (100, 60, 4, "bfloat16"),
                                         (33, 65, 32, "float32"), (700, 256, 8, "float32"), (20, 512, 10, "bfloat16"), (9, 1000, 32, "float32"), (3, 1024, 1, "float32")])
def test_gradient_sizes(env, t, e, k, dtype, score, renormalise):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(7 * e + t)
    logits = (torch.randn(t, e, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    ids, _ = loom.loom_route_tokens(logits, k, score=score)
    dw = torch.randn(t, k, generator=g, device="cuda")
    check_gradient(env, dw, logits, ids, score, renormalise, 2.5)
    # any ids: the same one twice, missing ones
    ids = torch.randint(-1, e, (t, k), generator=g, device="cuda", dtype=torch.int32)
    got = check_gradient(env, dw, logits, ids, score, renormalise)
    assert torch.equal(got, loom.loom_route_tokens_backward(dw, logits, ids, score=score, renormalise=renormalise))


@pytest.mark.parametrize("score,renormalise", KINDS)
def test_gradient_against_differences(env, score, renormalise):
    # central differences of the weights' definition, in 64 bits
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(11)
    logits, dw = torch.randn(6, 20, generator=g, device="cuda"), torch.randn(6, 5, generator=g, device="cuda")
    ids, _ = loom.loom_route_tokens(logits, 5, score=score)
    got = loom.loom_route_tokens_backward(dw, logits, ids, score=score, renormalise=renormalise, factor=1.5).double()

    def loss(l):
        w = scores(torch, l, score).gather(1, ids.long())
        w = w / w.sum(1, keepdim=True) if renormalise else w
        return (1.5 * w * dw.double()).sum(1)
    step = 1e-5
    for e in range(20):
        up, down = logits.double(), logits.double()
        up[:, e] += step
        down[:, e] -= step
        d = (loss(up) - loss(down)) / (2 * step)
        # differences: step^2 / 6 times a third derivative (below 10 |dw|), and 2^-52 / step
        assert bool(((got[:, e] - d).abs() <= 1e-8 + 5e-6 * dw.double().abs().sum(1)).all())


@pytest.mark.parametrize("score,renormalise", KINDS)
def test_gradient_at_the_edges(env, score, renormalise):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(12)
    logits = torch.randn(12, 40, generator=g, device="cuda")
    logits[0] = -INF
    logits[1] = float("nan")
    logits[2, 3:] = -INF
    logits[3, ::2] = float("nan")
    logits[4, 5], logits[4, 9] = INF, INF
    logits[5] = torch.finfo(torch.float32).min
    logits[7] = -200.0 - torch.arange(40, device="cuda")
    logits[8, 1:] = -1000.0
    logits[9] = 50.0
    dw = torch.randn(12, 6, generator=g, device="cuda")
    ids, _ = loom.loom_route_tokens(logits, 6, score=score)
    ids[10] = -1
    ids[11, 2] = 40
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = check_gradient(env, dw, logits, ids, score, renormalise, error=err)
    assert int(err) == loom.LOOM_DEVERR_COUNT_RANGE and bool(torch.isfinite(got).all()) and not bool(got[[0, 1, 10]].any())
    # in place, and strided
    wide = torch.randn(12, 50, generator=g, device="cuda")
    wide[:, 3:43] = logits
    view = wide[:, 3:43]
    kept = wide.clone()
    out = loom.loom_route_tokens_backward(dw, view, ids, score=score, renormalise=renormalise, dlogits=view)
    assert out is view and torch.equal(view, got) and torch.equal(wide[:, :3], kept[:, :3]) and torch.equal(wide[:, 43:], kept[:, 43:])


def test_gradient_recorded_in_a_graph(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(13)
    logits, dw = torch.randn(200, 64, generator=g, device="cuda"), torch.randn(200, 8, generator=g, device="cuda")

    def step():
        ids, w = loom.loom_route_tokens(logits, 8, score="sigmoid")
        return ids, w, loom.loom_route_tokens_backward(dw, logits, ids, score="sigmoid")
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    logits.copy_(torch.randn(200, 64, generator=g, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert math.isfinite(float(got[2].sum()))
