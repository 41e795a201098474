"""4-bit products on the GPU against the definition in 64 bits.

Tolerance of y, with u = 2^-24: every group's sum a is exact, so y = sx sum s a is a sum of products in
f32.  The sum is taken in pieces of 128 k at most (of a group, where those are shorter), which are
added in some chain or tree: N = ceil(k / min(group, 128)) + k / 256 + 16 roundings at most on the way of
each piece, the roundings by sx and of the bias's addition among the 16.  A piece's |s a| is at most the
sum of its words' |s a|, so |error| <= N u sx S + u |y| with S = sum over words |s a| (second-order terms are below
u N^2 u and covered by the 16).  Then the output's rounding: half an eps of |y| and half of f16's least subnormal."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def pack(torch, v):
    """int32 words of signed nibbles v [..., k]."""
    q = (v.to(torch.int64) & 15).view(*v.shape[:-1], v.shape[-1] // 8, 8)
    word = (q << (4 * torch.arange(8, device=v.device))).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def operands(torch, t, n, k, group, scale, seed, lead=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-8, 8, (*lead, n, k), generator=g, device="cuda", dtype=torch.int8)
    s = (0.002 + 0.01 * torch.rand((*lead, n, -(-k // group)), generator=g, device="cuda")).to(getattr(torch, scale))
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    return v, s, x, 0.001 + 0.01 * torch.rand(t, generator=g, device="cuda"), torch.randn((*lead, n), generator=g, device="cuda")


def definition(torch, v, s, x, sx, group, bias=None):
    """(y, S) in 64 bits."""
    n, k = v.shape
    t, words = x.shape[0], k // 8
    y, size = (torch.zeros(t, n, dtype=torch.float64, device="cuda") for _ in range(2))
    for j in range(words):
        a = x[:, 8 * j:8 * j + 8].double() @ v[:, 8 * j:8 * j + 8].double().t()
        term = a * s[:, 8 * j // group].double()
        y += term
        size += term.abs()
    y, size = y * sx.double()[:, None], size * sx.double()[:, None]
    return (y if bias is None else y + bias.double()), size


def check(torch, got, want, size, k, group):
    steps = -(-k // min(group, 128)) + k // 256 + 16
    tol = (steps * size + want.abs()) * 2.0 ** -24
    if got.dtype != torch.float32:
        tol = tol * 1.01 + want.abs() * torch.finfo(got.dtype).eps / 2 + 2.0 ** -25
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float((err / tol.clamp(min=1e-300)).max()))


SIZES = [(1, 1, 8, 32), (1, 8, 8192, 128), (2, 15, 32, 32), (3, 17, 40, 32), (4, 33, 264, 64), (5, 64, 1032, 128), (7, 100, 4104, 32), (8, 129, 512, 256),
         (9, 300, 2048, 64), (15, 31, 4096, 4096), (16, 257, 520, 32), (17, 1000, 1536, 128), (24, 48, 800, 512), (31, 65, 2056, 64), (32, 640, 1024, 32),
         (33, 500, 768, 128), (70, 41, 1288, 64), (130, 20, 16384, 128), (1, 5000, 256, 32), (6, 20000, 128, 128)]


@pytest.mark.parametrize("t,n,k,group", SIZES)
@pytest.mark.parametrize("scale,y_dtype,with_bias", [("float32", "float32", False), ("float16", "bfloat16", True), ("bfloat16", "float16", True)])
def test_sizes(env, t, n, k, group, scale, y_dtype, with_bias):
    torch, loom = env
    v, s, x, sx, bias = operands(torch, t, n, k, group, scale, 100 * t + k)
    bias = bias if with_bias else None
    y = loom.loom_i4_matvec(pack(torch, v), s, n, k, group, x, sx, t, bias=bias, y_dtype=getattr(torch, y_dtype))
    assert y.shape == (t, n) and y.dtype == getattr(torch, y_dtype)
    check(torch, y, *definition(torch, v, s, x, sx, group, bias), k, group)
    assert torch.equal(y, loom.loom_i4_matvec(pack(torch, v), s, n, k, group, x, sx, t, bias=bias, y_dtype=y.dtype))


@pytest.mark.parametrize("t", [1, 8, 9, 16, 32])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 1024, 1 << 30])
def test_sums_are_exact(env, t, group):
    # scales of one and whole sums below 2^24: whatever the order, the result is the sum
    torch, loom = env
    n, k = 90, 16384
    g = torch.Generator(device="cuda").manual_seed(group % 1000 + t)
    v = torch.randint(-8, 8, (n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    v[0], v[1], v[2] = -8, 7, -8
    x[0] = -128            # the largest sums there are: 8 * 128 * 16384 = 2^24
    if t > 1:
        x[1] = 127
    s = torch.ones(n, -(-k // group), device="cuda")
    y = loom.loom_i4_matvec(pack(torch, v), s, n, k, group, x, torch.ones(t, device="cuda"), t)
    assert torch.equal(y.double(), x.double() @ v.double().t())


def test_every_nibble_and_byte(env):
    # each place of a row alone: its nibble times its byte
    torch, loom = env
    k, n = 264, 16
    v = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    x = torch.zeros(8, k, dtype=torch.int8, device="cuda")
    one = torch.ones(n, -(-k // 32), device="cuda")
    for at in range(k):
        v.zero_(), x.zero_()
        v[:, at] = torch.arange(-8, 8, dtype=torch.int8, device="cuda")
        x[:, at] = torch.tensor([-128, -127, -1, 0, 1, 15, 16, 127], dtype=torch.int8, device="cuda")
        y = loom.loom_i4_matvec(pack(torch, v), one, n, k, 32, x, torch.ones(8, device="cuda"), 8)
        assert torch.equal(y.double(), x.double() @ v.double().t()), at


@pytest.mark.parametrize("k,offset", [(1024, 1), (1024, 2), (1048, 0), (1032, 3)])
def test_operands_off_16_bytes(env, k, offset):
    torch, loom = env
    t, n, group = 6, 77, 64
    v, s, x, sx, bias = operands(torch, t, n, k, group, "float16", k + offset)
    w = torch.empty(n * k // 8 + 8, dtype=torch.int32, device="cuda")[offset:offset + n * k // 8]
    w.copy_(pack(torch, v).view(-1))
    xb = torch.empty(t * k // 4 + 8, dtype=torch.int32, device="cuda")[offset:offset + t * k // 4]
    xb.copy_(x.view(torch.int32).view(-1))
    sb = torch.empty(s.numel() + 8, dtype=s.dtype, device="cuda")[offset:offset + s.numel()]
    sb.copy_(s.view(-1))
    y = loom.loom_i4_matvec(w, sb, n, k, group, xb, sx, t, bias=bias)
    check(torch, y, *definition(torch, v, s, x, sx, group, bias), k, group)
    assert torch.equal(y, loom.loom_i4_matvec(pack(torch, v), s, n, k, group, x, sx, t, bias=bias))


def test_outputs_in_place_of_the_callers(env):
    torch, loom = env
    t, n, k = 11, 45, 512
    v, s, x, sx, _ = operands(torch, t, n, k, 64, "float16", 3)
    y = torch.full((t + 2, n + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    want = loom.loom_i4_matvec(pack(torch, v), s, n, k, 64, x, sx, t, y_dtype=torch.bfloat16)
    assert loom.loom_i4_matvec(pack(torch, v), s, n, k, 64, x, sx, t, y=y) is y
    assert torch.equal(y[:t, :n], want) and int(torch.isnan(y).sum()) == y.numel() - t * n
    # no k: the bias alone; no tokens, no rows: nothing
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    bias = torch.randn(n, device="cuda")
    for some in (1, 2, t):
        y = loom.loom_i4_matvec(none, torch.empty(0, device="cuda"), n, 0, 32, none, sx, some, bias=bias)
        assert torch.equal(y, bias.expand(some, n))
    routed = loom.loom_i4_matvec_routed(none, torch.empty(0, device="cuda"), 3, n, 0, 32, none, sx, torch.tensor([[0, -1, 2]], dtype=torch.int32, device="cuda"), bias=bias.repeat(3))
    assert torch.equal(routed[0], bias) and not bool(routed[1].any()) and torch.equal(routed[2], bias)
    assert loom.loom_i4_matvec(pack(torch, v), s, n, k, 64, x, sx, 0).shape == (0, n)


def test_scales_that_are_not_numbers(env):
    # an infinite or NaN scale reaches its own row alone, a token's scale its own token
    torch, loom = env
    t, n, k = 5, 40, 512
    v, s, x, sx, _ = operands(torch, t, n, k, 128, "float32", 9)
    want = loom.loom_i4_matvec(pack(torch, v), s, n, k, 128, x, sx, t)
    s[3, 1], s[20, 2] = float("nan"), float("inf")
    sx[2] = float("nan")
    y = loom.loom_i4_matvec(pack(torch, v), s, n, k, 128, x, sx, t)
    rows = [r for r in range(n) if r not in (3, 20)]
    keep = [i for i in range(t) if i != 2]
    assert torch.equal(y[keep][:, rows], want[keep][:, rows])
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[:, 3]).all()) and not bool(torch.isfinite(y[:, 20]).any())


# ---- the experts' products ------------------------------------------------------------------
ROUTED = [(1, 4, 1, 16, 64, 32), (1, 64, 8, 200, 512, 128), (5, 3, 2, 33, 1032, 64), (16, 8, 2, 130, 256, 32), (40, 5, 3, 70, 768, 128),
          (33, 60, 4, 64, 1024, 64), (100, 1, 1, 48, 520, 256), (300, 16, 8, 24, 264, 32), (64, 1024, 6, 20, 128, 64)]


def routed_definition(torch, v, s, x, sx, ids, group, per_x, bias):
    pairs = ids.numel()
    want, size = (torch.zeros(pairs, v.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    flat = ids.view(-1)
    for e in torch.unique(flat).tolist():
        if 0 <= e < v.shape[0]:
            at = (flat == e).nonzero()[:, 0]
            want[at], size[at] = definition(torch, v[e], s[e], x[at // per_x], sx[at // per_x], group, None if bias is None else bias[e])
    return want, size


@pytest.mark.parametrize("t,experts,routes,n,k,group", ROUTED)
@pytest.mark.parametrize("own_rows,scale,y_dtype,with_bias", [(False, "float16", "float32", False), (True, "float32", "bfloat16", True)])
def test_experts(env, t, experts, routes, n, k, group, own_rows, scale, y_dtype, with_bias):
    torch, loom = env
    x_rows = t * routes if own_rows else t
    v, s, x, sx, bias = operands(torch, x_rows, n, k, group, scale, t + n, (experts,))
    bias = bias if with_bias else None
    g = torch.Generator(device="cuda").manual_seed(t)
    ids = torch.randint(0, experts, (t, routes), generator=g, device="cuda", dtype=torch.int32)     # an expert twice, too
    ids[torch.rand(t, routes, generator=g, device="cuda") < 0.1] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = loom.loom_i4_matvec_routed(pack(torch, v), s, experts, n, k, group, x, sx, ids, x_rows=x_rows, bias=bias, y_dtype=getattr(torch, y_dtype), error=err)
    check(torch, y, *routed_definition(torch, v, s, x, sx, ids, group, 1 if own_rows else routes, bias), k, group)
    assert int(err) == 0 and not bool(y[ids.view(-1) < 0].any())
    # a pair's row does not depend on its neighbours
    alone = loom.loom_i4_matvec_routed(pack(torch, v), s, experts, n, k, group, x[-1:], sx[-1:], ids[-1:, -1:], bias=bias, y_dtype=y.dtype)
    check(torch, alone, *(q[-1:] for q in routed_definition(torch, v, s, x, sx, ids, group, 1 if own_rows else routes, bias)), k, group)


def test_all_pairs_to_one_expert_and_none(env):
    torch, loom = env
    t, experts, routes, n, k = 300, 20, 7, 30, 256       # 2100 pairs: two launches
    v, s, x, sx, _ = operands(torch, t, n, k, 64, "float16", 5, (experts,))
    for fill in (19, 0, -1):
        ids = torch.full((t, routes), fill, dtype=torch.int32, device="cuda")
        y = loom.loom_i4_matvec_routed(pack(torch, v), s, experts, n, k, 64, x, sx, ids)
        check(torch, y, *routed_definition(torch, v, s, x, sx, ids, 64, routes, None), k, 64)
    assert not bool(y.any())


def test_ids_out_of_range_are_flagged(env):
    torch, loom = env
    v, s, x, sx, _ = operands(torch, 2, 10, 64, 32, "float16", 6, (3,))
    ids = torch.tensor([[3, 1], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = loom.loom_i4_matvec_routed(pack(torch, v), s, 3, 10, 64, 32, x, sx, ids, error=err)
    assert int(err) == loom.LOOM_DEVERR_COUNT_RANGE and not bool(y[[0, 2, 3]].any()) and bool(y[1].any())
    # no experts at all: every route is missing
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    y = torch.full((4, 10), float("nan"), device="cuda")
    loom.loom_i4_matvec_routed(none, torch.empty(0, device="cuda"), 0, 10, 64, 32, x, sx, torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), y=y)
    assert not bool(y.any())


def test_weights_past_31_bits(env):
    torch, loom = env
    experts, n, k = 40, 16384, 16384         # 5.4 GB of weights; the last experts' rows lie past 2^32 bytes
    w = torch.zeros(experts, n, k // 8, dtype=torch.int32, device="cuda")
    v, s, x, sx, _ = operands(torch, 2, n, k, 128, "float16", 7)
    w[-1] = pack(torch, v)
    scale = torch.zeros(experts, n, k // 128, dtype=torch.float16, device="cuda")
    scale[-1] = s
    ids = torch.full((2, 1), experts - 1, dtype=torch.int32, device="cuda")
    y = loom.loom_i4_matvec_routed(w, scale, experts, n, k, 128, x, sx, ids)
    assert torch.equal(y, loom.loom_i4_matvec_routed(w[-1:].clone(), s.clone(), 1, n, k, 128, x, sx, torch.zeros_like(ids)))
    check(torch, y[:, -50:], *definition(torch, v[-50:], s[-50:], x, sx, 128), k, 128)


@pytest.mark.parametrize("t,n,k", [((1 << 24) + 37, 1, 8), ((1 << 25) + 1, 2, 8)])
def test_tokens_of_several_launches(env, t, n, k):
    # whole sums: exact, whatever the order
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(n)
    v = torch.randint(-8, 8, (n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.where(torch.arange(t, device="cuda") % 3 == 0, 2.0, 0.5)
    y = torch.full((t + 3, n), 7.0, device="cuda")
    loom.loom_i4_matvec(pack(torch, v), torch.ones(n, 1, device="cuda"), n, k, 32, x, sx, t, y=y)
    want = (x.float() @ v.float().t()) * sx[:, None]       # (below 2^14: exact in f32 as well)
    assert torch.equal(y[:t], want) and bool((y[t:] == 7.0).all())
