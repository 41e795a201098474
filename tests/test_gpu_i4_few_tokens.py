"""4-bit products of one and two tokens: many rows a CTA, and rows off 16 bytes (definition and tolerance of test_gpu_i4_matvec.py)."""
import pytest

from test_gpu_i4_matvec import check, definition, env, operands, pack  # noqa: F401

pytestmark = pytest.mark.gpu


def whole(torch, t, n, k, seed, lead=()):
    """Operands whose scaled sums and biases are whole numbers below 2^24: exact in f32, in whatever order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-8, 8, (*lead, n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.where(torch.arange(t, device="cuda") % 2 == 0, 2.0, 1.0)
    return v, x, sx, torch.randint(-1000, 1000, (*lead, n), generator=g, device="cuda").float()


@pytest.mark.parametrize("t", [1, 2])
@pytest.mark.parametrize("n,k", [(200000, 64), (262144, 128), (330001, 72), (500003, 8)])
def test_more_rows_than_a_cta_holds_sums_of(env, t, n, k):  # noqa: F811
    # a CTA of two an SM has 658 rows and more; it holds the sums of 512
    torch, loom = env
    v, x, sx, bias = whole(torch, t, n, k, n + t)
    groups = -(-k // 32)
    y = loom.loom_i4_matvec(pack(torch, v), torch.ones(n, groups, device="cuda"), n, k, 32, x, sx, t, bias=bias)
    want = (x.float() @ v.float().t()) * sx[:, None] + bias        # (whole numbers: exact as well)
    assert torch.equal(y, want)


@pytest.mark.parametrize("k", [32, 40])
def test_more_rows_of_experts_than_a_cta_holds_sums_of(env, k):  # noqa: F811
    # 3 of 16 experts of 90001 rows: runs of a CTA that go on past 512 rows, and into the next matrix; one of them by two tokens
    torch, loom = env
    experts, n = 16, 90001
    v, x, sx, bias = whole(torch, 2, n, k, k, (experts,))
    ids = torch.tensor([[3, 15], [15, -1]], dtype=torch.int32, device="cuda")
    groups = -(-k // 32)
    y = loom.loom_i4_matvec_routed(pack(torch, v), torch.ones(experts, n, groups, device="cuda"), experts, n, k, 32, x, sx, ids, bias=bias)
    for pair, (token, e) in enumerate(((0, 3), (0, 15), (1, 15))):
        assert torch.equal(y[pair], (v[e].float() @ x[token].float()) * sx[token] + bias[e]), pair
    assert not bool(y[3].any())


@pytest.mark.parametrize("t", [1, 2])
@pytest.mark.parametrize("n,k,group,offset", [(77, 1024, 64, 1), (77, 1024, 128, 2), (50, 1032, 32, 0), (33, 1048, 64, 3), (90, 4104, 128, 0), (7, 16392, 256, 0), (1300, 4104, 32, 2),
                                              (400, 8200, 4096, 1), (1, 131064, 128, 0), (200, 40, 32, 3)])
def test_rows_off_16_bytes(env, t, n, k, group, offset):  # noqa: F811
    torch, loom = env
    v, s, x, sx, bias = operands(torch, t, n, k, group, "float16", k + offset + t)
    w = torch.empty(n * k // 8 + 8, dtype=torch.int32, device="cuda")[offset:offset + n * k // 8]
    w.copy_(pack(torch, v).view(-1))
    xb = torch.empty(t * k // 4 + 8, dtype=torch.int32, device="cuda")[offset:offset + t * k // 4]
    xb.copy_(x.view(torch.int32).view(-1))
    sb = torch.empty(s.numel() + 8, dtype=s.dtype, device="cuda")[offset:offset + s.numel()]
    sb.copy_(s.view(-1))
    y = loom.loom_i4_matvec(w, sb, n, k, group, xb, sx, t, bias=bias)
    check(torch, y, *definition(torch, v, s, x, sx, group, bias), k, group)
    assert torch.equal(y, loom.loom_i4_matvec(w, sb, n, k, group, xb, sx, t, bias=bias))


@pytest.mark.parametrize("n,k,offset", [(300, 1032, 0), (65, 1024, 3), (2000, 72, 1)])
def test_two_tokens_of_an_expert_off_16_bytes(env, n, k, offset):  # noqa: F811
    # 8 experts and 2 pairs of one: the kernel of one token, twice; all to the only expert: the kernel of two
    torch, loom = env
    for experts, ids in ((8, [[5], [5]]), (1, [[0], [0]])):
        v, s, x, sx, bias = operands(torch, 2, n, k, 32, "bfloat16", n + k, (experts,))
        w = torch.empty(v.numel() // 8 + 8, dtype=torch.int32, device="cuda")[offset:offset + v.numel() // 8]
        w.copy_(pack(torch, v).view(-1))
        at = torch.tensor(ids, dtype=torch.int32, device="cuda")
        y = loom.loom_i4_matvec_routed(w, s, experts, n, k, 32, x, sx, at, bias=bias)
        e = ids[0][0]
        check(torch, y, *definition(torch, v[e], s[e], x, sx, 32, bias[e]), k, 32)
