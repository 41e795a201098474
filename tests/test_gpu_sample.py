"""loom_sample_tokens on the GPU against the definition: whole-number weights from f32
steps (torch's exp of the same f32 argument), then a plain walk over the sorted tokens in
Python integers.  Tokens are compared for equality."""
import math

import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
FULL = 1 << 31


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _definition(torch, logits, u, temperature, top_k, top_p, min_p):
    """(token, log probability) of one row, by the definition."""
    l = logits.float()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    m = l.max()
    if float(m) == -math.inf:
        return -1, math.nan
    order = torch.sort(l, descending=True, stable=True)[1].tolist()
    if not temperature > 0:
        return order[0], 0.0
    inv = torch.ones((), device=l.device) / torch.tensor(temperature, dtype=torch.float32, device=l.device)
    e = torch.where(l == m, torch.ones_like(l), torch.exp((l - m) * inv))
    e = torch.where(l == -math.inf, torch.zeros_like(l), e)
    w = (e * float(FULL)).to(torch.int64).tolist()
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))   # noqa: E731
    kept = order[:top_k] if top_k > 0 else order
    if f32(top_p) < 1:
        target, run, some = f32(top_p) * sum(w[i] for i in kept), 0, []
        for i in kept:
            if run < target or not some:
                some.append(i)
            run += w[i]
        kept = some
    kept = sorted(i for i in kept if w[i] >= f32(min(max(min_p, 0.0), 1.0)) * FULL)
    total = sum(w[i] for i in kept)
    at = min(max(math.floor(u * total), 0), total - 1)
    run = 0
    for i in kept:
        run += w[i]
        if run > at:
            return i, math.log(w[i] / total)
    raise AssertionError("no token")


def _check(env, logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, err_want=0):
    torch, loom = env
    rows = logits.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    token, logprob = loom.loom_sample_tokens(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, error=err)
    at = lambda v, r: v[r].item() if isinstance(v, torch.Tensor) else v   # noqa: E731
    for r in range(rows):
        want, lp = _definition(torch, logits[r], float(u[r]), at(temperature, r), at(top_k, r), at(top_p, r), at(min_p, r))
        assert int(token[r]) == want, (r, int(token[r]), want)
        got = float(logprob[r])
        # one 64-bit logarithm, rounded once to f32
        assert (math.isnan(lp) and math.isnan(got)) or abs(got - lp) <= 2.0 ** -24 * abs(lp) + 1e-12, (r, got, lp)
    assert int(err) == err_want
    return token


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 1, 1.0, 0.0), (0.8, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.1), (0.9, 50, 0.95, 0.02),
            (1.0, 3, 0.3, 0.0), (1.0, 0, 0.0, 0.0), (2.0, 100000, 0.999, 0.0), (0.0, 5, 0.5, 0.5), (0.05, 10, 0.9, 0.0), (1.0, 0, 1.0, 1.0)]


@pytest.mark.parametrize("setting", SETTINGS)
@pytest.mark.parametrize("rows,vocab,dtype", [(3, 1, "float32"), (4, 2, "float16"), (3, 33, "bfloat16"), (3, 1000, "float32"), (2, 16385, "bfloat16"),
                                              (2, 50001, "float16"), (1, 131072, "float32"), (1, 140003, "float32")])
def test_settings(env, rows, vocab, dtype, setting):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    _check(env, logits, torch.rand(rows, generator=g, device="cuda"), *setting)


def test_largest_vocabulary(env):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn(1, 393216, generator=g, device="cuda") * 3
    _check(env, logits, torch.rand(1, generator=g, device="cuda"), 0.9, 200, 0.9, 0.0)
    _check(env, logits, torch.rand(1, generator=g, device="cuda"))


def test_settings_of_each_row(env):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = 24
    logits = torch.randn(rows, 2000, generator=g, device="cuda") * 2
    t = torch.tensor([0.0, 0.5, 1.0, -1.0, float("nan"), float("inf")] * 4, device="cuda")
    k = torch.tensor([0, -3, 1, 7, 5000, 2000] * 4, dtype=torch.int32, device="cuda").roll(1)
    p = torch.tensor([1.0, 0.5, 0.9, 2.0] * 6, device="cuda")
    mp = torch.tensor([0.0, 0.3, -1.0] * 8, device="cuda")
    _check(env, logits, torch.rand(rows, generator=g, device="cuda"), t, k, p, mp)


@pytest.mark.parametrize("vocab", [5, 700, 40000])
@pytest.mark.parametrize("setting", [(1.0, 0, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (1.0, 4, 0.6, 0.0), (0.0, 0, 1.0, 0.0)])
def test_equal_logits(env, vocab, setting):
    # all equal, then a few levels: what is cut among equals goes by index
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits = torch.stack([torch.full((vocab,), -2.5, device="cuda"), torch.randint(0, 3, (vocab,), generator=g, device="cuda").float(),
                          torch.zeros(vocab, device="cuda") * torch.where(torch.rand(vocab, generator=g, device="cuda") < 0.5, 1.0, -1.0)])
    for u in (0.0, 0.37, 0.9999999):
        _check(env, logits, torch.full((3,), u, device="cuda"), *setting)


@pytest.mark.parametrize("setting", SETTINGS[:6])
def test_masked_rows(env, setting):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(8)
    v = 3000
    x = torch.randn(9, v, generator=g, device="cuda")
    inf = float("inf")
    x[0] = -inf                                     # nothing left
    x[1] = float("nan")
    x[2], x[2, 1234] = -inf, -7.0                   # one left
    x[3, ::2] = -inf
    x[4, 5:9] = float("nan")
    x[5, [17, 2900]] = inf                          # infinities share everything
    x[6] = torch.finfo(torch.float32).min           # masks of the type's lowest value
    x[7], x[7, 40:50] = torch.finfo(torch.float32).min, torch.randn(10, generator=g, device="cuda")
    x[8, 0], x[8, 1] = 3e38, -3e38                  # a difference that is infinite
    _check(env, x, torch.rand(9, generator=g, device="cuda"), *setting, err_want=loom.LOOM_DEVERR_NO_TOKEN)


@pytest.mark.parametrize("top_k", [513, 700, 1500, 2040])
@pytest.mark.parametrize("setting", [(1.0, 1.0, 0.0), (0.7, 0.9, 0.0), (1.4, 0.97, 0.05)])
def test_many_of_top_k(env, top_k, setting):
    # long lists: spread logits, levels of many equals, one crowded level among others, neighbours in index
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(top_k)
    v = 30000
    x = torch.randn(5, v, generator=g, device="cuda")
    x[1] = torch.floor(x[1] * 40) / 40
    x[2] = torch.where(torch.rand(v, generator=g, device="cuda") < 0.06, 2.0, x[2])
    x[3] -= torch.arange(v, device="cuda") * 0.002
    x[4], x[4, 29000:] = -float("inf"), torch.randn(1000, generator=g, device="cuda")
    t, p, mp = setting
    _check(env, x, torch.rand(5, generator=g, device="cuda"), t, top_k, p, mp)


@pytest.mark.parametrize("temperature", [1e-30, 3e-37, 1e-37, 3e-39, 1e-40])
@pytest.mark.parametrize("setting", [(0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.8, 0.0), (900, 0.8, 0.01)])
def test_temperatures_near_zero(env, temperature, setting):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(3)
    v = 3000
    x = torch.randn(5, v, generator=g, device="cuda")
    x[1] *= temperature                             # differences of the temperature's size
    x[2] = torch.randint(0, 9, (v,), generator=g, device="cuda") * (0.5 * temperature)
    x[3] = torch.randint(0, 3, (v,), generator=g, device="cuda").float()
    x[4], x[4, 7] = x[4] * temperature, -float("inf")
    _check(env, x, torch.rand(5, generator=g, device="cuda"), temperature, *setting)


def test_random_numbers_at_and_past_the_ends(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(6, 5000, generator=g, device="cuda")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0, 0.5], device="cuda")
    _check(env, x, u, 1.0, 0, 0.9, 0.0)
    token, _ = loom.loom_sample_tokens(x[:1], torch.full((1,), float("nan"), device="cuda"))
    assert int(token) == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 3), (3, 1)])
def test_strides_and_alignment(env, dtype, off, pad):
    torch, _ = env
    g = torch.Generator(device="cuda").manual_seed(off)
    buf = (torch.randn(4 * (1001 + pad) + off, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    x = buf[off:].view(4, 1001 + pad)[:, :1001]
    _check(env, x, torch.rand(4, generator=g, device="cuda"), 0.9, 30, 0.9, 0.01)


def test_frequencies(env):
    # the drawn tokens follow the weights: 20000 draws of a 4-token row, 5 sigma
    torch, loom = env
    n = 20000
    g = torch.Generator(device="cuda").manual_seed(21)
    row = torch.log(torch.tensor([0.5, 0.3, 0.15, 0.05], device="cuda"))
    token, _ = loom.loom_sample_tokens(row.expand(n, 4).contiguous(), torch.rand(n, generator=g, device="cuda"))
    for i, want in enumerate((0.5, 0.3, 0.15, 0.05)):
        got = float((token == i).float().mean())
        assert abs(got - want) <= 5 * math.sqrt(want * (1 - want) / n)


def test_on_another_stream_and_outputs_given(env):
    torch, loom = env
    x, u = torch.randn(64, 4000, device="cuda"), torch.rand(64, device="cuda")
    first = loom.loom_sample_tokens(x, u, top_p=0.9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    token = torch.full((66,), -7, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    loom.loom_sample_tokens(x, u, top_p=0.9, token=token[1:65], want_logprob=False, stream=s)
    s.synchronize()
    assert torch.equal(token[1:65], first[0]) and int(token[0]) == -7 and int(token[65]) == -7
