"""loom_quantize_tokens and loom_i8_matmul on the GPU: whole numbers and defined roundings
are compared for equality, against int64 sums and the definition's own f32 steps."""
import numpy as np
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _bytes(torch, g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def _want_acc(torch, x, w):
    """int64 sums: f64 products of whole numbers below 2^53 are exact."""
    return torch.matmul(x.double(), w.double().t()).to(torch.int64)


def _want_y(torch, acc, sw, sx, bias, dtype):
    y = acc.float() * (sw[None, :] * sx[:, None])     # single f32 roundings, as defined
    if bias is not None:
        y = y + bias
    return y.to(dtype)


def _check(env, t, n, k, dtype, bias, path=0, seed=1, full=None):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(seed)
    if full is None:
        x, w = _bytes(torch, g, t, k), _bytes(torch, g, n, k)
    else:
        x, w = (torch.full((a, k), full, dtype=torch.int8, device="cuda") for a in (t, n))
    sx, sw = torch.rand(t, generator=g, device="cuda") + 1e-3, torch.rand(n, generator=g, device="cuda") + 1e-3
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    # rows between canaries, further apart than they are long
    y = torch.full((t + 2, n + 5), float("nan"), dtype=dtype, device="cuda")
    acc = torch.full((t + 2, n), -7777, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loom.loom_i8_matmul_ex(w, sw, n, k, x, sx, t, bias=b, y=y[1:t + 1, :n], acc=acc[1:t + 1], error=err,
                           tuning=loom.make_tuning(path=path))
    torch.cuda.synchronize()
    want = _want_acc(torch, x, w)
    assert int(err) == 0
    assert torch.equal(acc[1:t + 1].long(), want)
    assert torch.equal(y[1:t + 1, :n], _want_y(torch, want, sw, sx, b, dtype))
    assert bool((acc[0] == -7777).all()) and bool((acc[t + 1] == -7777).all())
    y[1:t + 1, :n] = float("nan")
    assert bool(torch.isnan(y).all())


PATHS = ("auto", "direct", "tensor")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t,n,k", [
    (1, 1, 4), (1, 7, 16), (2, 129, 64), (3, 1000, 260), (4, 257, 4096), (5, 64, 2052), (8, 300, 1040), (9, 31, 128),
    (16, 513, 2048), (17, 96, 100), (64, 255, 1024), (65, 1001, 516), (127, 128, 144), (128, 256, 3200), (129, 511, 1028),
    (200, 1000, 4108), (256, 2049, 272), (257, 33, 8192), (500, 777, 1536), (1025, 640, 384)])
def test_products(env, t, n, k, path):
    _check(env, t, n, k, env[0].float32, bias=True, path=_path(env[1], path))


def _path(loom, name):
    return {"auto": loom.LOOM_PATH_AUTO, "direct": loom.LOOM_PATH_DIRECT, "tensor": loom.LOOM_PATH_TENSOR}[name]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t,n,k,bias", [(1, 100, 64, False), (12, 259, 1040, True), (130, 300, 2048, False), (300, 513, 260, True)])
def test_output_types(env, t, n, k, bias, dtype):
    _check(env, t, n, k, getattr(env[0], dtype), bias)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", [1, 16, 130])
def test_largest_sums(env, t, path):
    # -128 x -128 over the longest row: |acc| = 2147418112, 2^31 - 65536
    _check(env, t, 40, 131068, env[0].float32, bias=False, path=_path(env[1], path), full=-128)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("t", [3, 40, 140])
def test_no_columns_and_no_work(env, t, path):
    torch, loom = env
    b = torch.arange(9, dtype=torch.float32, device="cuda")
    empty = torch.empty(0, dtype=torch.int8, device="cuda")
    one = torch.ones(max(t, 9), device="cuda")
    y, acc = loom.loom_i8_matmul_ex(empty, one, 9, 0, empty, one, t, bias=b, want_acc=True,
                                    tuning=loom.make_tuning(path=_path(loom, path)))
    assert torch.equal(y, b.expand(t, 9)) and not bool(acc.any())
    assert loom.loom_i8_matmul(empty, one, 9, 64, empty, one, 0)[0].shape == (0, 9)


@pytest.mark.parametrize("t", [2, 40, 300])
@pytest.mark.parametrize("wo,xo", [(4, 0), (0, 4), (12, 8)])
def test_rows_off_sixteen_bytes(env, t, wo, xo):
    torch, loom = env
    n, k = 300, 1024
    g = torch.Generator(device="cuda").manual_seed(t)
    w, x = _bytes(torch, g, n * k + 16), _bytes(torch, g, t * k + 16)
    w, x = w[wo:wo + n * k].view(n, k), x[xo:xo + t * k].view(t, k)
    sx, sw = torch.rand(t, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    y, acc = loom.loom_i8_matmul(w, sw, n, k, x, sx, t, want_acc=True)
    want = _want_acc(torch, x, w)
    assert torch.equal(acc.long(), want) and torch.equal(y, _want_y(torch, want, sw, sx, None, torch.float32))


def test_nan_scale_reaches_its_token_alone(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(3)
    w, x = _bytes(torch, g, 64, 128), _bytes(torch, g, 20, 128)
    sx, sw = torch.ones(20, device="cuda"), torch.ones(64, device="cuda")
    sx[7] = float("nan")
    y, _ = loom.loom_i8_matmul(w, sw, 64, 128, x, sx, 20)
    assert bool(torch.isnan(y[7]).all()) and int(torch.isnan(y).sum()) == 64


def test_on_another_stream_and_twice(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(5)
    w, x = _bytes(torch, g, 700, 2048), _bytes(torch, g, 150, 2048)
    sx, sw = torch.rand(150, generator=g, device="cuda"), torch.rand(700, generator=g, device="cuda")
    first, _ = loom.loom_i8_matmul(w, sw, 700, 2048, x, sx, 150)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(first)
    for _ in range(3):
        loom.loom_i8_matmul(w, sw, 700, 2048, x, sx, 150, y=y, stream=s)
    s.synchronize()
    assert torch.equal(first, y)


# ---- tokens to bytes -------------------------------------------------------------------
def _want_bytes(x):
    """The definition's f32 steps, in numpy (IEEE single)."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    tiny = ~(amax >= np.float32(2.0 ** -100))
    with np.errstate(all="ignore"):
        inv = np.where(tiny, np.float32(0), np.float32(127) / amax).astype(np.float32)
        scale = np.where(tiny, np.float32(0), amax / np.float32(127)).astype(np.float32)
        q = np.rint(x * inv[:, None])
    bad = ~np.isfinite(x).all(1)
    scale[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), scale, bool(bad.any())


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k,pad,off", [(1, 4, 0, 0), (3, 64, 0, 0), (9, 508, 4, 0), (5, 512, 8, 0), (2, 516, 1, 3), (4, 4108, 0, 0),
                                         (3, 16384, 0, 1), (2, 16388, 4, 0), (2, 40000, 0, 0), (2, 131068, 0, 0), (70, 128, 0, 0)])
def test_quantize(env, dtype, t, k, pad, off):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(k + pad)
    buf = (torch.randn(t * (k + pad) + off, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    x = buf[off:].view(t, k + pad)[:, :k]
    if t > 2:
        x[1] = 0
        x[2] = 1e-6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, scale = loom.loom_quantize_tokens(x, error=err)
    want_q, want_s, _ = _want_bytes(x.float().cpu().numpy())
    assert np.array_equal(q.view(torch.int8).cpu().numpy(), want_q) and np.array_equal(scale.cpu().numpy(), want_s)
    assert int(err) == 0


def test_quantize_special_values(env):
    torch, loom = env
    x = torch.randn(8, 256, device="cuda")
    x[0, 3], x[1, 255], x[2, 0] = float("nan"), float("inf"), -float("inf")
    x[3] = 1e-38                       # below 2^-100: nothing
    x[4] = 3.4e38                      # near the largest f32
    x[5, :] = -0.0
    x[6] = torch.linspace(-127, 127, 256, device="cuda").round() + 0.5   # ties
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, scale = loom.loom_quantize_tokens(x, error=err)
    want_q, want_s, bad = _want_bytes(x.cpu().numpy())
    assert np.array_equal(q.view(torch.int8).cpu().numpy(), want_q)
    assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)
    assert bad and int(err) == loom.LOOM_DEVERR_NONFINITE
    q, scale = loom.loom_quantize_tokens(torch.empty(3, 0, device="cuda"))
    assert not bool(scale.any())


def test_tokens_through_a_product(env):
    # float tokens -> bytes -> product stays within the quantisation's own error bound:
    # |x - q s| <= s / 2 (+ rounding) per element, so |y - x W^T sw| <= sw s/2 sum |w|
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(33, 512, generator=g, device="cuda")
    w = _bytes(torch, g, 200, 512)
    sw = torch.rand(200, generator=g, device="cuda") * 0.01
    q, s = loom.loom_quantize_tokens(x)
    y, _ = loom.loom_i8_matmul(w, sw, 200, 512, q, s, 33)
    want = torch.matmul(x.double(), w.double().t()) * sw.double()
    bound = 0.5001 * s.double()[:, None] * sw.double() * w.double().abs().sum(1) + 1e-6 * want.abs()
    assert bool(((y.double() - want).abs() <= bound).all())
