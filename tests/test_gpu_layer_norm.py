"""Layer norm on the GPU, forward, to bytes and backward, against the formulas in 64 bits,
and the gradients against differences.

Tolerances.  u = 2^-24.  A sum over a row passes at most 32 additions in a thread and 10
across threads, so it is within 42 u of the sum of magnitudes; the squares are taken about
a mean that is off by that much.  With a few more roundings per element every f32 result
stays within 128 u of the sum of the magnitudes it is made of (long rows: one addition more
per 1024 elements and thread).  16-bit results add half a unit of their type."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 0.0, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 1e-44, "float16": 2.0 ** -25, "bfloat16": 1e-40}
DTYPES = ("float32", "float16", "bfloat16")


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _rows(torch, g, rows, width, dtype, pad=0, off=0, shift=0.5):
    buf = torch.randn(rows * (width + pad) + off, generator=g, device="cuda") * 1.7 + shift
    return buf.to(getattr(torch, dtype))[off:].view(rows, width + pad)[:, :width]


def _forward(torch, x, gain, bias, eps):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = xhat if gain is None else xhat * gain.double()
    return (y if bias is None else y + bias.double()), mean, rstd, xhat


def _steps(width):
    return (128 + width / 1024) * U


SHAPES = [(1, 1), (3, 2), (5, 31), (4, 64), (7, 255), (9, 512), (3, 513), (2, 1000), (6, 2048), (3, 4097), (2, 5001), (2, 8192), (2, 8193),
          (2, 16384), (2, 16392), (2, 16385), (1, 32768), (2, 32769), (1, 40000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("pad,off,params", [(0, 0, True), (3, 1, False), (8, 0, True)])
def test_forward(env, rows, width, dtype, pad, off, params):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(width)
    x = _rows(torch, g, rows, width, dtype, pad, off)
    gain = 1 + 0.3 * torch.randn(width, generator=g, device="cuda") if params else None
    bias = torch.randn(width, generator=g, device="cuda") if params else None
    out = torch.full((rows + 2, width + pad), float("nan"), dtype=x.dtype, device="cuda")
    y, mean, rstd = loom.loom_layer_norm(x, gain, bias, 1e-5, y=out[1:rows + 1, :width])
    want, wm, wr, xhat = _forward(torch, x, gain, bias, 1e-5)
    e, size = _steps(width), x.double().abs().mean(1)
    assert bool(((mean.double() - wm).abs() <= e * size).all())
    # var is off by at most e var plus the square of the mean's error
    assert bool(((rstd.double() - wr).abs() <= e * wr + wr.pow(3) * (e * size).square()).all())
    scale = (gain.double().abs() if params else 1) * (xhat.abs() + (size * wr)[:, None]) + (bias.double().abs() if params else 0)
    assert bool(((y.double() - want).abs() <= e * scale + HALF[dtype] * want.abs() * 1.01 + TINY[dtype]).all())
    out[1:rows + 1, :width] = float("nan")
    assert bool(torch.isnan(out).all())


def test_forward_in_place_without_stats_and_offsets_far_from_zero(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(2)
    x = _rows(torch, g, 33, 700, "float32", shift=3000.0)
    want, _, wr, xhat = _forward(torch, x, None, None, 1e-5)
    size = x.double().abs().mean(1)
    y, mean, rstd = loom.loom_layer_norm(x, y=x, want_stats=False)
    assert mean is None and rstd is None and y.data_ptr() == x.data_ptr()
    assert bool(((y.double() - want).abs() <= 128 * U * (xhat.abs() + (size * wr)[:, None])).all())


def test_constant_and_non_finite_rows(env):
    torch, loom = env
    x = torch.randn(5, 300, device="cuda")
    x[1] = 2.5                       # no spread: y = bias
    x[2, 7] = float("nan")
    x[3, 0] = float("inf")
    bias = torch.randn(300, device="cuda")
    y, mean, rstd = loom.loom_layer_norm(x, None, bias, 1e-5)
    assert torch.equal(y[1], bias) and float(mean[1]) == 2.5
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isfinite(y[[0, 4]]).all())
    assert loom.loom_layer_norm(torch.empty(0, 8, device="cuda"))[0].shape == (0, 8)
    assert loom.loom_layer_norm(torch.empty(3, 0, device="cuda"))[0].shape == (3, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width,pad",
                         [(1, 4, 0), (5, 64, 0), (3, 512, 2), (4, 1028, 0), (2, 4096, 0), (2, 16384, 4), (2, 20000, 0), (2, 40000, 0)])
def test_to_bytes(env, rows, width, pad, dtype):
    # the bytes stand for values within half a step (and the f32 error) of the norm's output
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(width + 1)
    x = _rows(torch, g, rows, width, dtype, pad)
    gain, bias = 1 + 0.3 * torch.randn(width, generator=g, device="cuda"), torch.randn(width, generator=g, device="cuda")
    q, scale = loom.loom_layer_norm_i8(x, gain, bias, 1e-5)
    want, _, wr, xhat = _forward(torch, x, gain, bias, 1e-5)
    e = _steps(width)
    err = e * (gain.double().abs() * (xhat.abs() + (x.double().abs().mean(1) * wr)[:, None]) + bias.double().abs())
    amax = want.abs().amax(1)
    s = scale.double()
    assert bool(((s * 127 - amax).abs() <= err.amax(1) + 4 * U * amax).all())
    v = q.view(torch.int8).double() * s[:, None]
    assert bool(((v - want).abs() <= 0.5 * s[:, None] + err + 256 * U * s[:, None]).all())
    assert bool((q.view(torch.int8).abs().amax(1) == 127).all())


def test_to_bytes_flags_a_row_that_is_not_finite(env):
    torch, loom = env
    x = torch.randn(4, 64, device="cuda")
    x[2, 5] = float("inf")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, scale = loom.loom_layer_norm_i8(x, error=err)
    assert int(err) == loom.LOOM_DEVERR_NONFINITE and bool(torch.isnan(scale[2])) and int(torch.isnan(scale).sum()) == 1
    assert not bool(q[2].any())


# ---- backward --------------------------------------------------------------------------
def _backward(torch, dy, x, mean, rstd, gain):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (x - mean) * rstd
    g = dy if gain is None else dy * gain.double()
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd * (g - a - xhat * b)
    size = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0), size, (dy * xhat).abs().sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 64), (3, 7), (40, 256), (1000, 96), (7, 257), (50, 1000), (700, 512), (5, 4096), (3, 5001),
                                        (6, 8192), (5, 8193), (3, 8200), (4, 20000), (1, 40001)])
@pytest.mark.parametrize("pad,off,params", [(0, 0, True), (3, 1, False), (8, 0, True)])
def test_backward(env, rows, width, dtype, pad, off, params):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    x, dy = _rows(torch, g, rows, width, dtype, pad, off), _rows(torch, g, rows, width, dtype, pad, off, 0.1)
    gain = 1 + 0.3 * torch.randn(width, generator=g, device="cuda") if params else None
    _, mean, rstd, _ = _forward(torch, x, None, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    out = torch.full((rows + 2, width + pad), float("nan"), dtype=x.dtype, device="cuda")
    dx, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, dx=out[1:rows + 1, :width])
    want, wg, wb, size, sg, sb = _backward(torch, dy, x, mean, rstd, gain)
    e = _steps(width)
    assert bool(((dx.double() - want).abs() <= e * size + HALF[dtype] * want.abs() * 1.01 + TINY[dtype]).all())
    # a column's additions: its rows in a CTA, then partial sums (of at most one per row)
    steps = (rows + 24) * U
    assert bool(((dgain.double() - wg).abs() <= steps * sg).all())
    assert bool(((dbias.double() - wb).abs() <= steps * sb).all())
    out[1:rows + 1, :width] = float("nan")
    assert bool(torch.isnan(out).all())
    again = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain)
    assert torch.equal(again[1], dgain) and torch.equal(again[2], dbias)


@pytest.mark.parametrize("rows,width", [(6, 40), (4, 700), (3, 9000)])
def test_gradients_against_differences(env, rows, width):
    # the derivative of sum(y * dy) along random directions, by central differences of the
    # 64-bit formula: its error is h^2 times a third derivative, far below the f32 bound
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(width)
    x, dy = _rows(torch, g, rows, width, "float32"), _rows(torch, g, rows, width, "float32", shift=0.0)
    gain, bias = 1 + 0.3 * torch.randn(width, generator=g, device="cuda"), torch.randn(width, generator=g, device="cuda")
    _, mean, rstd = loom.loom_layer_norm(x, gain, bias, 1e-5)
    grads = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain)
    inputs = [x.double(), gain.double(), bias.double()]
    loss = lambda v: float((_forward(torch, v[0], v[1], v[2], 1e-5)[0] * dy.double()).sum())   # noqa: E731
    h = 1e-4
    for i, grad in enumerate(grads):
        d = torch.randn(inputs[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = ([v + s * h * d if j == i else v for j, v in enumerate(inputs)] for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * h)
        got = float((grad.double() * d).sum())
        assert abs(slope - got) <= 1e-5 * float((grad.double().abs() * d.abs()).sum()) + 1e-6


def test_backward_parts_in_place_and_no_rows(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dy = _rows(torch, g, 20, 600, "bfloat16"), _rows(torch, g, 20, 600, "bfloat16")
    _, mean, rstd = loom.loom_layer_norm(x)
    dx, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd)
    only_dx = loom.loom_layer_norm_backward(dy, x, mean, rstd, want_params=False, workspace=None)
    only_params = loom.loom_layer_norm_backward(dy, x, mean, rstd, want_dx=False)
    assert torch.equal(only_dx[0], dx) and only_dx[1] is None and only_params[0] is None
    assert torch.equal(only_params[1], dgain) and torch.equal(only_params[2], dbias)
    copy = dy.clone()
    assert torch.equal(loom.loom_layer_norm_backward(copy, x, mean, rstd, dx=copy)[0], dx)
    none = x[:0]
    dx, dgain, dbias = loom.loom_layer_norm_backward(none, none, mean[:0], rstd[:0])
    assert dx.shape == (0, 600) and not bool(dgain.any()) and not bool(dbias.any())
    with pytest.raises(loom.LoomError) as e:
        loom.loom_layer_norm_backward(dy, x, mean, rstd, workspace=None)
    assert e.value.status == loom.LOOM_ERR_ARG
    short = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(loom.LoomError) as e:
        loom.loom_layer_norm_backward(dy, x, mean, rstd, workspace=short)
    assert e.value.status == loom.LOOM_ERR_ARG


def test_on_another_stream(env):
    torch, loom = env
    x = torch.randn(300, 1024, device="cuda")
    first = loom.loom_layer_norm(x)
    grads = loom.loom_layer_norm_backward(x, x, first[1], first[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        y, mean, rstd = loom.loom_layer_norm(x, stream=s)
        got = loom.loom_layer_norm_backward(x, x, mean, rstd, stream=s)
        for t in (y, mean, rstd) + got:
            t.record_stream(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first + grads, (y, mean, rstd) + got))
