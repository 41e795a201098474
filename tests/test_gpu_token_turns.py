"""Work that takes a CTA several turns: rows walked over through the read-ahead ring (more turns than the
ring has stages, so that slots are filled again), and products of more tiles than fit the GPU at a time.

Tolerances as in test_gpu_layer_norm.py: u = 2^-24, an f32 result within 128 u (and one addition more per
1024 elements and thread) of the sum of the magnitudes it is made of; 16-bit results half a unit of their
type more.  A column's sum over the rows takes an addition for each row of its CTA, one for each 32
CTAs and at most 32 after, and its terms a few roundings: 24 u."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"float32": 0.0, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 1e-44, "float16": 2.0 ** -25, "bfloat16": 1e-40}


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _turns(torch, loom, op, rows, width, dtype, matrices):
    """(turns of a CTA, CTAs), from the geometry; a ring with fewer stages than that is asked for."""
    code = {"float32": loom.LOOM_F32, "float16": loom.LOOM_F16, "bfloat16": loom.LOOM_BF16}[dtype]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    L = loom.loom_token_launch_config(op, [rows, width, code, 1, sms])
    slot = (width * (4 if dtype == "float32" else 2) + 30) // 16 * 16 * matrices * L["units_per_cta"]
    stages, turns = L["smem_bytes"] // (slot + 8), rows // (L["grid"][0] * L["units_per_cta"])
    assert 2 <= stages < turns
    return turns + 1, L["grid"][0], L["units_per_cta"]


def _matrix(torch, g, rows, width, dtype, pad, off, shift):
    buf = torch.randn(rows * (width + pad) + off, generator=g, device="cuda") * 1.7 + shift
    return buf.to(getattr(torch, dtype))[off:].view(rows, width + pad)[:, :width]


def _statistics(x, eps=1e-5):
    x = x.double()
    mean = x.mean(1)
    return mean, 1 / (((x - mean[:, None]).square().mean(1) + eps).sqrt())


# every width takes another number of columns and rows a thread and a turn, or another kind of copy
SHAPES = [(2501, 8192, "bfloat16"), (2501, 8192, "float32"), (2501, 5001, "float32"), (3001, 5001, "bfloat16"), (12001, 1028, "float16"),
          (25001, 516, "bfloat16"), (30001, 513, "float32"), (16001, 2048, "bfloat16"), (6001, 4096, "float32")]


@pytest.mark.parametrize("rows,width,dtype", SHAPES + [(701, 20000, "bfloat16")])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (8, 0)])
def test_forward_over_many_turns(env, rows, width, dtype, pad, off):
    torch, loom = env
    _turns(torch, loom, loom.LOOM_OP_LAYER_NORM, rows, width, dtype, 1)
    g = torch.Generator(device="cuda").manual_seed(width)
    x = _matrix(torch, g, rows, width, dtype, pad, off, 0.5)
    gain, bias = 1 + 0.3 * torch.randn(width, generator=g, device="cuda"), torch.randn(width, generator=g, device="cuda")
    out = torch.full((rows + 2, width + pad), float("nan"), dtype=x.dtype, device="cuda")
    y, mean, rstd = loom.loom_layer_norm(x, gain, bias, 1e-5, y=out[1:rows + 1, :width])
    wm, wr = _statistics(x)
    xhat = (x.double() - wm[:, None]) * wr[:, None]
    want, e, size = xhat * gain.double() + bias.double(), (128 + width / 1024) * U, x.double().abs().mean(1)
    assert bool(((mean.double() - wm).abs() <= e * size).all())
    assert bool(((rstd.double() - wr).abs() <= e * wr + wr.pow(3) * (e * size).square()).all())
    scale = gain.double().abs() * (xhat.abs() + (size * wr)[:, None]) + bias.double().abs()
    assert bool(((y.double() - want).abs() <= e * scale + HALF[dtype] * want.abs() * 1.01 + TINY[dtype]).all())
    bytes_ = [loom.loom_layer_norm_i8(x, gain, bias), loom.loom_quantize_tokens(x)] if width % 4 == 0 else []
    # a few rows at a time, of one turn each: the same bits
    for at in (0, 1, rows // 2, rows - 100):
        part = x[at:at + 100]
        assert all(torch.equal(a, b[at:at + 100]) for a, b in zip(loom.loom_layer_norm(part, gain, bias, 1e-5), (y, mean, rstd)))
        for call, whole in zip((lambda p: loom.loom_layer_norm_i8(p, gain, bias), loom.loom_quantize_tokens), bytes_):
            assert all(torch.equal(a, b[at:at + 100]) for a, b in zip(call(part), whole))
    # quantisation's own definition: single f32 roundings
    if bytes_:
        q, s = bytes_[1]
        f = x.float()
        amax = f.abs().amax(1)
        full = torch.full_like(amax, 127.0)
        assert torch.equal(s, amax / full)
        assert torch.equal(q.view(torch.int8), torch.round(f * (full / amax)[:, None]).to(torch.int8))
    # in place
    keep = y.clone()
    loom.loom_layer_norm(x, gain, bias, 1e-5, y=x)
    assert torch.equal(x, keep)
    out[1:rows + 1, :width] = float("nan")
    assert bool(torch.isnan(out).all())


@pytest.mark.parametrize("rows,width,dtype", SHAPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (8, 0)])
def test_backward_over_many_turns(env, rows, width, dtype, pad, off):
    torch, loom = env
    turns, ctas, rows_a_turn = _turns(torch, loom, loom.LOOM_OP_LAYER_NORM_BACKWARD, rows, width, dtype, 2)
    g = torch.Generator(device="cuda").manual_seed(width + 1)
    x, dy = _matrix(torch, g, rows, width, dtype, pad, off, 0.5), _matrix(torch, g, rows, width, dtype, pad, off, 0.1)
    gain = 1 + 0.3 * torch.randn(width, generator=g, device="cuda")
    mean, rstd = (v.float() for v in _statistics(x))
    out = torch.full((rows + 2, width + pad), float("nan"), dtype=x.dtype, device="cuda")
    dx, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, dx=out[1:rows + 1, :width])
    r = rstd.double()[:, None]
    xhat, d = (x.double() - mean.double()[:, None]) * r, dy.double()
    gd = d * gain.double()
    want = r * (gd - gd.mean(1, keepdim=True) - xhat * (gd * xhat).mean(1, keepdim=True))
    size = r * (gd.abs() + gd.abs().mean(1, keepdim=True) + xhat.abs() * (gd * xhat).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= 128 * U * size + HALF[dtype] * want.abs() * 1.01 + TINY[dtype]).all())
    steps = (turns * rows_a_turn + ctas / 32 + 32 + 24) * U
    assert bool(((dgain.double() - (d * xhat).sum(0)).abs() <= steps * (d * xhat).abs().sum(0)).all())
    assert bool(((dbias.double() - d.sum(0)).abs() <= steps * d.abs().sum(0)).all())
    for at in (0, 1, rows // 2, rows - 100):
        cut = slice(at, at + 100)
        assert torch.equal(loom.loom_layer_norm_backward(dy[cut], x[cut], mean[cut], rstd[cut], gain)[0], dx[cut])
    only = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, want_dx=False)
    assert only[0] is None and torch.equal(only[1], dgain) and torch.equal(only[2], dbias)
    keep = dx.clone()
    assert torch.equal(loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, want_params=False, workspace=None)[0], keep)
    loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, dx=dy)            # in dy's place
    assert torch.equal(dy, keep)
    out[1:rows + 1, :width] = float("nan")
    assert bool(torch.isnan(out).all())


# single CTAs (up to 32 tokens), pairs, and pairs with tiles of two halves; k below and above the 1024 of
# one accumulator, whole 16-byte rows and not; over 16 tiles of tokens
@pytest.mark.parametrize("t,n,k", [(20, 25000, 2052), (20, 25000, 272), (32, 40001, 1040), (40, 25000, 272), (40, 25000, 1044), (128, 30001, 2064),
                                   (100, 25003, 132), (300, 15000, 1044), (300, 15000, 2064), (256, 40000, 144), (201, 25000, 260),
                                   (4500, 1300, 132), (4500, 1300, 1056), (8200, 700, 528)])
def test_products_of_more_tiles_than_the_gpu_holds(env, t, n, k):
    torch, loom = env
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    L = loom.loom_token_launch_config(loom.LOOM_OP_I8_MATMUL, [t, n, k, 1, loom.LOOM_PATH_TENSOR, sms])
    channels = 128 if t <= 32 else 256
    assert -(-n // channels) * -(-t // 256) > L["grid"][0] // L["cluster"][0]
    g = torch.Generator(device="cuda").manual_seed(t + n + k)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sx, sw, bias = (torch.rand(s, generator=g, device="cuda") + 1e-3 for s in (t, n, n))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, acc = loom.loom_i8_matmul_ex(w, sw, n, k, x, sx, t, bias=bias, want_acc=True, error=err, tuning=loom.make_tuning(path=loom.LOOM_PATH_TENSOR))
    want = torch.matmul(x.double(), w.double().t())          # whole numbers below 2^53: exact
    assert int(err) == 0 and torch.equal(acc.double(), want)
    assert torch.equal(y, want.float() * (sw[None, :] * sx[:, None]) + bias)
