"""Layer norm's backward pass on rows wider than 8192, where a row's sums and its columns'
sums are taken by different launches: which outputs need a workspace, and the widest rows.

Tolerances as in test_gpu_layer_norm.py: u = 2^-24, a sum within 128 u (and one addition more
per 1024 elements and thread) of the sum of its magnitudes."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _inputs(torch, rows, width, dtype, pad=0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = (torch.randn(rows, width + pad, generator=g, device="cuda").to(getattr(torch, dtype))[:, :width] for _ in range(2))
    gain = 1 + 0.3 * torch.randn(width, generator=g, device="cuda")
    xd = x.double()
    mean = xd.mean(1)
    rstd = 1 / torch.sqrt((xd - mean[:, None]).square().mean(1) + 1e-5)
    return x, dy, gain, mean.float(), rstd.float()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,width,pad", [(3, 8193, 0), (5, 9000, 0), (4, 16384, 8), (1, 40001, 3)])
def test_dx_alone_needs_no_workspace(env, rows, width, pad, dtype):
    torch, loom = env
    x, dy, gain, mean, rstd = _inputs(torch, rows, width, dtype, pad)
    dx, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain)
    for workspace in (None, "auto", torch.empty(loom.loom_layer_norm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")):
        alone = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, want_params=False, workspace=workspace)
        assert torch.equal(alone[0], dx) and alone[1] is None and alone[2] is None
    for into in (dy.clone(), x.clone()):                      # in the place of either input
        args = (into, x) if torch.equal(into, dy) else (dy, into)
        assert torch.equal(loom.loom_layer_norm_backward(*args, mean, rstd, gain, dx=into, want_params=False, workspace=None)[0], dx)
    only = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, want_dx=False)
    assert only[0] is None and torch.equal(only[1], dgain) and torch.equal(only[2], dbias)
    with pytest.raises(loom.LoomError) as e:                  # the columns' sums do need one
        loom.loom_layer_norm_backward(dy, x, mean, rstd, gain, workspace=None)
    assert e.value.status == loom.LOOM_ERR_ARG


def test_rows_of_over_sixteen_million_columns(env):
    # more than 65535 blocks of 256 columns, an odd width: one element an access
    torch, loom = env
    rows, width = 2, 65535 * 256 + 1
    x, dy, gain, mean, rstd = _inputs(torch, rows, width, "float32")
    dx, dgain, dbias = loom.loom_layer_norm_backward(dy, x, mean, rstd, gain)
    e = (128 + width / 1024) * U
    for r in range(rows):
        xhat, g = (x[r].double() - mean[r].double()) * rstd[r].double(), dy[r].double() * gain.double()
        want = rstd[r].double() * (g - g.mean() - xhat * (g * xhat).mean())
        size = rstd[r].double() * (g.abs() + g.abs().mean() + xhat.abs() * (g * xhat).abs().mean())
        assert bool(((dx[r].double() - want).abs() <= e * size).all())
    terms = dy.double() * (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    steps = (rows + 24) * U
    assert bool(((dgain.double() - terms.sum(0)).abs() <= steps * terms.abs().sum(0)).all())
    assert bool(((dbias.double() - dy.double().sum(0)).abs() <= steps * dy.double().abs().sum(0)).all())
