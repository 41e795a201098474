"""The token operators' tensors and streams as the binding takes them on a GPU."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def _refused(loom, call, *args, **kw):
    with pytest.raises(loom.LoomError) as e:
        call(*args, **kw)
    return e.value.status


def test_product_operands_on_the_host(env):
    torch, loom = env
    n, k, t = 40, 64, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    w, x = (torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((n, k), (t, k)))
    sw, sx, bias = (torch.rand(s, generator=g, device="cuda") for s in (n, t, n))
    want = loom.loom_i8_matmul(w, sw, n, k, x, sx, t, bias=bias, want_acc=True)
    args = [w, sw, n, k, x, sx, t]
    for i in (1, 4, 5):
        host = list(args)
        host[i] = host[i].cpu()
        assert _refused(loom, loom.loom_i8_matmul, *host) == loom.LOOM_ERR_ARG
    for more in ({"bias": bias.cpu()}, {"y": torch.empty(t, n)}, {"acc": torch.empty(t, n, dtype=torch.int32)}):
        assert _refused(loom, loom.loom_i8_matmul, *args, **more) == loom.LOOM_ERR_ARG
    assert _refused(loom, loom.loom_i8_matmul_ex, *args, error=torch.zeros(1, dtype=torch.int32)) == loom.LOOM_ERR_ARG
    # pinned host memory is the device's to read, and addresses are taken as they are
    got = loom.loom_i8_matmul(*args, bias=bias.cpu().pin_memory(), want_acc=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(loom.loom_i8_matmul(*args, bias=bias.data_ptr())[0], want[0])
    # outputs with room around them, in the caller's type
    y = torch.full((t + 1, n + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert loom.loom_i8_matmul(*args, bias=bias, y=y)[0] is y
    assert torch.equal(y[:t, :n], want[0].to(torch.bfloat16)) and int(torch.isnan(y).sum()) == (t + 1) * (n + 3) - t * n
