"""The row operators' copies ahead, when they do not land: the waits end, the rows are read directly,
and the results are those of a call whose copies came (the same bits, no error)."""
import pytest

from gpu_util import injected_stall, loom_module, loom_test_module, require_gpu

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module(), loom_test_module()


def _turns(loom, op, rows, width, dtype):
    L = loom.loom_token_launch_config(op, [rows, width, dtype, 1, SMS])
    return -(-rows // (L["grid"][0] * L["units_per_cta"]))


@pytest.mark.parametrize("rows,width,dtype,pad", [(1500, 8192, "bfloat16", 0), (1301, 5001, "float32", 1), (4000, 1028, "float16", 4)])
def test_rows_whose_copies_do_not_land(env, rows, width, dtype, pad):
    torch, loom, hooks = env
    code = {"float32": loom.LOOM_F32, "float16": loom.LOOM_F16, "bfloat16": loom.LOOM_BF16}[dtype]
    assert _turns(loom, loom.LOOM_OP_LAYER_NORM, rows, width, code) > 2
    assert _turns(loom, loom.LOOM_OP_LAYER_NORM_BACKWARD, rows, width, code) > 2
    g = torch.Generator(device="cuda").manual_seed(width)
    x, dy = (torch.randn(rows, width + pad, generator=g, device="cuda").to(getattr(torch, dtype))[:, :width] for _ in range(2))
    gain, bias = torch.randn(width, generator=g, device="cuda"), torch.randn(width, generator=g, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def calls(m):
        y, mean, rstd = m.loom_layer_norm(x, gain, bias)
        out = [y, mean, rstd, *m.loom_layer_norm_backward(dy, x, mean, rstd, gain)]
        if width % 4 == 0:
            out += [*m.loom_quantize_tokens(x, error=err), *m.loom_layer_norm_i8(x, gain, bias, error=err)]
        return out

    want = calls(loom)
    with injected_stall(hooks):
        got = calls(hooks)
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and int(err) == 0
    in_place = x.clone()
    with injected_stall(hooks):
        hooks.loom_layer_norm(in_place, gain, bias, y=in_place)
        torch.cuda.synchronize()
    assert torch.equal(in_place, want[0])
    assert all(torch.equal(a, b) for a, b in zip(want, calls(hooks)))        # and the next calls are as ever
