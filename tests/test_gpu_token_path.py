"""The token operators together (examples/next_token.py), and what only a whole call shows:
device waits that run out, refusals that need a device, graphs, and the tensor-core product
with row counts around its tiles."""
import importlib.util
import os

import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


@pytest.fixture(scope="module")
def example(env):
    spec = importlib.util.spec_from_file_location("next_token", os.path.join(ROOT, "examples", "next_token.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_serving_path(env, example):
    torch, _ = env
    head = example.Head(512, 5000, seed=3)
    x = torch.randn(20, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    # the greedy token is the largest of the path's own logits, and those are near the product of
    # the unquantised operands: both sides of a product are off by half a step at most
    logits = head.logits(x)
    token, logprob = head.next_token(x, torch.zeros(20, device="cuda"), temperature=0.0)
    assert torch.equal(token.long(), logits.float().argmax(1)) and not bool(logprob.any())
    w = head.weight.view(torch.int8).double()
    xd = x.double()
    norm = (xd - xd.mean(1, keepdim=True)) / torch.sqrt(xd.var(1, unbiased=False, keepdim=True) + 1e-5)
    step = norm.abs().amax(1, keepdim=True) / 127
    want = norm @ (w * head.scale.double()[:, None]).t()
    bound = 0.51 * step * (w * head.scale.double()[:, None]).abs().sum(1) + 2.0 ** -8 * want.abs() + 1e-4
    assert bool(((logits.double() - want).abs() <= bound).all())
    tokens, logprobs = head.generate(x, 4, temperature=0.9, top_k=40, top_p=0.9)
    again, _ = head.generate(x, 4, temperature=0.9, top_k=40, top_p=0.9)
    assert torch.equal(tokens, again) and bool((tokens >= 0).all()) and bool((tokens < 5000).all())
    assert bool((logprobs <= 0).all()) and bool(torch.isfinite(logprobs).all())


def test_training_path(env, example):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(256, 300, generator=g, device="cuda")
    gain, bias = 1 + 0.3 * torch.randn(300, generator=g, device="cuda"), torch.randn(300, generator=g, device="cuda")
    target = loom.loom_layer_norm(x, gain, bias)[0]
    got_gain, got_bias, losses = example.fit_norm(x, target)
    assert losses[-1] < 1e-6 * losses[0]
    assert float((got_gain - gain).abs().max()) < 1e-2 and float((got_bias - bias).abs().max()) < 1e-2


@pytest.mark.parametrize("tokens", [20, 100, 300])
@pytest.mark.parametrize("k", [2048, 2052])
def test_waits_that_run_out(env, tokens, k):
    # a limit of one nanosecond: whatever wait is not over at once runs out (on a given call there
    # may be none); the outputs that this touches are NaN and the call says so, all others and
    # the next call are right
    torch, loom = env
    w = torch.ones(500, k, dtype=torch.int8, device="cuda")
    x = torch.ones(tokens, k, dtype=torch.int8, device="cuda")
    sw, sx = torch.ones(500, device="cuda"), torch.ones(tokens, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, acc = loom.loom_i8_matmul_ex(w, sw, 500, k, x, sx, tokens, want_acc=True, error=err,
                                    tuning=loom.make_tuning(path=loom.LOOM_PATH_TENSOR, wait_ns=1))
    torch.cuda.synchronize()
    late = torch.isnan(y)
    assert int(err) == (loom.LOOM_DEVERR_TIMEOUT if bool(late.any()) else int(err) & loom.LOOM_DEVERR_TIMEOUT)
    assert torch.equal(late, acc == -2 ** 31)
    assert bool((y[~late] == k).all())
    y, _ = loom.loom_i8_matmul(w, sw, 500, k, x, sx, tokens)
    assert bool((y == k).all())


def test_tensor_path_wants_aligned_matrices(env):
    torch, loom = env
    buf = torch.zeros(64 * 64 + 16, dtype=torch.int8, device="cuda")
    one = torch.ones(64, device="cuda")
    for w, x in ((buf[4:4 + 64 * 64], buf[:64 * 64]), (buf[:64 * 64], buf[8:8 + 64 * 64])):
        with pytest.raises(loom.LoomError) as e:
            loom.loom_i8_matmul_ex(w, one, 64, 64, x, one, 64, tuning=loom.make_tuning(path=loom.LOOM_PATH_TENSOR))
        assert e.value.status == loom.LOOM_ERR_ALIGN
    with pytest.raises(loom.LoomError) as e:       # tensors on the host
        loom.loom_quantize_tokens(torch.zeros(4, 64))
    assert e.value.status == loom.LOOM_ERR_ARG


@pytest.mark.parametrize("t", [1, 2, 3, 4, 31, 33, 128, 129, 255, 257])
@pytest.mark.parametrize("n,k", [(1, 20), (2, 4), (3, 36), (4, 12), (5, 1044), (127, 132), (129, 124), (255, 2052), (258, 1020)])
def test_tensor_product_around_its_tiles(env, t, n, k):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(1000 * t + n)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones(max(t, n), device="cuda")
    _, acc = loom.loom_i8_matmul_ex(w, one, n, k, x, one, t, want_acc=True, tuning=loom.make_tuning(path=loom.LOOM_PATH_TENSOR))
    assert torch.equal(acc.long(), (x.double() @ w.double().t()).long())


def test_in_a_graph(env):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(12, 1024, generator=g, device="cuda")
    w = torch.randint(-128, 128, (3000, 1024), generator=g, device="cuda", dtype=torch.int8)
    sw, u = torch.rand(3000, generator=g, device="cuda") * 0.01, torch.rand(12, generator=g, device="cuda")

    def step():
        q, s = loom.loom_layer_norm_i8(x)
        y, _ = loom.loom_i8_matmul(w, sw, 3000, 1024, q, s, 12)
        return y, loom.loom_sample_tokens(y, u, top_k=20)[0]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.mul_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_offsets_past_31_bits(env):
    # rows whose elements lie past 2^31 of their buffer: a stride of 2^29 f32 over 9 rows would take
    # 16 GiB, so the rows are few and the stride large
    torch, loom = env
    width, stride = 1024, (1 << 30) + 8
    buf = torch.empty(2 * stride + width, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, width), (stride, 1))
    x.copy_(torch.randn(3, width, device="cuda"))
    dense = x.contiguous()
    y, mean, rstd = loom.loom_layer_norm(x)
    want = loom.loom_layer_norm(dense)
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd), want))
    assert torch.equal(loom.loom_layer_norm_backward(dense, x, mean, rstd)[0], loom.loom_layer_norm_backward(dense, dense, mean, rstd)[0])
    assert all(torch.equal(a, b) for a, b in zip(loom.loom_quantize_tokens(x), loom.loom_quantize_tokens(dense)))
    u = torch.full((3,), 0.4, device="cuda")
    assert torch.equal(loom.loom_sample_tokens(x, u)[0], loom.loom_sample_tokens(dense, u)[0])
