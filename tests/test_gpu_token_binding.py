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


def test_other_operands_on_the_host(env):
    torch, loom = env
    rows, width = 6, 64
    x, dy = torch.randn(rows, width, device="cuda"), torch.randn(rows, width, device="cuda")
    gain = torch.rand(width, device="cuda")
    y, mean, rstd = loom.loom_layer_norm(x, gain)
    host = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)   # noqa: E731
    word = host(1, dtype=torch.int32)
    cases = [(loom.loom_layer_norm, (x, gain.cpu()), {}), (loom.loom_layer_norm, (x,), {"bias": host(width)}),
             (loom.loom_layer_norm, (x,), {"y": host(rows, width)}), (loom.loom_layer_norm, (x,), {"mean": host(rows)}),
             (loom.loom_layer_norm_i8, (x, gain.cpu()), {}), (loom.loom_layer_norm_i8, (x,), {"error": word}),
             (loom.loom_quantize_tokens, (x,), {"q": host(rows, width // 4, dtype=torch.int32)}), (loom.loom_quantize_tokens, (x,), {"scale": host(rows)}),
             (loom.loom_quantize_tokens, (x,), {"error": word})]
    grad = (dy, x, mean, rstd)
    cases += [(loom.loom_layer_norm_backward, tuple(t.cpu() if j == i else t for j, t in enumerate(grad)), {}) for i in (0, 2, 3)]
    cases += [(loom.loom_layer_norm_backward, grad, {name: t}) for name, t in (("gain", gain.cpu()), ("dx", host(rows, width)), ("dgain", host(width)),
                                                                             ("workspace", host(1 << 16)))]
    u = torch.rand(rows, device="cuda")
    cases += [(loom.loom_sample_tokens, (x, u.cpu()), {})]
    cases += [(loom.loom_sample_tokens, (x, u), {name: t}) for name, t in (("temperature", host(rows)), ("top_k", host(rows, dtype=torch.int32)),
                                                                          ("token", host(rows, dtype=torch.int32)), ("logprob", host(rows)), ("error", word))]
    for call, args, more in cases:
        assert _refused(loom, call, *args, **more) == loom.LOOM_ERR_ARG, (call.__name__, list(more))
    # a device-readable pinned gain, and outputs given as tensors, work
    again, m2, r2 = torch.empty_like(x), torch.empty(rows + 1, device="cuda"), torch.empty(rows, device="cuda")
    loom.loom_layer_norm(x, gain.cpu().pin_memory(), y=again, mean=m2, rstd=r2)
    assert torch.equal(again, y) and torch.equal(m2[:rows], mean) and torch.equal(r2, rstd)
    q, scale = loom.loom_quantize_tokens(x)
    q2, s2 = torch.empty(rows, width, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    loom.loom_quantize_tokens(x, q=q2, scale=s2)
    assert torch.equal(q2, q.view(torch.int8)) and torch.equal(s2, scale)
    tok, lp = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    want = loom.loom_sample_tokens(x, u)
    loom.loom_sample_tokens(x, u, token=tok, logprob=lp)
    assert torch.equal(tok, want[0]) and torch.equal(lp, want[1])


def _busy(torch, nbytes, ms=100):
    """The current stream will write all of a block of `nbytes` that its allocator holds free, `ms` from now."""
    torch.cuda._sleep(int(ms * 2e6))
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    block.fill_(0xff)          # as f32, f16 or bf16: NaN
    del block


@pytest.mark.parametrize("as_handle", [False, True])
def test_outputs_of_a_call_on_another_stream_are_not_what_the_current_one_has_queued(env, as_handle):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, width, n = 512, 4096, 4096
    x = torch.randn(rows, width, generator=g, device="cuda")
    gain, u = torch.rand(width, generator=g, device="cuda"), torch.rand(rows, generator=g, device="cuda")
    w, sw = torch.randint(-128, 128, (n, width), generator=g, device="cuda", dtype=torch.int8), torch.rand(n, generator=g, device="cuda")
    q, scale = loom.loom_quantize_tokens(x)
    _, mean, rstd = loom.loom_layer_norm(x, gain)
    side = torch.cuda.Stream()
    s = side.cuda_stream if as_handle else side
    for call in (lambda **k: loom.loom_layer_norm(x, gain, **k), lambda **k: loom.loom_quantize_tokens(x, **k),
                 lambda **k: loom.loom_layer_norm_i8(x, gain, **k), lambda **k: loom.loom_i8_matmul(w, sw, n, width, q, scale, rows, want_acc=True, **k),
                 lambda **k: loom.loom_layer_norm_backward(x, x, mean, rstd, gain, **k), lambda **k: loom.loom_sample_tokens(x, u, **k)):
        want = call()
        sizes = sorted({t.numel() * t.element_size() for t in want})
        torch.cuda.synchronize()
        for nbytes in sizes:
            torch.cuda.empty_cache()
            _busy(torch, nbytes)
            got = call(stream=s)
            side.synchronize()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_workspace_of_a_call_on_another_stream(env):
    # the current stream writes blocks of the workspace's size while the other one takes gradients
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(4)
    rows, width = 2000, 4096
    x, gain = torch.randn(rows, width, generator=g, device="cuda"), torch.rand(width, generator=g, device="cuda")
    _, mean, rstd = loom.loom_layer_norm(x, gain)
    want = loom.loom_layer_norm_backward(x, x, mean, rstd, gain, want_dx=False)[1:]
    nbytes = loom.loom_layer_norm_backward_workspace_bytes(rows, width)
    side = torch.cuda.Stream()
    out = []
    for ms in (0.2, 0.4, 0.6, 0.8, 1.0, 1.3, 1.6, 2.0, 2.5, 3.0) * 2:      # the writes begin about when the call does
        dgain, dbias = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(int(ms * 2e6))
        for _ in range(200):
            torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(0xff)
        out.append(loom.loom_layer_norm_backward(x, x, mean, rstd, gain, want_dx=False, dgain=dgain, dbias=dbias, stream=side)[1:])
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got in out for a, b in zip(want, got))


def test_null_and_current_streams(env):
    torch, loom = env
    x = torch.randn(9, 128, device="cuda")
    want = loom.loom_layer_norm(x)
    torch.cuda.synchronize()
    for s in (0, torch.cuda.default_stream(), torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
        assert torch.equal(loom.loom_layer_norm(x, stream=s)[0], want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in (0, side, side.cuda_stream, None):
            y = loom.loom_layer_norm(x, stream=s)[0]
            torch.cuda.synchronize()
            assert torch.equal(y, want[0])
