"""What the binding refuses of the token operators' tensors before the library is called, on a
machine without a GPU: tensors of the host that are in order get as far as the refusal of the host
(LOOM_ERR_ARG), the others are refused for what is wrong with them."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def loom():
    import __graft_entry__
    __graft_entry__.build()
    import int8_dequant_dot_gb300 as m
    return m


def refused(loom, call, *args, **kw):
    with pytest.raises(loom.LoomError) as e:
        call(*args, **kw)
    return e.value.status


N, K, T = 24, 64, 5


def product(loom, ex=False, **change):
    a = {"w": torch.zeros(N, K, dtype=torch.int8), "sw": torch.ones(N), "n": N, "k": K, "x": torch.zeros(T, K // 4, dtype=torch.int32),
         "sx": torch.ones(T), "t": T}
    more = {key: change.pop(key) for key in list(change) if key not in a}
    a.update(change)
    return refused(loom, loom.loom_i8_matmul_ex if ex else loom.loom_i8_matmul, *a.values(), **more)


def test_product_in_order_reaches_the_device_check(loom):
    z = torch.zeros
    for good in ({}, {"w": z(N * K // 4, dtype=torch.int32)}, {"w": z(N + 3, K, dtype=torch.int8)}, {"sw": torch.ones(N + 9)}, {"bias": z(N)},
                 {"y": z(T, N)}, {"y": z(T + 2, N + 5)[1:T + 1, :N]}, {"y": z(T, N, dtype=torch.bfloat16)}, {"y": z(T + 1, N + 3)},
                 {"acc": z(T, N, dtype=torch.int32)}, {"want_acc": True}, {"x": z(0, dtype=torch.int8), "sx": z(0), "t": 0},
                 {"w": z(0, dtype=torch.int8), "sw": z(0), "n": 0}):
        assert product(loom, **good) == loom.LOOM_ERR_ARG
    assert product(loom, ex=True, error=z(1, dtype=torch.int32)) == loom.LOOM_ERR_ARG


@pytest.mark.parametrize("change", [
    {"w": torch.zeros(N - 1, K, dtype=torch.int8)}, {"w": torch.zeros(N, K)}, {"w": torch.zeros(N, 2 * K, dtype=torch.int8)[:, :K]},
    {"w": torch.zeros(K, N, dtype=torch.int8).t()}, {"x": torch.zeros(T, K // 4 - 1, dtype=torch.int32)},
    {"x": torch.zeros(2 * T, K, dtype=torch.int8)[::2]}, {"x": torch.zeros(T, K, dtype=torch.float16)},
    {"sw": torch.ones(N, dtype=torch.float64)}, {"sw": torch.ones(N - 1)}, {"sw": torch.ones(2 * N)[::2]},
    {"sx": torch.ones(T, dtype=torch.bfloat16)}, {"sx": torch.ones(T - 1)}, {"sx": torch.ones(1).expand(T)},
    {"bias": torch.zeros(N - 1)}, {"bias": torch.zeros(N, dtype=torch.float16)},
    {"y": torch.zeros(T - 1, N)}, {"y": torch.zeros(T, N - 1)}, {"y": torch.zeros(N, T).t()}, {"y": torch.zeros(T * N)},
    {"acc": torch.zeros(T, N - 1, dtype=torch.int32)}, {"acc": torch.zeros(T, N, dtype=torch.int64)},
    {"acc": torch.zeros(T, 2 * N, dtype=torch.int32)[:, :N]}, {"n": -1}, {"t": -1}])
def test_product_operands_that_do_not_fit(loom, change):
    assert product(loom, **change) == loom.LOOM_ERR_SHAPE


def test_product_error_word(loom):
    for error in (torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
        assert product(loom, ex=True, error=error) == loom.LOOM_ERR_SHAPE


R, W = 6, 32
Z = torch.zeros


@pytest.mark.parametrize("norm", [False, True])
def test_outputs_of_the_calls_to_bytes(loom, norm):
    call = loom.loom_layer_norm_i8 if norm else loom.loom_quantize_tokens
    x = Z(R, W)
    for good in ({}, {"q": Z(R, W // 4, dtype=torch.int32)}, {"q": Z(R * W, dtype=torch.int8)}, {"scale": Z(R + 2)},
                 {"error": Z(1, dtype=torch.int32)}, {"q": 0x10000, "scale": 0x10000, "error": 0x10000}):
        assert refused(loom, call, x, **good) == loom.LOOM_ERR_ARG
    for bad in ({"q": Z(R - 1, W // 4, dtype=torch.int32)}, {"q": Z(R, W)}, {"q": Z(R, 2 * W, dtype=torch.int8)[:, :W]}, {"scale": Z(R - 1)},
                {"scale": Z(R, dtype=torch.float64)}, {"scale": Z(2 * R)[::2]}, {"error": Z(1)}, {"error": Z(0, dtype=torch.int32)}):
        assert refused(loom, call, x, **bad) == loom.LOOM_ERR_SHAPE


def test_outputs_of_layer_norm(loom):
    x = Z(R, W)
    for good in ({}, {"mean": Z(R), "rstd": Z(R + 1)}, {"mean": 0x10000}, {"y": Z(R, W + 4)[:, :W]}):
        assert refused(loom, loom.loom_layer_norm, x, **good) == loom.LOOM_ERR_ARG
    for bad in ({"mean": Z(R - 1)}, {"rstd": Z(R, dtype=torch.float16)}, {"rstd": Z(2 * R)[::2]}, {"y": Z(R, W - 1)}, {"y": Z(W, R).t()},
                {"mean": Z(R - 1), "want_stats": False}):
        assert refused(loom, loom.loom_layer_norm, x, **bad) == loom.LOOM_ERR_SHAPE


def test_operands_of_layer_norm_backward(loom):
    def back(**change):
        a = {"dy": Z(R, W), "x": Z(R, W), "mean": Z(R), "rstd": Z(R)}
        a.update({key: change.pop(key) for key in list(change) if key in a})
        return refused(loom, loom.loom_layer_norm_backward, *a.values(), **change)
    for good in ({}, {"workspace": Z(9, dtype=torch.uint8)}, {"workspace": (0x10000, 16)}, {"workspace": None}, {"want_params": False}):
        assert back(**good) == loom.LOOM_ERR_ARG
    for bad in ({"dy": Z(R - 1, W)}, {"dy": Z(R, W, dtype=torch.float16)}, {"dy": Z(W, R).t()}, {"mean": Z(R + 1)}, {"rstd": Z(2 * R)[::2]},
                {"gain": Z(W - 1)}, {"dx": Z(R, W - 1)}, {"dgain": Z(W, dtype=torch.float64)}, {"dbias": Z(W + 1)},
                {"workspace": Z(8, 8)[:, :4]}):
        assert back(**bad) == loom.LOOM_ERR_SHAPE


def test_outputs_of_sampling(loom):
    l, u = Z(R, W), Z(R)
    i32 = torch.int32
    for good in ({}, {"token": Z(R, dtype=i32), "logprob": Z(R)}, {"token": 0x10000}, {"temperature": Z(R)}, {"want_logprob": False}):
        assert refused(loom, loom.loom_sample_tokens, l, u, **good) == loom.LOOM_ERR_ARG
    for bad in ({"token": Z(R - 1, dtype=i32)}, {"token": Z(R, dtype=torch.int64)}, {"token": Z(2 * R, dtype=i32)[::2]}, {"logprob": Z(R - 1)},
                {"logprob": Z(R, dtype=torch.float16)}, {"error": Z(1)}, {"temperature": Z(R - 1)}, {"top_k": Z(R, dtype=torch.int64)}):
        assert refused(loom, loom.loom_sample_tokens, l, u, **bad) == loom.LOOM_ERR_SHAPE
