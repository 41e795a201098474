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
