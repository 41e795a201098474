"""The token operators (loom_token.h) on a machine without a GPU: refusals and launch
geometry.  No call here reaches the device."""
import ctypes

import pytest

A = 0x10000   # a 16-byte aligned fake device address (never dereferenced)
SMS = 152


@pytest.fixture(scope="module")
def loom():
    import __graft_entry__
    __graft_entry__.build()
    import int8_dequant_dot_gb300 as m
    return m


def test_quantize_refusals(loom):
    q = lambda x=A, dt=0, t=4, k=64, stride=64, out=A, sc=A, err=None: loom.library().loom_quantize_tokens(  # noqa: E731
        x, dt, t, k, stride, out, sc, err, None)
    assert q(t=0, x=None, out=None, sc=None) == loom.LOOM_OK
    for bad in ({"x": None}, {"out": None}, {"sc": None}):
        assert q(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"x": A + 2}, {"out": A + 2}, {"sc": A + 1}, {"err": A + 2}, {"x": A + 1, "dt": 1}):
        assert q(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"k": 62}, {"k": -4}, {"k": 131072, "stride": 131072}, {"t": -1}, {"stride": 63}, {"t": 1 << 31}):
        assert q(**bad) == loom.LOOM_ERR_SHAPE
    for dt in (-1, 3):
        assert q(dt=dt) == loom.LOOM_ERR_ARG


def test_matmul_refusals(loom):
    def m(w=A, sw=A, n=8, k=64, x=A, sx=A, t=4, bias=None, y=A, dt=0, stride=8, acc=None, err=None, tuning=None):
        tp = ctypes.byref(tuning) if tuning is not None else None
        return loom.library().loom_i8_matmul_ex(w, sw, n, k, x, sx, t, bias, y, dt, stride, acc, err, tp, None)
    assert m(t=0, w=None, x=None, y=None) == loom.LOOM_OK and m(n=0, w=None, y=None) == loom.LOOM_OK
    for bad in ({"w": None}, {"sw": None}, {"x": None}, {"sx": None}, {"y": None}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"w": A + 2}, {"x": A + 1}, {"sw": A + 2}, {"sx": A + 2}, {"bias": A + 1}, {"y": A + 2},
                {"y": A + 1, "dt": 2}, {"acc": A + 2}, {"err": A + 1}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"k": 66}, {"k": 131072}, {"k": -4}, {"n": -1}, {"t": -1}, {"stride": 7}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"dt": 3}, {"dt": -1}, {"tuning": loom.make_tuning(path=loom.LOOM_PATH_STAGED)},
                {"tuning": loom.make_tuning(path=4)}, {"tuning": loom.make_tuning(wait_ns=-1)}):
        assert m(**bad) == loom.LOOM_ERR_ARG


def test_layer_norm_refusals(loom):
    f = lambda x=A, dt=0, r=4, w=60, xs=60, g=None, b=None, eps=1e-5, y=A, ys=60, mean=None, rstd=None: \
        loom.library().loom_layer_norm(x, dt, r, w, xs, g, b, eps, y, ys, mean, rstd, None)   # noqa: E731
    assert f(r=0, x=None, y=None) == loom.LOOM_OK and f(w=0, x=None, y=None) == loom.LOOM_OK
    assert f(x=None) == loom.LOOM_ERR_NULL and f(y=None) == loom.LOOM_ERR_NULL
    for bad in ({"x": A + 2}, {"y": A + 1, "dt": 1}, {"g": A + 2}, {"b": A + 1}, {"mean": A + 2}, {"rstd": A + 3}):
        assert f(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"r": -1}, {"w": -1}, {"xs": 59}, {"ys": 0}, {"r": 1 << 31}):
        assert f(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"dt": 7}, {"eps": -1.0}, {"eps": float("nan")}):
        assert f(**bad) == loom.LOOM_ERR_ARG
    q = lambda w=64, xs=64, eps=1e-5, sc=A: loom.library().loom_layer_norm_i8(A, 2, 4, w, xs, A, A, eps, A, sc, None, None)  # noqa: E731
    assert q(w=62) == loom.LOOM_ERR_SHAPE and q(xs=60) == loom.LOOM_ERR_SHAPE
    assert q(eps=-1.0) == loom.LOOM_ERR_ARG and q(sc=None) == loom.LOOM_ERR_NULL


def test_layer_norm_backward_refusals(loom):
    f = lambda dy=A, x=A, dt=0, r=4, w=60, s=60, mean=A, rstd=A, dx=A, dxs=60, dg=None, db=None, ws=None, wsb=0: \
        loom.library().loom_layer_norm_backward(dy, s, x, s, dt, r, w, None, mean, rstd, dx, dxs, dg, db, ws, wsb, None)  # noqa: E731
    assert f(r=0) == loom.LOOM_OK and f(w=0, dg=A) == loom.LOOM_OK and f(dx=None) == loom.LOOM_OK
    for bad in ({"dy": None}, {"x": None}, {"mean": None}, {"rstd": None}):
        assert f(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"dy": A + 2}, {"x": A + 2}, {"dx": A + 2}, {"mean": A + 1}, {"dg": A + 2}, {"ws": A + 8, "dg": A}):
        assert f(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"r": -1}, {"w": -2}, {"s": 59}, {"dxs": 59}):
        assert f(**bad) == loom.LOOM_ERR_SHAPE
    assert f(dt=5) == loom.LOOM_ERR_ARG
    assert loom.library().loom_layer_norm_backward_workspace_bytes(4, 60, None) == loom.LOOM_ERR_NULL


def test_sample_refusals(loom):
    f = lambda l=A, dt=0, r=4, v=100, s=100, dT=None, T=1.0, tp=1.0, mp=0.0, u=A, tok=A, lp=None: \
        loom.library().loom_sample_tokens(l, dt, r, v, s, dT, T, None, 0, None, tp, None, mp, u, tok, lp, None, None)  # noqa: E731
    assert f(r=0, l=None, u=None, tok=None) == loom.LOOM_OK
    for bad in ({"l": None}, {"u": None}, {"tok": None}):
        assert f(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"l": A + 2}, {"u": A + 1}, {"tok": A + 2}, {"lp": A + 2}, {"dT": A + 2}, {"l": A + 1, "dt": 2}):
        assert f(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"r": -1}, {"v": 0}, {"v": 393217, "s": 393217}, {"s": 99}):
        assert f(**bad) == loom.LOOM_ERR_SHAPE
    nan = float("nan")
    for bad in ({"dt": 3}, {"T": -1.0}, {"T": nan}, {"tp": nan}, {"tp": -0.5}, {"mp": -1.0}, {"mp": nan}):
        assert f(**bad) == loom.LOOM_ERR_ARG
    assert f(T=nan, dT=A + 2) == loom.LOOM_ERR_ALIGN   # a host value is not read where a device one is given


def test_binding_refusals(loom):
    torch = pytest.importorskip("torch")
    with pytest.raises(loom.LoomError):
        loom.loom_quantize_tokens(torch.zeros(4, 8, dtype=torch.int32))
    with pytest.raises(loom.LoomError):
        loom.loom_layer_norm(torch.zeros(8, 4).t())             # rows that are not contiguous
    with pytest.raises(loom.LoomError):
        loom.loom_layer_norm(torch.zeros(4, 8), torch.ones(7))
    with pytest.raises(loom.LoomError):
        loom.loom_sample_tokens(torch.zeros(4, 8), torch.zeros(4), top_k=torch.zeros(4))   # not int32


def test_launch_geometry(loom):
    cfg = loom.loom_token_launch_config
    for rows, width in ((1, 1), (5, 512), (5, 513), (7, 16384), (7, 16385), (2, 32768), (2, 32769)):
        L = cfg(loom.LOOM_OP_LAYER_NORM, [rows, width, loom.LOOM_BF16, 1, SMS])
        assert L["grid"][0] == -(-rows // L["units_per_cta"]) and 32 <= L["block"][0] <= 1024
        assert L["kernel"] == (loom.LOOM_KERNEL_NORM_LONG if width > 32768 else loom.LOOM_KERNEL_NORM_ROWS)
        # the threads of a row hold all of it: 16 columns each, from 4097 columns on 32
        if width <= 512:
            assert L["block"][0] == 32 * L["units_per_cta"]
        elif width <= 32768:
            assert L["block"][0] * (16 if width <= 4096 else 32) >= width
    L = cfg(loom.LOOM_OP_LAYER_NORM, [10 ** 6, 8192, loom.LOOM_BF16, 1, SMS])
    assert L["grid"][0] == 2 * SMS and L["block"][0] == 256          # CTAs that walk over the rows
    for rows, width in ((1, 1), (100000, 64), (3, 8192), (3, 8193), (100000, 20000)):
        L = cfg(loom.LOOM_OP_LAYER_NORM_BACKWARD, [rows, width, loom.LOOM_F32, 1, SMS])
        assert 1 <= L["grid"][0] <= rows and L["block"][0] <= 1024
    for vocab, ranks in ((1, 1), (16384, 1), (16385, 2), (65536, 4), (65537, 8), (393216, 8)):
        L = cfg(loom.LOOM_OP_SAMPLE_TOKENS, [3, vocab, loom.LOOM_F32, SMS])
        assert L["cluster"][0] >= 1 and L["grid"][0] == 3 * L["cluster"][0] and L["smem_bytes"] <= 227 * 1024
    for bad in ([3, 0, 0], [3, 393217, 0], [-1, 5, 0]):
        with pytest.raises(loom.LoomError) as e:
            cfg(loom.LOOM_OP_SAMPLE_TOKENS, bad)
        assert e.value.status == loom.LOOM_ERR_SHAPE
    for op, bad in ((99, [1, 1, 1]), (loom.LOOM_OP_LAYER_NORM, [1, 1]), (loom.LOOM_OP_LAYER_NORM, [1, 1, 9]),
                    (loom.LOOM_OP_I8_MATMUL, [1, 1])):
        with pytest.raises(loom.LoomError) as e:
            cfg(op, bad)
        assert e.value.status == loom.LOOM_ERR_ARG
    for t, n, k in ((1, 8192, 16384), (8, 1, 4), (9, 5001, 4100), (4096, 16384, 8192), (1, 1 << 30, 16)):
        L = cfg(loom.LOOM_OP_I8_MATMUL, [t, n, k, 1, loom.LOOM_PATH_DIRECT, SMS])
        assert L["kernel"] == loom.LOOM_KERNEL_I8_MATMUL_DP4A
        assert L["units_per_cta"] <= 1024 and L["grid"][0] == -(-n // L["units_per_cta"])


@pytest.mark.parametrize("t,n,k,tensor", [(1, 65536, 16384, False), (4, 65536, 16384, False), (5, 8192, 16384, True), (8, 4096, 4096, False),
                                          (8, 32768, 2048, True), (16, 1024, 1024, False), (16, 4096, 4096, True), (24, 1024, 1024, False),
                                          (24, 2048, 4096, True), (25, 64, 64, True), (4096, 64, 64, True)])
def test_engine_by_tokens_and_weights(loom, t, n, k, tensor):
    want = loom.LOOM_KERNEL_I8_MATMUL_TENSOR if tensor else loom.LOOM_KERNEL_I8_MATMUL_DP4A
    assert loom.loom_token_launch_config(loom.LOOM_OP_I8_MATMUL, [t, n, k, 1, loom.LOOM_PATH_AUTO, SMS])["kernel"] == want
