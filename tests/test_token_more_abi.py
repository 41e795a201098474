"""4-bit products, routing and the adjustment of logits on a machine without a GPU: what the
library and the binding refuse.  No call here reaches the device."""
import pytest

A = 0x10000   # a 16-byte aligned fake device address (never dereferenced)
SMS = 152


@pytest.fixture(scope="module")
def loom():
    import __graft_entry__
    __graft_entry__.build()
    import int8_dequant_dot_gb300 as m
    return m


def test_matvec_refusals(loom):
    def m(w=A, sw=A, sdt=1, n=8, k=64, group=32, x=A, sx=A, t=4, bias=None, y=A, dt=0, stride=8):
        return loom.library().loom_i4_matvec(w, sw, sdt, n, k, group, x, sx, t, bias, y, dt, stride, None)
    assert m(t=0, w=None, x=None, y=None) == loom.LOOM_OK and m(n=0, w=None, y=None, stride=0) == loom.LOOM_OK
    for bad in ({"w": None}, {"sw": None}, {"x": None}, {"sx": None}, {"y": None}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"w": A + 2}, {"x": A + 1}, {"sw": A + 1}, {"sw": A + 2, "sdt": 0}, {"sx": A + 2}, {"bias": A + 1}, {"y": A + 2},
                {"y": A + 1, "dt": 2}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"k": 60}, {"k": -8}, {"k": 131072}, {"n": -1}, {"t": -1}, {"stride": 7}, {"group": 16}, {"group": 0}, {"group": 48},
                {"group": -32}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"sdt": 3}, {"sdt": -1}, {"dt": 3}, {"dt": -1}):
        assert m(**bad) == loom.LOOM_ERR_ARG


def test_matvec_routed_refusals(loom):
    def m(w=A, sw=A, sdt=1, e=4, n=8, k=64, group=32, x=A, sx=A, xr=3, ids=A, t=3, r=2, bias=None, y=A, dt=0, stride=8, err=None):
        return loom.library().loom_i4_matvec_routed(w, sw, sdt, e, n, k, group, x, sx, xr, ids, t, r, bias, y, dt, stride, err, None)
    assert m(t=0, xr=0, w=None, ids=None, y=None) == loom.LOOM_OK and m(r=0, xr=0, ids=None) == loom.LOOM_OK
    for bad in ({"w": None}, {"sw": None}, {"x": None}, {"sx": None}, {"y": None}, {"ids": None}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"ids": A + 2}, {"err": A + 1}, {"w": A + 2}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"e": -1}, {"e": 1025}, {"r": -1}, {"r": 65}, {"xr": 5}, {"xr": 0}, {"t": -1}, {"stride": 7}, {"k": 12}, {"t": 1 << 30, "xr": 1 << 30, "r": 4}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE


def test_route_refusals(loom):
    def m(l=A, dt=0, t=4, e=64, stride=64, bias=None, score=0, groups=1, top=1, best=1, k=8, renorm=1, factor=1.0, ids=A, w=A, counts=None):
        return loom.library().loom_route_tokens(l, dt, t, e, stride, bias, score, groups, top, best, k, renorm, factor, ids, w, counts, None)
    assert m(t=0, l=None, ids=None, w=None) == loom.LOOM_OK
    for bad in ({"l": None}, {"ids": None}, {"w": None}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"l": A + 2}, {"l": A + 1, "dt": 2}, {"bias": A + 2}, {"ids": A + 1}, {"w": A + 2}, {"counts": A + 2}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"t": -1}, {"t": 1 << 31}, {"e": 0}, {"e": 1025, "stride": 2000}, {"stride": 63}, {"k": 0}, {"k": 33}, {"k": 9, "e": 8}, {"groups": 0},
                {"groups": 5}, {"groups": 8, "top": 0}, {"groups": 8, "top": 9}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"dt": 3}, {"score": 2}, {"score": -1}, {"best": 0}, {"best": 3}, {"factor": float("nan")}, {"factor": float("inf")}):
        assert m(**bad) == loom.LOOM_ERR_ARG


def test_route_backward_refusals(loom):
    def m(dw=A, l=A, dt=0, t=4, e=64, stride=64, ids=A, score=0, k=8, renorm=1, factor=1.0, d=A, dstride=64, err=None):
        return loom.library().loom_route_tokens_backward(dw, l, dt, t, e, stride, ids, score, k, renorm, factor, d, dstride, err, None)
    assert m(t=0, dw=None, l=None, ids=None, d=None) == loom.LOOM_OK
    for bad in ({"dw": None}, {"l": None}, {"ids": None}, {"d": None}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"dw": A + 2}, {"l": A + 2}, {"ids": A + 1}, {"d": A + 2}, {"err": A + 2}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"t": -1}, {"e": 0}, {"e": 1025, "stride": 2000, "dstride": 2000}, {"stride": 63}, {"dstride": 63}, {"k": 0}, {"k": 33}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"dt": 3}, {"score": 2}, {"factor": float("nan")}):
        assert m(**bad) == loom.LOOM_ERR_ARG


def test_adjust_refusals(loom):
    def m(l=A, dt=0, rows=4, vocab=100, stride=100, hist=None, n=0, hs=0, lens=None, prompts=None, dr=None, r=1.0, df=None, f=0.0, dp=None, p=0.0,
          bi=None, bv=None, b=0, mask=None, masks=0, mr=None, y=A, ys=100, err=None):
        return loom.library().loom_adjust_logits(l, dt, rows, vocab, stride, hist, n, hs, lens, prompts, dr, r, df, f, dp, p, bi, bv, b, mask, masks, mr,
                                                 y, ys, err, None)
    assert m(rows=0, l=None, y=None) == loom.LOOM_OK
    for bad in ({"l": None}, {"y": None}, {"bi": A, "b": 3}, {"bv": A, "b": 3}):
        assert m(**bad) == loom.LOOM_ERR_NULL
    for bad in ({"l": A + 2}, {"y": A + 2}, {"hist": A + 2, "n": 5, "hs": 5}, {"lens": A + 1}, {"prompts": A + 2}, {"dr": A + 2}, {"df": A + 2}, {"dp": A + 2},
                {"bi": A + 2, "bv": A, "b": 3}, {"bi": A, "bv": A + 2, "b": 3}, {"mask": A + 2, "masks": 1}, {"mr": A + 2}, {"err": A + 2}):
        assert m(**bad) == loom.LOOM_ERR_ALIGN
    for bad in ({"rows": -1}, {"rows": 1 << 31}, {"vocab": 0}, {"vocab": 393217, "stride": 400000, "ys": 400000}, {"stride": 99}, {"ys": 99}, {"hist": A, "n": 5, "hs": 4},
                {"n": -1}, {"n": 1 << 20}, {"b": -1}, {"b": 1025}, {"masks": -1}, {"mask": A, "masks": 3}, {"mask": A, "masks": 0}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    for bad in ({"dt": 3}, {"r": 0.0}, {"r": -1.0}, {"r": float("nan")}, {"r": float("inf")}, {"f": float("nan")}, {"f": float("inf")}, {"p": float("-inf")}):
        assert m(**bad) == loom.LOOM_ERR_ARG


def test_launch_config(loom):
    cfg = loom.loom_token_launch_config
    for op, work in ((loom.LOOM_OP_I4_MATVEC, [1, 8192, 16384, 128, 0, 1, SMS]), (loom.LOOM_OP_I4_MATVEC, [300, 2048, 4096, 32, 64, 8, SMS]),
                     (loom.LOOM_OP_ROUTE_TOKENS, [16384, 256, SMS]), (loom.LOOM_OP_ROUTE_TOKENS_BACKWARD, [1, 1024, SMS]),
                     (loom.LOOM_OP_ADJUST_LOGITS, [256, 131072, 1, SMS]), (loom.LOOM_OP_ADJUST_LOGITS, [1, 393216, 0, SMS])):
        L = cfg(op, work)
        assert L["grid"][0] >= 1 and L["smem_bytes"] <= 227 * 1024 and 32 <= L["block"][0] <= 1024
    for op, work, status in ((loom.LOOM_OP_I4_MATVEC, [1, 8, 64], loom.LOOM_ERR_ARG), (loom.LOOM_OP_I4_MATVEC, [1, 8, 60, 32], loom.LOOM_ERR_SHAPE),
                             (loom.LOOM_OP_I4_MATVEC, [1, 8, 64, 33], loom.LOOM_ERR_SHAPE), (loom.LOOM_OP_ROUTE_TOKENS, [1, 1025, SMS], loom.LOOM_ERR_SHAPE),
                             (loom.LOOM_OP_ROUTE_TOKENS, [1], loom.LOOM_ERR_ARG), (loom.LOOM_OP_ADJUST_LOGITS, [1, 393217, 1, SMS], loom.LOOM_ERR_SHAPE)):
        with pytest.raises(loom.LoomError) as e:
            cfg(op, work)
        assert e.value.status == status


# ---- the binding: tensors of the host in order get as far as the refusal of the host (LOOM_ERR_ARG) ----
def refused(loom, call, *args, **kw):
    with pytest.raises(loom.LoomError) as e:
        call(*args, **kw)
    return e.value.status


def test_binding_matvec(loom):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    n, k, t, i32 = 24, 64, 5, torch.int32

    def m(**change):
        a = {"w": z(n, k // 8, dtype=i32), "sw": z(n, 2, dtype=torch.float16), "n": n, "k": k, "group": 32, "x": z(t, k, dtype=torch.int8), "sx": z(t), "t": t}
        more = {key: change.pop(key) for key in list(change) if key not in a}
        a.update(change)
        return refused(loom, loom.loom_i4_matvec, *a.values(), **more)
    for good in ({}, {"bias": z(n)}, {"y": z(t + 1, n + 1, dtype=torch.bfloat16)}, {"sw": z(2 * n)}, {"x": z(t, k // 4, dtype=i32)}):
        assert m(**good) == loom.LOOM_ERR_ARG
    for bad in ({"w": z(n, k // 8 - 1, dtype=i32)}, {"w": z(n, k // 8)}, {"sw": z(n, 1)}, {"sw": z(4 * n)[::2]}, {"x": z(t - 1, k, dtype=torch.int8)},
                {"sx": z(t - 1)}, {"bias": z(n - 1)}, {"y": z(t, n - 1)}, {"t": -1}, {"n": -1}):
        assert m(**bad) == loom.LOOM_ERR_SHAPE
    assert m(sw=z(n, 2, dtype=torch.float64)) == loom.LOOM_ERR_ARG

    def r(**change):
        a = {"w": z(3, n, k // 8, dtype=i32), "sw": z(3, n, 2), "e": 3, "n": n, "k": k, "group": 32, "x": z(t, k, dtype=torch.int8), "sx": z(t),
             "ids": z(t, 2, dtype=i32)}
        more = {key: change.pop(key) for key in list(change) if key not in a}
        a.update(change)
        return refused(loom, loom.loom_i4_matvec_routed, *a.values(), **more)
    assert r() == loom.LOOM_ERR_ARG and r(bias=z(3, n), error=z(1, dtype=i32)) == loom.LOOM_ERR_ARG
    for bad in ({"w": z(2, n, k // 8, dtype=i32)}, {"sw": z(3, n)}, {"ids": z(t, 2, dtype=torch.int64)}, {"ids": z(t, dtype=i32)}, {"x_rows": 2 * t}, {"bias": z(n)},
                {"y": z(t, n)}, {"error": z(1)}):
        assert r(**bad) == loom.LOOM_ERR_SHAPE


def test_binding_route(loom):
    torch = pytest.importorskip("torch")
    z, i32 = torch.zeros, torch.int32
    f = lambda l=z(4, 16), k=3, **kw: refused(loom, loom.loom_route_tokens, l, k, **kw)   # noqa: E731
    for good in ({}, {"bias": z(16)}, {"counts": z(16, dtype=i32)}, {"score": "sigmoid"}, {"score": loom.LOOM_SCORE_SIGMOID}, {"ids": z(4, 3, dtype=i32)}):
        assert f(**good) == loom.LOOM_ERR_ARG
    for bad in ({"bias": z(15)}, {"bias": z(16, dtype=torch.float64)}, {"counts": z(15, dtype=i32)}, {"ids": z(4, 2, dtype=i32)}, {"weights": z(4, 3, dtype=torch.float16)},
                {"l": z(16, 4).t()}):
        assert f(**bad) == loom.LOOM_ERR_SHAPE
    assert f(score="relu") == loom.LOOM_ERR_ARG and f(l=z(4, 16, dtype=torch.float64)) == loom.LOOM_ERR_ARG
    b = lambda dw=z(4, 3), l=z(4, 16), ids=z(4, 3, dtype=i32), **kw: refused(loom, loom.loom_route_tokens_backward, dw, l, ids, **kw)   # noqa: E731
    assert b() == loom.LOOM_ERR_ARG and b(dlogits=z(4, 20)[:, :16]) == loom.LOOM_ERR_ARG
    for bad in ({"dw": z(4, 2)}, {"dw": z(4, 3, dtype=torch.float16)}, {"ids": z(3, 3, dtype=i32)}, {"ids": z(4, 3)}, {"dlogits": z(4, 15)}, {"error": z(1)}):
        assert b(**bad) == loom.LOOM_ERR_SHAPE


def test_binding_adjust(loom):
    torch = pytest.importorskip("torch")
    z, i32 = torch.zeros, torch.int32
    f = lambda l=z(4, 100), **kw: refused(loom, loom.loom_adjust_logits, l, **kw)   # noqa: E731
    ok = {"history": z(4, 9, dtype=i32), "lengths": z(4, dtype=i32), "prompts": z(4, dtype=i32), "repetition": z(4), "bias_ids": z(4, 2, dtype=i32),
          "bias_values": z(4, 2), "mask": z(2, 4, dtype=i32), "mask_rows": z(4, dtype=i32)}
    assert f() == loom.LOOM_ERR_ARG and f(**ok) == loom.LOOM_ERR_ARG and f(history=z(4, 12, dtype=i32)[:, 1:]) == loom.LOOM_ERR_ARG
    for bad in ({"history": z(3, 9, dtype=i32)}, {"history": z(4, 9)}, {"lengths": z(3, dtype=i32)}, {"lengths": z(4)}, {"prompts": z(4, dtype=torch.int64)},
                {"repetition": z(3)}, {"frequency": z(4, dtype=torch.float64)}, {"bias_values": z(4, 3)}, {"bias_ids": z(3, 2, dtype=i32)},
                {"mask": z(2, 3, dtype=i32)}, {"mask": z(2, 4)}, {"mask": z(8, dtype=i32)}, {"mask_rows": z(3, dtype=i32)}, {"y": z(4, 99)}, {"error": z(1)}):
        assert f(**{**ok, **bad}) == loom.LOOM_ERR_SHAPE
    assert f(bias_ids=z(4, 2, dtype=i32)) == loom.LOOM_ERR_NULL and f(bias_values=z(4, 2)) == loom.LOOM_ERR_NULL


def test_launch_config_of_the_most_tokens(loom):
    for work in ([(1 << 31) - 1, 1, 8, 32, 0, 1, SMS], [(1 << 31) - 1, 8, 64, 32, 4, 1, SMS], [(1 << 24) + 1, 8192, 16384, 128, 0, 1, SMS]):
        L = loom.loom_token_launch_config(loom.LOOM_OP_I4_MATVEC, work)
        assert 1 <= L["grid"][0] <= 2 * SMS and L["smem_bytes"] <= 227 * 1024


def test_in_place_with_two_strides_is_refused(loom):
    lib = loom.library()
    def adjust(rows, stride, y_stride):
        return lib.loom_adjust_logits(A, 3, rows, 100, stride, None, 0, 0, None, None, None, 1.0, None, 0.0, None, 0.0, None, None, 0, None, 0, None, A,
                                      y_stride, None, None)
    def gradient(tokens, stride, dstride):
        return lib.loom_route_tokens_backward(A + 64, A, 3, tokens, 64, stride, A + 128, 0, 8, 1, 1.0, A, dstride, None, None)
    for call in (adjust, gradient):             # (an unknown type is what is refused otherwise)
        assert call(2, 200, 100) == call(2, 100, 200) == loom.LOOM_ERR_SHAPE
        assert call(2, 200, 200) == call(1, 200, 100) == loom.LOOM_ERR_ARG
