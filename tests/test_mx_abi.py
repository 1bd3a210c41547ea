"""The 4-bit floating-point, routing and experts calls without a GPU: sizes,
and argument errors that come back before anything touches the device."""
import pytest
import torch

from oracle import mx_oracle as O

A = 1 << 20  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lq():
    import dequant_gemv_group_b200 as m
    return m


def test_packed_bytes(lq):
    for fmt in ("mxfp4", "nvfp4"):
        for n, k in [(1, 32), (33, 96), (128, 256), (129, 288), (28672, 8192)]:
            assert lq.lutq_mx_packed_bytes(n, k, fmt) == O.packed_bytes(n, k, fmt)
        for n, k in [(0, 32), (-1, 32), (8, 0), (8, 16), (8, 48), (1 << 30, 32), (8, 1 << 30)]:
            assert lq.lutq_mx_packed_bytes(n, k, fmt) == -1
    with pytest.raises(ValueError):
        lq.lutq_mx_packed_bytes(8, 32, "fp4")
    assert lq.lib.lutq_mx_packed_bytes(8, 32, 2) == -1


def test_quantize_arguments(lq):
    f = lq.lib.lutq_mx_quantize
    good = [A, 0, 1, 8, 64, 0, A, None, None]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_0=None) == 1 and call(_6=None) == 1 and call(_1=3) == 1 and call(_5=2) == 1
    assert call(_0=A + 8) == 4 and call(_6=A + 4) == 4
    assert call(_4=48) == 2 and call(_4=0) == 2 and call(_3=-1) == 2 and call(_2=65536) == 2
    assert call(_2=-1) == 2
    assert call(_2=0) == 0 and call(_3=0, _0=None, _6=None) == 0     # nothing to do


def test_dequantize_and_pack_arguments(lq):
    f = lq.lib.lutq_mx_dequantize
    assert f(None, 1, 8, 64, 0, A, 0, None) == 1 and f(A, 1, 8, 64, 0, None, 0, None) == 1
    assert f(A, 1, 8, 64, 0, A, 5, None) == 1 and f(A, 1, 8, 33, 0, A, 0, None) == 2
    assert f(A + 1, 1, 8, 64, 0, A, 0, None) == 4
    g = lq.lib.lutq_mx_pack
    assert g(None, A, None, 1, 8, 64, 1, A, None) == 1
    assert g(A, A, A + 4, 1, 8, 64, 1, A, None) == 4
    assert g(A, A, None, 1, 8, 40, 1, A, None) == 2


@pytest.mark.parametrize("name", ["lutq_mx_gemm", "lutq_mx_gemv"])
def test_product_arguments(lq, name):
    fn = getattr(lq.lib, name)

    def f(x=A, m=4, w=A, n=8, k=64, fmt=0, y=A, yt=2, xt=0):
        head = [x, m, w] if name == "lutq_mx_gemm" else [x, xt, m, w]
        return fn(*head, n, k, fmt, y, yt, None, None)

    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1 and f(yt=3) == 1 and f(fmt=-1) == 1
    assert f(x=A + 8) == 4 and f(w=A + 8) == 4 and f(y=A + 8) == 4
    assert f(m=-1) == 2 and f(n=0) == 2 and f(k=33) == 2 and f(m=1 << 30) == 2
    assert f(m=0, x=None, y=None) == 0
    if name == "lutq_mx_gemv":
        assert f(m=17) == 2 and f(xt=9) == 1


def test_route_arguments(lq):
    def f(z=A, dt=2, t=4, e=64, bias=None, score=0, groups=1, top_groups=1, best=1, k=4, ids=A,
          w=A):
        return lq.lib.lutq_route(z, dt, t, e, bias, score, groups, top_groups, best, k, 1, 1.0,
                                 ids, w, None, None)

    assert f(z=None) == 1 and f(ids=None) == 1 and f(w=None) == 1 and f(dt=3) == 1
    assert f(score=2) == 1
    for bad in (dict(t=-1), dict(e=0), dict(e=1025), dict(groups=0), dict(groups=3),
                dict(groups=64), dict(top_groups=0), dict(top_groups=2), dict(best=0),
                dict(best=3), dict(k=0), dict(k=33), dict(e=8, k=9),
                dict(groups=8, top_groups=1, k=9)):
        assert f(**bad) == 2, bad
    assert f(z=A + 2) == 4 and f(bias=A + 2) == 4 and f(ids=A + 1) == 4 and f(z=A + 1, dt=0) == 4
    assert f(t=0, z=None) == 0


def test_experts_arguments(lq):
    ws = lq.lutq_mx_experts_workspace_bytes
    assert ws(0, 2, 8, 64, 32, "mxfp4") == 0
    need = ws(5, 2, 8, 64, 32, "mxfp4")
    assert need > 0 and ws(6, 2, 8, 64, 32, "mxfp4") >= need

    def f(x=A, dt=0, t=5, ids=A, w=A, k=2, e=8, gate=A, up=A, down=A, d=64, ff=32, fmt=0, y=A,
          space=A, nb=need):
        return lq.lib.lutq_mx_experts(x, dt, t, ids, w, k, e, gate, up, down, d, ff, fmt, y, space,
                                      nb, None, None)

    for name in ("x", "ids", "w", "gate", "up", "down", "y"):
        assert f(**{name: None}) == 1, name
    for name in ("x", "gate", "up", "down", "y", "space"):
        assert f(**{name: A + 8}) == 4, name
    assert f(ids=A + 2) == 4 and f(w=A + 1) == 4
    assert f(dt=4) == 1 and f(fmt=2) == 1
    assert f(space=None) == 9 and f(nb=need - 1) == 9
    for bad in (dict(t=-1), dict(k=0), dict(k=65), dict(e=0), dict(e=1025), dict(d=48),
                dict(ff=16), dict(t=1 << 23, k=4), dict(d=(1 << 20) + 32), dict(ff=1 << 21)):
        assert f(**bad) == 2, bad
        if "t" not in bad or bad["t"] > 0:
            a = dict(t=5, k=2, e=8, d=64, ff=32) | bad
            assert ws(a["t"], a["k"], a["e"], a["d"], a["ff"], "mxfp4") == -1
    assert f(t=0, x=None, space=None) == 0


def test_binding_refuses_host_tensors(lq):
    x = torch.ones(4, 64)
    with pytest.raises(ValueError):
        lq.lutq_mx_quantize(x, "mxfp4")
    with pytest.raises(ValueError):
        lq.lutq_route(x, 2)
    with pytest.raises(ValueError):
        lq.lutq_mx_gemv(x, x, 4, 64, "mxfp4")
    with pytest.raises(ValueError):
        lq.lutq_mx_pack(x.to(torch.uint8), x.to(torch.uint8), "mxfp4")
