"""What the router's, the rows' and the loss's entry points refuse, on a machine
without a GPU: arguments are checked before the device is asked for."""
import pytest

import tiled_tensor_core_persistent_gb300 as tcg
from tiled_tensor_core_persistent_gb300 import _build

INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3
X, Y, Z, W, V, I, J = (0x100000 * i for i in range(1, 8))
BIG = 2 ** 31 - 4095     # one more than an extent may be


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where nothing can be launched")
    _build.build()


def code(f, *args, **kw):
    """The status of a call; 0 where it raised nothing."""
    try:
        f(*args, **kw)
    except tcg.TcgError as e:
        return e.code
    return 0


def ready(c):
    return c in (4, 6)      # everything but the device is in order


def vary(base, call):
    def f(**change):
        assert set(change) <= set(base)
        return call({**base, **change})
    return f


route = vary(dict(tokens=8, experts=16, k=2, logits=X, ld=16, dtype="f32", mask=None, topk=I, ld_topk=2, weights=W, ld_weights=2),
             lambda a: code(tcg.moe_route, a["tokens"], a["experts"], a["k"], a["logits"], a["ld"], a["dtype"], a["mask"], True, a["topk"],
                            a["ld_topk"], a["weights"], a["ld_weights"]))
route_back = vary(dict(tokens=8, experts=16, k=2, logits=X, ld=16, dtype="f32", topk=I, ld_topk=2, g=W, ld_g=2, d=Y, ldd=16, d_dtype="f32"),
                  lambda a: code(tcg.moe_route_backward, a["tokens"], a["experts"], a["k"], a["logits"], a["ld"], a["dtype"], a["topk"], a["ld_topk"],
                                 True, a["g"], a["ld_g"], False, a["d"], a["ldd"], a["d_dtype"]))


@pytest.mark.parametrize("f", [route, route_back])
def test_router(f):
    assert ready(f())
    assert f(tokens=0, logits=None, topk=None) == 0
    for bad in (dict(tokens=-1), dict(experts=0), dict(k=0), dict(k=17), dict(dtype="e4m3"), dict(logits=None), dict(ld=15), dict(topk=None),
                dict(ld_topk=1)):
        assert f(**bad) == INVALID, bad
    for big in (dict(experts=1025, ld=1025), dict(experts=64, ld=64, k=33, ld_topk=33), dict(tokens=BIG)):
        assert f(**big) == UNSUPPORTED, big
    for off in (dict(logits=X + 2), dict(topk=I + 1)):
        assert f(**off) == MISALIGNED, off
    assert ready(f(dtype="bf16", logits=X + 2))


def test_router_outputs():
    assert route(weights=None) == INVALID and route(ld_weights=1) == INVALID and route(weights=W + 2) == MISALIGNED
    assert route_back(g=None) == INVALID and route_back(ld_g=1) == INVALID and route_back(g=W + 1) == MISALIGNED
    assert route_back(d=None) == INVALID and route_back(ldd=15) == INVALID and route_back(d=Y + 2) == MISALIGNED
    assert route_back(d_dtype="e5m2") == INVALID


def test_sort():
    f = vary(dict(tokens=8, experts=16, k=2, topk=I, ld=2, offsets=J, row_token=X, row_of=Y, ld_row_of=2),
             lambda a: code(tcg.moe_sort, a["tokens"], a["experts"], a["k"], a["topk"], a["ld"], None, a["offsets"], a["row_token"], a["row_of"],
                            a["ld_row_of"], workspace=W, workspace_bytes=1 << 30))
    assert ready(f()) and ready(f(offsets=None)) and ready(f(tokens=0, topk=None, row_token=None, row_of=None))
    for bad in (dict(tokens=-1), dict(experts=0), dict(k=0), dict(topk=None), dict(ld=1), dict(row_token=None), dict(row_of=None), dict(ld_row_of=1)):
        assert f(**bad) == INVALID, bad
    for big in (dict(experts=1025), dict(tokens=2 ** 30, k=2), dict(tokens=2 ** 31 - 1), dict(tokens=65536, k=32768, ld=32768, ld_row_of=32768)):
        assert f(**big) == UNSUPPORTED, big
    for off in (dict(topk=I + 1), dict(offsets=J + 2), dict(row_token=X + 3), dict(row_of=Y + 1)):
        assert f(**off) == MISALIGNED, off
    assert tcg.moe_sort_workspace_size(-1, 4, 1) == 0 and tcg.moe_sort_workspace_size(4, 1025, 1) == 0
    small, large = tcg.moe_sort_workspace_size(8, 16, 2), tcg.moe_sort_workspace_size(100000, 256, 8)
    assert small == tcg.moe_balance_workspace_size() and large > small


dispatch = vary(dict(tokens=8, k=2, cols=64, rows=16, x=X, ldx=64, x_dtype="bf16", row_of=I, ld=2, out=Y, ldo=64, out_dtype="bf16"),
                lambda a: code(tcg.moe_dispatch, a["tokens"], a["k"], a["cols"], a["rows"], a["x"], a["ldx"], a["x_dtype"], a["row_of"], a["ld"],
                               a["out"], a["ldo"], a["out_dtype"]))
combine = vary(dict(tokens=8, k=2, cols=64, rows=16, x=X, ldx=64, x_dtype="bf16", row_of=I, ld=2, w=W, ldw=2, out=Y, ldo=64, out_dtype="bf16"),
               lambda a: code(tcg.moe_combine, a["tokens"], a["k"], a["cols"], a["rows"], a["x"], a["ldx"], a["x_dtype"], a["row_of"], a["ld"], a["w"],
                              a["ldw"], a["out"], a["ldo"], a["out_dtype"]))
combine_back = vary(dict(tokens=8, k=2, cols=64, rows=16, x=X, ldx=64, x_dtype="bf16", row_of=I, ld=2, w=W, ldw=2, dy=Z, lddy=64, dy_dtype="f32",
                         out=Y, ldo=64, dw=V, lddw=2),
                    lambda a: code(tcg.moe_combine_backward, a["tokens"], a["k"], a["cols"], a["rows"], a["x"], a["ldx"], a["x_dtype"], a["row_of"],
                                   a["ld"], a["w"], a["ldw"], a["dy"], a["lddy"], a["dy_dtype"], a["out"], a["ldo"], a["dw"], a["lddw"]))


@pytest.mark.parametrize("f", [dispatch, combine, combine_back])
def test_rows(f):
    assert ready(f()) and f(tokens=0, x=None, out=None, row_of=None) == 0
    for bad in (dict(tokens=-1), dict(k=0), dict(cols=-1), dict(rows=-1), dict(row_of=None), dict(ld=1), dict(x=None), dict(ldx=63), dict(out=None),
                dict(ldo=63), dict(x_dtype="e4m3")):
        assert f(**bad) == INVALID, bad
    for big in (dict(tokens=BIG), dict(rows=BIG), dict(cols=65535 * 4096 + 1, ldx=2 ** 30, ldo=2 ** 30)):
        assert f(**big) == UNSUPPORTED, big
    for off in (dict(x=X + 1), dict(out=Y + 1), dict(row_of=I + 2)):
        assert f(**off) == MISALIGNED, off
    assert ready(f(ldx=77, ldo=65, x=X + 2, out=Y + 2))


def test_rows_weights_and_gradients():
    for f in (combine, combine_back):
        assert ready(f(w=None, ldw=0)) and f(ldw=1) == INVALID and f(w=W + 2) == MISALIGNED
    assert combine(out_dtype="nvfp4") == INVALID and dispatch(out_dtype="nvfp4") == INVALID
    assert combine_back(dy=None) == INVALID and combine_back(lddy=1) == INVALID and combine_back(dy=Z + 2) == MISALIGNED
    assert combine_back(lddw=1) == INVALID and combine_back(dw=V + 1) == MISALIGNED
    assert ready(combine_back(dw=None, lddw=0, x=None))
    # no rows: x and the rows' gradient need not be there
    assert ready(combine(rows=0, x=None)) and ready(combine_back(rows=0, x=None, out=None)) and dispatch(rows=0, out=None) == 0
    assert dispatch(cols=0) == 0 and combine(cols=0) == 0 and ready(combine_back(cols=0))


xent = vary(dict(T=8, V=100, H=64, dtype="bf16", x=X, ldx=64, w=W, ldw=64, target=I, lse=Y, loss=Z, mean=V, valid=J),
            lambda a: code(tcg.linear_xent, a["T"], a["V"], a["H"], a["dtype"], a["x"], a["ldx"], a["w"], a["ldw"], a["target"], a["lse"], a["loss"],
                           a["mean"], a["valid"], workspace=0x10000000, workspace_bytes=1 << 40))
xent_back = vary(dict(T=8, V=100, H=64, dtype="bf16", x=X, ldx=64, w=W, ldw=64, target=I, lse=Y, valid=J, gm=V, gl=None, dx=Z, lddx=64, dx_dtype="bf16",
                      beta=0.0, dw=Z + 0x1000, lddw=64, dw_dtype="f32"),
                 lambda a: code(tcg.linear_xent_backward, a["T"], a["V"], a["H"], a["dtype"], a["x"], a["ldx"], a["w"], a["ldw"], a["target"], a["lse"],
                                a["valid"], a["gm"], a["gl"], a["dx"], a["lddx"], a["dx_dtype"], a["beta"], a["dw"], a["lddw"], a["dw_dtype"],
                                workspace=0x10000000, workspace_bytes=1 << 40))


@pytest.mark.parametrize("f", [xent, xent_back])
def test_cross_entropy(f):
    assert ready(f()) and ready(f(dtype="f16")) and ready(f(T=0, x=None, target=None, lse=None))
    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(dtype="f32"), dict(dtype="e4m3"), dict(x=None), dict(ldx=56), dict(w=None), dict(ldw=56),
                dict(target=None), dict(lse=None), dict(valid=None)):
        assert f(**bad) == INVALID, bad
    for big in (dict(T=2 ** 30), dict(V=2 ** 30), dict(H=2 ** 29, ldx=2 ** 30, ldw=2 ** 30), dict(T=2 ** 29, V=2 ** 20), dict(x=X + 8), dict(ldx=68),
                dict(w=W + 8), dict(ldw=68)):
        assert f(**{**({"lddx": 2 ** 30, "lddw": 2 ** 30} if f is xent_back and "H" in big else {}), **big}) == UNSUPPORTED, big
    for off in (dict(x=X + 1), dict(w=W + 1), dict(target=I + 2), dict(lse=Y + 2), dict(valid=J + 1)):
        assert f(**off) == MISALIGNED, off


def test_cross_entropy_outputs():
    assert ready(xent(loss=None)) and xent(mean=None) == INVALID and xent(loss=Z + 2) == MISALIGNED and xent(mean=V + 1) == MISALIGNED
    assert ready(xent_back(dx=None)) and ready(xent_back(dw=None, lddw=0)) and ready(xent_back(gm=None))
    assert xent_back(lddx=63) == INVALID and xent_back(lddw=63) == INVALID and xent_back(dx_dtype="e4m3") == INVALID
    assert xent_back(dw_dtype="mxfp4") == INVALID
    assert xent_back(dx=Z + 1) == MISALIGNED and xent_back(dw=Z + 2) == MISALIGNED and xent_back(gm=V + 2) == MISALIGNED
    assert xent_back(gl=V + 2) == MISALIGNED


def test_cross_entropy_workspace_is_bounded_by_a_piece_of_the_vocabulary():
    """It grows with the tokens, not with tokens times vocabulary: 1/16 of an
    fp32 logit and less is kept of each, and one piece of the gradient."""
    size = tcg.linear_xent_workspace_size
    assert size(-1, 5, 5) == size(5, 0, 5) == size(5, 5, 0) == 0
    for T, V, H in ((1, 1, 1), (1000, 50021, 1280), (8192, 131072, 4096), (65536, 131072, 4096)):
        forward, backward = size(T, V, H, False), size(T, V, H, True)
        assert forward <= backward
        assert forward <= T * V * 4 / 30 + 16 * T + T * 8 * 4 + (1 << 17)
        assert backward <= forward + (600 << 20) + T * H * 4 + min(V, (1 << 28) // (2 * T) + 512) * H * 4 + (1 << 30)
