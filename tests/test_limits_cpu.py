"""The largest sizes that the router's, the rows' and the loss's entry points take,
and the next ones, which they refuse; as in test_routing_rules_cpu.py without a GPU."""
import pytest

from test_routing_rules_cpu import UNSUPPORTED, _lib, combine, combine_back, dispatch, ready, route, route_back, xent, xent_back  # noqa: F401

EXTENT = 2 ** 31 - 4096


@pytest.mark.parametrize("f", [route, route_back, dispatch, combine, combine_back])
def test_tokens(f):
    assert ready(f(tokens=EXTENT)) and f(tokens=EXTENT + 1) == UNSUPPORTED


@pytest.mark.parametrize("f", [dispatch, combine, combine_back])
def test_rows_and_columns(f):
    most = 65535 * 2048 - 8
    wide = dict(ldx=2 ** 28, ldo=2 ** 28, **(dict(lddy=2 ** 28) if f is combine_back else {}))
    assert ready(f(rows=EXTENT)) and f(rows=EXTENT + 1) == UNSUPPORTED
    assert ready(f(cols=most, **wide)) and f(cols=most + 1, **wide) == UNSUPPORTED


@pytest.mark.parametrize("f", [xent, xent_back])
def test_loss(f):
    half, wide = EXTENT // 2, dict(ldx=2 ** 29, ldw=2 ** 29, **(dict(lddx=2 ** 29, lddw=2 ** 29) if f is xent_back else {}))
    for name in ("T", "V"):
        other = dict(V=2) if name == "T" else dict(T=1)
        assert ready(f(**{name: half}, **other)) and f(**{name: half + 1}, **other) == UNSUPPORTED
    assert ready(f(H=EXTENT // 4, **wide)) and f(H=EXTENT // 4 + 1, **wide) == UNSUPPORTED
    # blocks of 128 x 128 logits
    assert ready(f(T=128 * (2 ** 15 - 1), V=128 * 2 ** 15)) and f(T=128 * 2 ** 15, V=128 * 2 ** 15) == UNSUPPORTED
