"""What the block-scaled operators and the balance loss refuse, on a machine
without a GPU: combinations of arguments that would otherwise give a wrong
answer."""
import pytest

import tiled_tensor_core_persistent_gb300 as tcg
from tiled_tensor_core_persistent_gb300 import _build

from test_block128_cpu import INVALID, UNSUPPORTED, P, balance, code, cols, no_gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return tcg.lib()


def test_offsets_without_groups_are_refused():
    """Offsets of no groups at all would leave every row out: only padding would be written."""
    assert code(lambda: cols(offsets=P, num_groups=0)) == INVALID
    assert code(lambda: cols(num_groups=2)) == INVALID
    assert no_gpu(lambda: cols(offsets=P, num_groups=1))
    assert no_gpu(lambda: cols(num_groups=1))
    assert no_gpu(lambda: cols(num_groups=0))


def test_assignments_past_the_counts_range_are_refused():
    """Counts and offsets are 32-bit: more assignments than they hold would wrap."""
    assert code(lambda: balance(t=2 ** 30, k=2)) == UNSUPPORTED
    assert code(lambda: balance(t=3, k=2 ** 30, ldt=2 ** 30)) == UNSUPPORTED
    assert no_gpu(lambda: balance(t=2 ** 30 - 1, k=2))
    assert no_gpu(lambda: balance(t=2 ** 28 - 1, k=8, ldt=8))
