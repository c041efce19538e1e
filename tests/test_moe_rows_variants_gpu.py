"""The kernels that combine and its gradient have for whole words: one, two or four
of a token's rows on their way at once.  Which one a size gets goes by the CTAs of
its launch, so every size here says which it is for, and the rule is asked.
References and tolerances are test_moe_rows_gpu.py's.
"""
import pytest
import torch

import test_moe_rows_gpu as rows

pytestmark = pytest.mark.gpu

THREADS = 256


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()


def at_once(T, k, cols, gradient, sms):
    """Rows on their way where all start on 16 bytes: four, where there are more than two and all CTAs run at once."""
    steps = 4 if gradient else 2
    lanes = 32
    while lanes < min(-(-cols // (8 * steps)), THREADS):
        lanes *= 2
    ctas = -(-T // (THREADS // lanes)) * (1 if gradient else -(-cols // (lanes * 8 * steps)))
    return 1 if k == 1 else 2 if k == 2 or ctas > 2 * sms else 4


WHOLE = [("bf16", "bf16", 0), ("f16", "f32", 8), ("f32", "bf16", 0), ("bf16", "f16", 16), ("f32", "f32", 0)]
# tokens, experts, k, columns, rows on their way
CASES = [(900, 12, 5, 4096, 2), (3000, 16, 3, 264, 2), (1300, 20, 4, 2048, 2), (700, 64, 8, 8200, 2), (2600, 9, 7, 64, 2), (700, 8, 2, 4096, 2),
         (100, 16, 5, 1032, 4), (9, 4, 7, 4096, 4), (1, 3, 3, 24, 4), (40, 8, 6, 512, 4), (12, 8, 8, 4096, 4), (77, 5, 33, 80, 4),
         (1200, 6, 1, 520, 1), (3, 2, 1, 4096, 1)]


@pytest.mark.parametrize("x,y,pad", WHOLE)
@pytest.mark.parametrize("T,E,k,cols,want", CASES)
def test_rows_on_their_way(T, E, k, cols, want, x, y, pad):
    assert all((cols + pad) * (4 if t == "f32" else 2) % 16 == 0 for t in (x, y))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert at_once(T, k, cols, False, sms) == at_once(T, k, cols, True, sms) == want
    rows.test_combine(T, E, k, cols, x, y, pad, 0)
    rows.test_combine_backward(T, E, k, cols, x, y, pad, 0)
    rows.test_dispatch(T, E, k, cols, x, y, pad, 0)
