"""What the loss's gradient takes of the workspace: dz of a piece of the
vocabulary in 16 bits, which is all of it where that fits 512 MB and at least 256
words otherwise; fp32 sums of dX where there are several pieces; partial sums of
split tiles; next to nothing else."""
import pytest

import tiled_tensor_core_persistent_gb300 as tcg
from tiled_tensor_core_persistent_gb300 import _build

REST = 1 << 16                     # status, counters, the balance loss's totals, alignment
PARTIAL = 16 * 128 * 32 * 4        # of a split tile's piece, at most one for each SM


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1024


def up(n, m):
    return -(-n // m) * m


@pytest.mark.parametrize("T,V,H,words", [(1, 1, 1, 1), (64, 32768, 4096, 32768), (1000, 50021, 1280, 50021), (4096, 65536, 4096, 65536),   # one piece
                                         (4097, 65536, 4096, 32768), (8192, 131072, 4096, 32768), (8192, 100000, 512, 25088),              # several
                                         (65536, 131072, 4096, 4096), (1 << 21, 50000, 64, 256)])
def test_gradients_workspace(T, V, H, words):
    size = tcg.linear_xent_workspace_size(T, V, H, True)
    dz = T * up(words, 32) * 2
    assert dz <= max(512 << 20, T * 256 * 2) + 64 * T
    sums = T * up(H, 32) * 4 if words < V else 0
    forward = tcg.linear_xent_workspace_size(T, V, H, False)
    assert forward <= up(V, 128) // 64 * T * 8 + 8 * T + REST
    want = max(dz + sums + sms() // 2 * 2 * PARTIAL, forward)
    assert want <= size <= want + REST
