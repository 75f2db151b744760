"""Cuts of short sequences in wide tables, as a server has them whose tables are as wide as its longest sequence may
grow: bit for bit, at every width of the kernels."""
import pytest
import torch

import test_gpu_evict as evict

pytestmark = pytest.mark.gpu

from test_gpu_evict import built  # noqa: E402,F401


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("T", [1024, 2048, 4096, 8192, 16384, 16640, 51200, 65536])
@pytest.mark.parametrize("lens,new,fresh", [([513, 40, 0, 65], [512, 1, 0, 65], [1, 40, 0, 2]), ([700, 333, 1], [256, 332, 0], [700, 1, 1])])
def test_short_rows_in_wide_tables(lens, new, fresh, T, same):
    ps = 64
    W = max(1, max(-(-x // ps) for x in lens))
    evict.check(lens, new, fresh, NL=1, H=2, D=32, ps=ps, recent=7, sink=3, extra=T // ps - W, same=same, seed=T + len(lens), dtype=torch.float32)
