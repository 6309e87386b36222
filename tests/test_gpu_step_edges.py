"""The calls around a drafted block at the edges of what they accept."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


@pytest.mark.parametrize("first", [0, 3])
def test_append_keeps_to_the_columns_of_its_table(first):
    # columns `first`.. of a wider table: a length past them is flagged and writes nothing, though the
    # wider table names pages there (and, in the last row, its storage may end there)
    ps, width = 4, 3
    k, v = (torch.zeros(1, 12, ps, 1, 8, device="cuda") for _ in range(2))
    cache = xp.Cache(k, v)
    wide = ints([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]])
    table = wide[:, first:first + width]
    new = torch.randn(2, 2, 1, 8, device="cuda")
    want_k, want_v = k.clone(), v.clone()
    xp.xp_cache_append(cache.handle, 0, new, new, table, ints([width * ps + 1, 5]))
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_ELENGTH
    last, row = int(table[0, width - 1]), table[1].tolist()
    for pool in (want_k, want_v):
        pool[0, last, ps - 1] = new[0, 0]              # the token that still fits
        pool[0, row[0], ps - 1] = new[1, 0]
        pool[0, row[1], 0] = new[1, 1]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
