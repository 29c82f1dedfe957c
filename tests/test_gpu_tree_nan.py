"""NaN among what a node sees reaches its output, alone in what a warp, a split or a tile takes too; on both kernels of the history
(which go by the query rows and by the width of the page tables)."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import tree_case as tc

pytestmark = pytest.mark.gpu
KERNELS = pytest.mark.parametrize("nodes,extra", [(3, 0), (16, 30000), (24, 30000), (12, 30000), (8, 30000), (24, 0)])


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    torch.cuda.synchronize()


@KERNELS
@pytest.mark.parametrize("splits", [1, 4])
def test_a_key_of_nan_alone_in_its_tile_reaches_those_who_see_it(nodes, extra, splits):
    """Node 1 sees the cache and itself, and its key, NaN, is the one row of its 16 positions that it sees."""
    sees = [np.eye(nodes, dtype=bool)]
    c = tc.TreeCache([400], [nodes], n_kv=1, seed=31, sees=sees, extra_pages=extra)
    want = c.attention()
    at = 401
    c.bk[c.tb[0, at // 16], at % 16] = np.nan
    out, lse = c.upload().run(splits=splits)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    keep = np.arange(nodes) != 1
    got, ref, err = out.double().cpu().numpy()[keep], want[0][keep], c.output_error()
    assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))


@KERNELS
@pytest.mark.parametrize("splits", [1, 6, 30])
def test_history_rows_of_nan_reach_every_node(nodes, extra, splits):
    """A run of 128 positions whose keys are NaN, all that a split or a warp takes."""
    c = tc.TreeCache([1000], [nodes], n_kv=1, seed=32, extra_pages=extra)
    for p in range(256, 384):
        c.sz[c.t4[0, p // 16], 0, p % 16, :, 0] = np.nan
    out, lse = c.upload().run(splits=splits)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
