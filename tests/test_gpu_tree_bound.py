"""Which kernel takes the history goes by the bound that the call and the split count are given, not by the page tables' width."""
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import tree_case as tc

pytestmark = pytest.mark.gpu
LONG = 480000                                                    # a bound that every tree here takes to the kernel of long histories


def bounded(c, most, splits):
    out = torch.full((c.n, c.L.n_q_heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse, part = torch.full((c.n, c.L.n_q_heads), 7.0, device="cuda"), ob.Partials.empty(c.L, c.n, splits)
    ob.oscar_tree_attention_int4_bounded(c.L, c.dq, c.dbegin, c.dmask, c.most, c.bfp, c.db, c.int4, c.d4, most, c.dT, c.dh, c.sm_scale, part, out, lse)
    return out, lse


def widened(c, columns):
    more = torch.full((c.B, columns), -1, dtype=torch.int32, device="cuda")
    c.d4, c.db = (torch.cat([t, more], 1).contiguous() for t in (c.d4, c.db))


# 32, 64 and 96 query rows a kv head: 4, 2 and 1 copies of them on the kernel of long histories
@pytest.mark.parametrize("nodes", [8, 16, 24])
@pytest.mark.parametrize("splits", [1, 4])
def test_the_bound_chooses_the_kernel(nodes, splits):
    """Narrow tables and wide ones give the same bits under the same bound, and other bits under the other one."""
    c = tc.TreeCache([2000, 700], [nodes, nodes], n_kv=2, seed=nodes).upload()
    ref = c.attention()
    short, plain, long = bounded(c, 2000, splits), c.run(splits), bounded(c, LONG, splits)
    for got in (short, long):
        c.check(*got, ref)
    assert all(torch.equal(a, b) for a, b in zip(short, plain))
    assert not torch.equal(short[1], long[1])                    # (log-sum-exps of different kernels: their last bits differ)
    widened(c, 30000)
    wide = bounded(c, 2000, splits), c.run(splits), bounded(c, LONG, splits)
    for got, want in zip(wide, (short, long, long)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_histories_longer_than_the_bound_are_met_in_full():
    c = tc.TreeCache([3000], [24], n_kv=1, seed=3).upload()
    ref = c.attention()
    for most in (1, 100, LONG, 2 ** 31 - 1):
        c.check(*bounded(c, most, 3), ref)
    assert ob.oscar_get_device_status() == 0


def test_the_binding_checks_the_bound():
    c = tc.TreeCache([300], [4], n_kv=1, seed=4).upload()
    with pytest.raises(ob.OscarError):
        bounded(c, 0, 2)
    with pytest.raises(ob.OscarError):
        bounded(c, 2 ** 31, 2)
    with pytest.raises(TypeError):
        bounded(c, 1.5, 2)
