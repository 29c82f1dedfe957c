"""Tree attention in the order of its stream and beside itself, on both kernels of the history and at every number of copies of the
query rows (32, 64 and more of them a kv head)."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import tree_case as tc
from tests.test_gpu_tree_bound import LONG, bounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [2000, LONG])
@pytest.mark.parametrize("nodes", [3, 8, 16, 24])
def test_rows_that_the_kernels_before_wrote_are_read(nodes, most):
    """The nodes' and the recent rows, the lengths and the page tables change in place right before each call, by copies, fills and
    oscar_append_kv."""
    c = tc.TreeCache([1500, 600], [nodes, nodes], n_kv=2, page=16, seed=nodes).upload()
    want = bounded(c, most, 3)
    c.check(*want)
    keep = {n: getattr(c, n).clone() for n in ("dT", "dh", "db", "d4", "dbegin", "dmask")}
    k, v = c.bfp.k.clone(), c.bfp.v.clone()
    x = torch.randn((c.n, 2, 128), device="cuda").to(torch.bfloat16)
    i32 = lambda a: torch.tensor(np.concatenate(a), dtype=torch.int32, device="cuda")  # noqa: E731
    req, pos = i32([[b] * nodes for b in range(2)]), i32([c.seq[b] + np.arange(nodes) for b in range(2)])
    for _ in range(20):
        ob.oscar_append_kv(c.L, None, x, x, c.bfp, c.db, req, pos)           # other rows of the nodes
        other = bounded(c, most, 3)
        c.bfp.k.zero_()
        c.bfp.v.fill_(3.0)
        for n in keep:
            getattr(c, n).zero_()
        c.bfp.k.copy_(k)
        c.bfp.v.copy_(v)
        for n, t in keep.items():
            getattr(c, n).copy_(t)
        got = bounded(c, most, 3)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(other[0], want[0])
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("nodes", [(8, 24), (24, 24), (3, 16)])
def test_two_calls_of_the_same_kernel_at_once(nodes):
    """On two streams, with outputs and partials of their own made before and kept until both are done."""
    cases = [tc.TreeCache([3000, 700], [n, n], n_kv=2, seed=40 + i).upload() for i, n in enumerate(nodes)]
    want = [bounded(c, LONG, 4) for c in cases]
    sets = [[(torch.empty_like(w[0]), torch.empty_like(w[1]), ob.Partials.empty(c.L, c.n, 4)) for _ in range(10)] for c, w in zip(cases, want)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(10):
        for c, s, mine in zip(cases, streams, sets):
            o, l, part = mine[i]
            ob.oscar_tree_attention_int4_bounded(c.L, c.dq, c.dbegin, c.dmask, c.most, c.bfp, c.db, c.int4, c.d4, LONG, c.dT, c.dh, c.sm_scale, part, o, l, stream=s)
    torch.cuda.synchronize()
    for mine, w in zip(sets, want):
        assert all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for o, l, _ in mine)
