"""The accepted path's rows where a request or a page is bad: whole pools compared, what moves and what stays."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests.test_gpu_tree_accept import BAD_BF16, BAD_LENGTH, Trees, walk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    torch.cuda.synchronize()


def every_second(t):
    """Trees whose path takes every second node: all rows but the first move."""
    for b in range(t.B):
        lo, n = int(t.begin[b]), int(t.nodes[b])
        t.parents[lo:lo + n] = np.maximum(np.arange(n) - 2, 0)
        t.draft[lo:lo + n] = np.arange(n)
        t.target[lo:lo + n] = np.minimum(np.arange(n) + 2, n - 1)
    return t


def expected(t, skipped=(), bad=()):
    """Pools after the call; bad: (request, page of its table) that holds no page."""
    ps, k, v = t.L.page_size, t.k.clone(), t.v.clone()
    for b in range(t.B):
        lo, hi, T = t.begin[b], t.begin[b + 1], t.seq[b]
        for i, w in enumerate([] if b in skipped else walk(t.target[lo:hi], t.draft[lo:hi], t.parents[lo:hi])):
            if (b, (T + w) // ps) in bad or (b, (T + i) // ps) in bad:
                continue
            s, d = (t.table[b, (T + w) // ps], (T + w) % ps), (t.table[b, (T + i) // ps], (T + i) % ps)
            k[:, d[0], d[1]], v[:, d[0], d[1]] = t.k[:, s[0], s[1]], t.v[:, s[0], s[1]]
    return k, v


def moved(t, k, v):
    assert torch.equal(t.k, k) and torch.equal(t.v, v)


@pytest.mark.parametrize("seq", [-1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 256, 10 ** 6])
def test_rows_of_a_skipped_request_stay_and_the_others_move(seq):
    t = every_second(Trees([12, 9, 40], [33, 70, 20], seed=7))
    before = t.k.clone()
    k, v = expected(t, skipped=[1])
    t.seq[1] = seq
    acc, path, tokens, length = t.run()
    assert ob.oscar_get_device_status() == BAD_LENGTH
    assert acc.tolist() == [6, 0, 20] and np.all(path[1] == -1) and np.all(tokens[1] == -1) and length[1] == seq
    moved(t, k, v)
    assert not torch.equal(t.k, before)


@pytest.mark.parametrize("begin", [[0, 12, 61, 61], [0, -1, 9, 40], [0, 12, 5, 61]])
def test_rows_of_bad_node_ranges_stay(begin):
    t = every_second(Trees([12, 9, 40], [33, 70, 20], seed=8))
    good = [b for b in range(3) if begin[b] == t.begin[b] and begin[b + 1] == t.begin[b + 1]]
    k, v = expected(t, skipped=[b for b in range(3) if b not in good])
    if begin == [0, -1, 9, 40]:                                  # the last request's range is one, of other nodes: a path of one
        t.target[9:40] = -7
    if begin == [0, 12, 5, 61]:                                  # 56 nodes are more than the 40 of the call
        assert begin[3] - begin[2] > t.most
    t.begin = np.array(begin)
    acc, *_ = t.run()
    assert ob.oscar_get_device_status() == BAD_LENGTH
    for b in good:
        assert acc[b] == (t.nodes[b] + 1) // 2
    moved(t, k, v)


@pytest.mark.parametrize("column", [2, 3, 4])
@pytest.mark.parametrize("page", [-1, 10 ** 6, 2 ** 31 - 1])
def test_rows_from_and_to_a_bad_page_stay_and_the_others_move(column, page):
    t = every_second(Trees([40, 30], [37, 5], seed=9, layers=2))
    k, v = expected(t, bad={(0, column)})
    t.table[0, column] = page
    acc, path, *_ = t.run()
    assert ob.oscar_get_device_status() == BAD_BF16
    assert acc.tolist() == [20, 15] and path[0, :20].tolist() == list(range(0, 40, 2))
    moved(t, k, v)


@pytest.mark.parametrize("order", [[0, 1, 2], [2, 1, 0], [1, 2, 0]])
def test_pools_in_any_order_of_their_addresses(order):
    t = every_second(Trees([12, 9], [33, 70], seed=10))
    k, v = expected(t)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = [i32([0, 0]), i32([[0] * 12] * 2), i32([[0] * 12] * 2)]
    ob.oscar_tree_accept(t.L, i32(t.target), i32(t.draft), i32(t.parents), i32(t.begin), t.most, i32(t.seq), *out,
                         pools=[ob.Bf16Pool(t.v[i], t.k[i]) if i == 1 else ob.Bf16Pool(t.k[i], t.v[i]) for i in order], page_table=i32(t.table))
    moved(t, k, v)
