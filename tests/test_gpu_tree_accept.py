"""The accepted path of a tree and its rows moved, on the GPU; and a whole step of speculative decoding."""
import math

import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic
from tests import tree_case as tc

pytestmark = pytest.mark.gpu
D = 128
BAD_BF16, BAD_LENGTH = 0x2, 0x4


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def walk(target, draft, parents):
    way = [0] if len(target) else []
    while way:
        kids = [j for j in range(1, len(target)) if parents[j] == way[-1] and draft[j] == target[way[-1]] and j > way[-1]]
        if not kids:
            break
        way.append(kids[0])
    return way


class Trees:
    def __init__(self, nodes, seq, seed, n_kv=2, page=16, layers=3, hit=0.8, tokens=50):
        self.rng = rng = np.random.default_rng(seed)
        self.L, self.nodes, self.seq = ob.Layout(n_kv, 4, page), np.asarray(nodes), np.asarray(seq)
        self.B, self.most, self.begin = len(nodes), max(1, int(max(nodes))), np.concatenate([[0], np.cumsum(nodes)])
        n = int(self.begin[-1])
        self.parents = np.concatenate([tc.random_parents(c, rng, 5) for c in nodes if c] or [np.zeros(0, np.int32)])
        self.draft, self.target = rng.integers(0, tokens, n), rng.integers(0, tokens, n)
        for b in range(self.B):
            lo, hi = self.begin[b], self.begin[b + 1]
            for i in range(lo, hi):
                kids = np.flatnonzero(self.parents[lo:hi] == i - lo)
                kids = kids[kids > i - lo]
                if len(kids) and rng.random() < hit:
                    self.target[i] = self.draft[lo + rng.choice(kids)]
        self.max_pages = -(-int((self.seq + self.nodes).max()) // page) + 1
        self.table, n_pages = ic.tables(self.B, [[(int(t), int(t + c))] for t, c in zip(self.seq, self.nodes)], page, self.max_pages, rng)
        self.k, self.v = (torch.randn((layers, n_pages, page, n_kv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
        self.layers = layers

    def run(self, stride=None, new_len=True, pools=True, stream=None):
        stride = stride or self.most
        self.out = accepted, path, tokens, length = i32([-9] * self.B), torch.full((self.B, stride), -9, dtype=torch.int32, device="cuda"), \
            torch.full((self.B, stride), -9, dtype=torch.int32, device="cuda"), i32([-9] * self.B)
        ob.oscar_tree_accept(self.L, i32(self.target), i32(self.draft), i32(self.parents), i32(self.begin), self.most, i32(self.seq), accepted, path,
                             tokens, length if new_len else None, pools=[ob.Bf16Pool(k, v) for k, v in zip(self.k, self.v)] if pools else (),
                             page_table=i32(self.table) if pools else None, stream=stream)
        return [x.cpu().numpy() for x in self.out]

    def expect(self, stride=None, moved=True):
        ps, k, v = self.L.page_size, self.k.clone(), self.v.clone()
        acc, path, tokens = np.zeros(self.B, int), np.full((self.B, stride or self.most), -1), np.full((self.B, stride or self.most), -1)
        for b in range(self.B):
            lo, hi, T = self.begin[b], self.begin[b + 1], self.seq[b]
            way = walk(self.target[lo:hi], self.draft[lo:hi], self.parents[lo:hi])
            acc[b] = len(way)
            path[b, :len(way)], tokens[b, :len(way)] = way, self.target[lo:hi][way] if way else []
            for i, w in enumerate(way if moved else []):
                s, d = (self.table[b, (T + w) // ps], (T + w) % ps), (self.table[b, (T + i) // ps], (T + i) % ps)
                k[:, d[0], d[1]], v[:, d[0], d[1]] = self.k[:, s[0], s[1]], self.v[:, s[0], s[1]]
        return acc, path, tokens, self.seq + acc, k, v


@pytest.mark.parametrize("nodes,seq", [([1], [0]), ([2, 3], [15, 16]), ([7, 1, 30], [100, 0, 63]), ([256], [1000]), ([33, 64, 65, 200], [5, 300, 31, 77]),
                                       ([0, 5, 0], [9, 9, 9])])
@pytest.mark.parametrize("n_kv,page", [(1, 16), (8, 64), (5, 32)])
def test_paths_and_rows(nodes, seq, n_kv, page):
    t = Trees(nodes, seq, seed=len(nodes) + n_kv, n_kv=n_kv, page=page, hit=0.9)
    acc, path, tokens, length, k, v = t.expect()
    got = t.run()
    for g, w in zip(got, (acc, path, tokens, length)):
        assert np.array_equal(g, w)
    assert torch.equal(t.k, k) and torch.equal(t.v, v)
    assert ob.oscar_get_device_status() == 0


def test_a_chain_of_the_most_nodes_accepted_whole():
    t = Trees([256, 255], [40, 3], seed=1)
    for b in range(2):
        lo, hi = t.begin[b], t.begin[b + 1]
        t.parents[lo:hi] = np.arange(-1, hi - lo - 1)
        t.target[lo:hi - 1] = t.draft[lo + 1:hi]
    k, v = t.k.clone(), t.v.clone()
    acc, path, *_ = t.run(stride=300)
    assert acc.tolist() == [256, 255] and path[0, :256].tolist() == list(range(256)) and np.all(path[1, 255:] == -1)
    assert torch.equal(t.k, k) and torch.equal(t.v, v)           # nothing had to move


def test_every_second_node_moves_over_pages():
    """A path that takes every second row: rows are read that others are about to overwrite."""
    t = Trees([200], [13], seed=2, layers=2)
    t.parents[:] = np.maximum(np.arange(200) - 2, 0)
    t.parents[0] = -1
    t.draft[:] = np.arange(200)
    t.target[:] = np.minimum(np.arange(200) + 2, 199)
    want = t.expect()
    got = t.run()
    assert got[0][0] == want[0][0] == 100 and torch.equal(t.k, want[4]) and torch.equal(t.v, want[5])


def test_the_lowest_of_equal_children():
    t = Trees([6], [20], seed=3)
    t.parents[:] = [-1, 0, 0, 0, 2, 3]
    t.draft[:] = [0, 4, 7, 7, 1, 1]
    t.target[:] = [7, 0, 1, 1, 9, 9]
    acc, path, tokens, *_ = t.run()
    assert acc[0] == 3 and path[0, :3].tolist() == [0, 2, 4] and tokens[0, :3].tolist() == [7, 1, 9]


def test_parents_out_of_order_have_no_children():
    t = Trees([5], [20], seed=4)
    t.parents[:] = [3, 1, 7, -2, 4]                              # itself, later, outside
    t.draft[:] = t.target[:] = 5
    acc, path, *_ = t.run()
    assert acc[0] == 1 and path[0].tolist() == [0, -1, -1, -1, -1]


@pytest.mark.parametrize("layers", [64, 65, 130])
def test_many_layers(layers):
    t = Trees([12, 9], [33, 70], seed=5, n_kv=1, layers=layers, hit=1.0)
    want = t.expect()
    got = t.run()
    assert np.array_equal(got[1], want[1]) and torch.equal(t.k, want[4]) and torch.equal(t.v, want[5])


def test_without_pools_or_lengths():
    t = Trees([12, 9], [33, 70], seed=6)
    want = t.expect(moved=False)
    got = t.run(new_len=False, pools=False)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and np.all(got[3] == -9)
    assert torch.equal(t.k, want[4])


def test_bad_requests_are_skipped():
    t = Trees([12, 9, 4], [33, 70, 20], seed=7, hit=1.0)
    want = t.expect()
    t.seq[1] = -5
    k = t.k.clone()
    acc, path, tokens, length = t.run()
    assert ob.oscar_get_device_status() == BAD_LENGTH
    assert acc[1] == 0 and np.all(path[1] == -1) and length[1] == -5 and acc[0] == want[0][0] and acc[2] == want[0][2]
    t = Trees([12, 9], [33, 70], seed=7)
    t.seq[1] = t.max_pages * 16 - 8                              # the last node lies behind the page table
    acc, *_ = t.run()
    assert acc[1] == 0 and ob.oscar_get_device_status() == BAD_LENGTH
    del k


def test_bad_pages_are_not_moved():
    t = Trees([30], [40], seed=8, hit=1.0)
    want = t.expect()
    assert want[0][0] > 2
    t.table[0, 40 // 16] = 10 ** 6                               # (the path's first rows go there)
    t.run()
    assert ob.oscar_get_device_status() == BAD_BF16


def test_captured():
    t = Trees([20, 31], [100, 7], seed=9, hit=1.0)
    want = t.expect()
    a = dict(target=i32(t.target), draft=i32(t.draft), parents=i32(t.parents), begin=i32(t.begin), seq=i32(t.seq), table=i32(t.table))
    out = [i32([0, 0]), torch.zeros((2, 40), dtype=torch.int32, device="cuda"), torch.zeros((2, 40), dtype=torch.int32, device="cuda"), i32([0, 0])]
    pools = [ob.Bf16Pool(k, v) for k, v in zip(t.k, t.v)]
    call = lambda: ob.oscar_tree_accept(t.L, a["target"], a["draft"], a["parents"], a["begin"], t.most, a["seq"], *out, pools=pools, page_table=a["table"])  # noqa: E731
    k, v = t.k.clone(), t.v.clone()
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    t.k.copy_(k)
    t.v.copy_(v)
    g.replay()
    assert torch.equal(t.k, want[4]) and torch.equal(t.v, want[5]) and np.array_equal(out[0].cpu().numpy(), want[0])


def test_a_step_of_speculative_decoding():
    """Append the nodes, attend, sample, accept, and the next token's decode: equal to a cache in which the accepted tokens were
    appended one after another."""
    rng = np.random.default_rng(11)
    nodes, seq = [9, 5, 14], [700, 64, 380]
    c = tc.TreeCache(seq, nodes, n_kv=2, gqa=4, page=16, seed=11, extra_pages=1).upload()
    L, n, B = c.L, int(c.begin[-1]), 3
    rope = torch.from_numpy(np.concatenate([f(np.arange(900)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)) for f in (np.cos, np.sin)], 1).astype(np.float32)).cuda()
    x = torch.randn((n, 8 + 4, D), device="cuda").to(torch.bfloat16)
    req, node = np.repeat(np.arange(B), nodes), np.concatenate([np.arange(m) for m in nodes])
    depth = np.zeros(n, int)
    for i in range(n):
        if node[i]:
            depth[i] = depth[c.begin[req[i]] + c.parents[req[i]][node[i]]] + 1
    place = np.asarray(seq)[req] + node
    for b in range(B):                                           # the table's spare page of each request may be touched
        c.tb[b, (seq[b] + nodes[b] - 1) // 16] = c.tb[b, (seq[b] + nodes[b] - 1) // 16]
    q = torch.empty((n, 8, D), dtype=torch.bfloat16, device="cuda")
    ob.oscar_append_kv(L, x[:, :8], x[:, 8:10], x[:, 10:], c.bfp, c.db, i32(req), i32(place), q, rope=rope, rope_positions=i32(np.asarray(seq)[req] + depth))
    c.dq, c.q = q, q.double().cpu().numpy()
    c.bk, c.bv = c.bfp.k.double().cpu().numpy(), c.bfp.v.double().cpu().numpy()
    out, lse = c.run()
    c.check(out, lse)
    head = torch.randn((8 * D, 300), device="cuda") / math.sqrt(8 * D)
    scores = out.float().view(n, -1) @ head * 4
    tokens, u = torch.empty(n, dtype=torch.int32, device="cuda"), torch.rand(n, device="cuda")
    ob.oscar_sample(scores, torch.full((n,), 0.8, device="cuda"), u, tokens, top_k=i32([40] * n), top_p=torch.full((n,), 0.95, device="cuda"))
    parents, draft = np.concatenate(c.parents), rng.integers(0, 300, n)
    for i, t in enumerate(tokens.cpu().numpy()):                 # drafts that were right more often than not
        kids = np.flatnonzero((parents == node[i]) & (req == req[i]))
        if len(kids) and rng.random() < 0.8:
            draft[kids[-1]] = t
    accepted, path, got, length = i32([0] * B), i32([[0] * 14] * B), i32([[0] * 14] * B), i32([0] * B)
    before = c.bfp.k.clone(), c.bfp.v.clone()
    ob.oscar_tree_accept(L, tokens, i32(draft), i32(parents), c.dbegin, 14, c.dT, accepted, path, got, length, pools=[c.bfp], page_table=c.db)
    acc, way = accepted.cpu().numpy(), path.cpu().numpy()
    assert acc.max() > 1
    # the same tokens appended in order to the cache as it was
    k2, v2 = (a.clone() for a in before)
    rows = np.concatenate([c.begin[b] + way[b, :acc[b]] for b in range(B)])
    req2, pos2 = np.repeat(np.arange(B), acc), np.concatenate([seq[b] + np.arange(acc[b]) for b in range(B)])
    ob.oscar_append_kv(L, None, x[rows, 8:10].contiguous(), x[rows, 10:].contiguous(), ob.Bf16Pool(k2, v2), c.db, i32(req2), i32(pos2), rope=rope)
    for b in range(B):
        p = seq[b] + np.arange(acc[b])
        pg, sl = c.tb[b, p // 16], p % 16
        assert torch.equal(c.bfp.k[pg, sl], k2[pg, sl]) and torch.equal(c.bfp.v[pg, sl], v2[pg, sl])
    assert np.array_equal(length.cpu().numpy(), np.asarray(seq) + acc)
    o1, o2 = (torch.empty((B, 8, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for pool, o in ((c.bfp, o1), (ob.Bf16Pool(k2, v2), o2)):
        ob.oscar_decode_attention_int4(L, q[:B].contiguous(), pool, c.db, c.int4, c.d4, length, c.dh, c.sm_scale, ob.Partials.empty(L, B, 3), out=o)
    assert torch.equal(o1, o2) and ob.oscar_get_device_status() == 0
