"""Attention of trees of drafted tokens over the 4-bit history, on the GPU, against 64-bit arithmetic."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import tree_case as tc

pytestmark = pytest.mark.gpu
D = 128
EXTRA = 0
BAD_BF16, BAD_LENGTH, BAD_INT4 = 0x2, 0x4, 0x10


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    torch.cuda.synchronize()


# Which kernel takes the history goes by the query rows and by what the page tables could hold: every test runs with tables as short
# as its lengths allow and with long ones, most of them empty.
@pytest.fixture(autouse=True, params=[0, 30000], ids=["short_tables", "long_tables"])
def tables(request):
    global EXTRA
    EXTRA = request.param


def make(*args, extra_pages=0, **kw):
    return tc.TreeCache(*args, extra_pages=extra_pages + EXTRA, **kw)


# layouts and trees on both sides of what one tile of query rows holds (16 rows, and 32, 64, 128 of them)
@pytest.mark.parametrize("n_kv,gqa,page,group,nodes", [
    (2, 4, 16, 128, 1), (2, 4, 16, 128, 4), (1, 1, 32, 128, 7), (3, 2, 64, 128, 9), (2, 4, 16, 128, 8), (2, 8, 64, 128, 5), (1, 4, 32, 128, 16),
    (1, 8, 64, 128, 33), (2, 2, 16, 128, 50), (1, 4, 64, 128, 100), (2, 4, 64, 64, 6), (1, 8, 16, 32, 9), (5, 1, 32, 32, 40)])
def test_trees_match_64_bits(n_kv, gqa, page, group, nodes):
    c = make([1024, 700, 333, 2500], [nodes, max(1, nodes // 2), 1, nodes], n_kv=n_kv, gqa=gqa, page=page, group=group, seed=nodes).upload()
    c.check(*c.run())
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("nodes", [2, 12])
@pytest.mark.parametrize("seq,hist", [
    ([0, 1, 5], None), ([63, 64, 65], None), ([320, 321, 319], None), ([352, 448, 449], None), ([500, 500, 500], [64, 500, 100]), ([16, 80, 96], [16, 80, 96])])
def test_lengths_at_the_regions_borders(seq, hist, nodes):
    c = make(seq, [nodes, 1, nodes], hist=hist, n_kv=1, seed=5).upload()
    c.check(*c.run())
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("sink,nodes", [(0, 3), (0, 20), (16, 20), (128, 20), (192, 3)])
def test_other_sinks(sink, nodes):
    c = make([900, 40], [nodes, nodes], n_kv=1, sink=sink, recent=100, page=16, seed=sink).upload()
    c.check(*c.run())


@pytest.mark.parametrize("nodes", [3, 40, 256])
def test_a_chain_is_a_causal_chunk(nodes):
    c = make([800, 0], [nodes, nodes], n_kv=1, gqa=2, chain=True, seed=nodes).upload()
    first = c.run()
    c.check(*first)
    c.dmask = torch.from_numpy(c.mask).cuda()                   # the same, spelled out
    assert all(torch.equal(a, b) for a, b in zip(first, c.run()))


def test_one_node_is_the_decode_call():
    """A single node is the newest token: the decode call with that token's row counted into its length."""
    c = make([1500, 400, 70], [1, 1, 1], seed=3).upload()
    out, _ = c.run()
    L = c.L
    part, o2 = ob.Partials.empty(L, 3, 4), torch.empty_like(out)
    ob.oscar_decode_attention_int4(L, c.dq, c.bfp, c.db, c.int4, c.d4, c.dT + 1, c.dh, c.sm_scale, part, out=o2)
    # two roundings of half a step, and what each call may be off by
    assert torch.all((out.double() - o2.double()).abs() <= 2.0 ** -7 * o2.double().abs() + 3 * c.output_error())


@pytest.mark.parametrize("nodes", [4, 30])
@pytest.mark.parametrize("splits", [1, 2, 7, 64])
def test_any_number_of_splits(nodes, splits):
    c = make([1300, 200, 64], [nodes, 2, nodes], n_kv=1, seed=splits).upload()
    c.check(*c.run(splits=splits))


@pytest.mark.parametrize("nodes", [3, 20])
def test_masks_of_any_bits(nodes):
    """Nodes that see nothing, not themselves, later nodes; with and without a cache; more mask words than nodes."""
    rng = np.random.default_rng(7)
    sees = [rng.random((nodes, nodes)) < 0.4 for _ in range(3)]
    sees[0][1] = sees[1][1] = False
    sees[0][0] = True
    c = make([0, 600, 90], [nodes] * 3, n_kv=1, sees=sees, words=5, seed=1).upload()
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -np.inf)


@pytest.mark.parametrize("nodes", [4, 24])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_is_not_seen_is_not_met(nodes, bad):
    """A node's key and value of infinities or NaN reach the nodes that see it, and no other."""
    c = make([400, 30], [nodes, nodes], n_kv=1, seed=2)
    want = c.attention()
    for b in range(2):
        at = c.seq[b] + 1
        c.bk[c.tb[b, at // 16], at % 16] = bad
        c.bv[c.tb[b, at // 16], at % 16] = bad
    c.upload()
    out, lse = c.run()
    hit = np.concatenate([s[:, 1] for s in c.sees])
    assert not torch.isfinite(out[torch.from_numpy(hit).cuda()]).any()
    keep = ~hit
    got, ref = out.double().cpu().numpy()[keep], want[0][keep]
    err = c.output_error()
    assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    assert torch.isfinite(lse[torch.from_numpy(keep).cuda()]).all()


@pytest.mark.parametrize("nodes", [4, 24])
def test_a_query_of_infinities_stays_its_own(nodes):
    c = make([900], [nodes], n_kv=1, seed=4)
    c.q[1, 2, 5] = np.inf
    c.q[2, 1, :] = np.nan
    c.upload()
    out, _ = c.run()
    c.q[1, 2, 5] = 0
    c.q[2, 1, :] = 0
    ref = c.attention()[0]
    got, err = out.double().cpu().numpy(), c.output_error()
    keep = np.ones(ref.shape[:2], bool)
    keep[1, 2] = keep[2, 1] = False
    assert np.all(np.abs(got - ref)[keep] <= (err + 2.0 ** -8 * (np.abs(ref) + err))[keep])
    assert np.isnan(got[2, 1]).all()


@pytest.mark.parametrize("nodes", [4, 24])
@pytest.mark.parametrize("scale_v,q_size", [(1e-12, 1.0), (1e12, 1.0), (1.0, 12.0), (1.0, 1e-6), (2.0 ** -60, 3.0)])
def test_sizes_of_values_and_queries(nodes, scale_v, q_size):
    c = make([1200], [nodes], n_kv=1, scale_v=scale_v, q_size=q_size, seed=6).upload()
    c.check(*c.run())


@pytest.mark.parametrize("nodes", [4, 24])
def test_a_huge_scale_without_weight(nodes):
    """A history row whose value scale is 2^40 above the others' and whose weight vanishes leaves the others' bits alone."""
    c = make([1000], [nodes], n_kv=1, seed=8)
    at = 200
    pg, sl = c.t4[0, at // 16], at % 16
    c.ck[pg, 0, sl] = 0
    c.sz[pg, 0, sl, 0] = [0.0, 0.0, 2.0 ** 40, 0.0]
    c.cv[pg, 0, sl] = 0                                          # its value is 0 all the same
    c.q = np.abs(c.q)
    for p in range(64, int(c.hist[0])):                          # the other rows' logits are some hundred above its 0
        c.sz[c.t4[0, p // 16], 0, p % 16, 0, :2] = [0.3, 4.0] if p != at else [0.0, 0.0]
    c.upload()
    out, lse = c.run()
    ref, want = c.attention()
    # its share of the bounds: weight 2^-60 or less times 2^40
    sane = c.sz[..., 2].copy()
    c.sz[pg, 0, sl, 0, 2] = 0.0
    err = c.output_error()
    assert np.nanmax(sane) == 2.0 ** 40
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))


def test_long_history_keeps_its_precision():
    c = make([20000], [12], n_kv=1, page=64, seed=9).upload()
    out, lse = c.run(splits=1)
    c.check(out, lse)
    ref = c.attention()[0]
    far = np.sqrt(((out.double().cpu().numpy() - ref) ** 2).mean() / (ref ** 2).mean())
    assert far <= 2.0 ** -8                                     # (rounding to bf16 alone: 2^-9.2)


def test_rows_behind_the_last_node_stay():
    c = make([300, 500], [3, 9], extra_rows=5, seed=10).upload()
    out, lse = c.run()
    c.check(out, lse)
    assert torch.all(out[12:] == 7) and torch.all(lse[12:] == 7)


def test_requests_without_nodes():
    c = make([300, 500, 40, 90], [0, 9, 0, 2], seed=11).upload()
    c.check(*c.run())
    assert ob.oscar_get_device_status() == 0


def test_bad_node_ranges_skip_their_request():
    c = make([300, 500, 200], [3, 9, 4], seed=12).upload()
    whole, _ = c.run()
    for begin in ([0, 3, 17, 16], [-1, 3, 12, 16], [0, 13, 12, 16], [0, 3, 12, 99]):
        c.dbegin = torch.tensor(begin, dtype=torch.int32, device="cuda")
        out, _ = c.run()
        assert ob.oscar_get_device_status() == BAD_LENGTH
        for b, (lo, hi) in enumerate(zip(begin, begin[1:])):
            if 0 <= lo <= hi <= 16 and hi - lo == c.nodes[b] and lo == c.begin[b]:
                assert torch.equal(out[lo:hi], whole[lo:hi])


def test_nodes_that_pass_the_page_table_skip_their_request():
    c = make([300, 310], [9, 9], page=16, seed=13).upload()             # 20 pages: 320 positions
    c.db, c.d4, c.max_pages = c.db[:, :20].contiguous(), c.d4[:, :20].contiguous(), 20
    c.dT = torch.tensor([300, 315], dtype=torch.int32, device="cuda")
    out, lse = c.run()
    assert ob.oscar_get_device_status() == BAD_LENGTH
    assert torch.all(out[9:] == 7) and torch.all(lse[9:] == 7) and not torch.any(out[:9] == 7)


@pytest.mark.parametrize("nodes", [2, 20])
def test_bad_pages_are_flagged_and_not_seen(nodes):
    c = make([600], [nodes], n_kv=1, page=32, seed=14).upload()
    c.d4[0, 5] = 10 ** 6
    out, lse = c.run()
    assert ob.oscar_get_device_status() == BAD_INT4
    keep = np.ones(600 + nodes, bool)
    keep[160:192] = False
    K, V = c.rows(0, 0, 0), c.rows(0, 0, 1)
    err = c.output_error()
    for i in range(nodes):
        on = keep & np.concatenate([np.ones(600, bool), c.sees[0][i]])
        z = c.q[i] @ K[on].T * c.sm_scale
        p = np.exp(z - z.max(1, keepdims=True))
        ref = p @ V[on] / p.sum(1, keepdims=True)
        assert np.all(np.abs(out[i].double().cpu().numpy() - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    c.upload()
    c.db[0, 0] = -5
    c.run()
    assert ob.oscar_get_device_status() == BAD_BF16


@pytest.mark.parametrize("nodes", [2, 20])
def test_results_do_not_depend_on_the_run(nodes):
    c = make([3000, 1100], [nodes, nodes], seed=15).upload()
    out, lse = c.run()
    for _ in range(5):
        o, l = c.run()
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("nodes", [2, 20])
def test_captured_and_replayed_on_new_lengths(nodes):
    """One graph, replayed after its inputs changed in place; the shapes' upper bounds stay."""
    big = make([1000, 900], [nodes, nodes], seed=16, extra_pages=2).upload()
    S = 5
    out, lse, part = torch.zeros((big.n, 8, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((big.n, 8), device="cuda"), ob.Partials.empty(big.L, big.n, S)
    big.run(S, out, lse, part)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        big.run(S, out, lse, part)
    g.replay()
    big.check(out, lse)
    big.q = np.roll(big.q, 1, axis=0)                            # other queries, and a request without nodes
    big.dq.copy_(torch.from_numpy(big.q).to(torch.bfloat16))
    g.replay()
    big.check(out, lse)
    big.dbegin.copy_(torch.tensor([0, 0, nodes], dtype=torch.int32))
    big.nodes, big.begin, big.sees[0] = np.array([0, nodes]), np.array([0, 0, nodes]), np.zeros((0, 0), bool)
    big.dmask[:nodes] = big.dmask[nodes:].clone()
    out.fill_(7.0)
    lse.fill_(7.0)
    g.replay()
    big.check(out, lse)


def test_streams_of_their_own():
    """Two calls at once on two streams, with partials and outputs of their own, made before and kept until both are done; a call on
    a stream that is not the current one."""
    a, b = (make([2000, 700], [n, n], seed=20 + n).upload() for n in (3, 20))
    wa, wb = a.run(), b.run()
    rounds = range(10)
    sets = [[(torch.empty_like(w[0]), torch.empty_like(w[1]), ob.Partials.empty(c.L, c.n, 3)) for _ in rounds] for c, w in ((a, wa), (b, wb))]
    wa, wb = a.run(3), b.run(3)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for i in rounds:
        a.run(3, *sets[0][i], stream=s1)
        b.run(3, *sets[1][i], stream=s2)
    torch.cuda.synchronize()
    for got, want in zip(sets, (wa, wb)):
        assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l, _ in got)


def test_what_the_call_before_wrote_is_read():
    """The order of the stream holds after a kernel, a copy and a fill of the call's inputs."""
    c = make([1500], [24], seed=30).upload()
    want, _ = c.run()
    q = c.dq.clone()
    for _ in range(5):
        c.dq.zero_()
        c.dq.copy_(q)
        out, _ = c.run()
        c.dq.fill_(3.0)
        assert torch.equal(out, want)
        c.dq.copy_(q)
