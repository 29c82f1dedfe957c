"""The 4-bit history on the GPU: append, demote and promote, decode attention, attention weights, eviction."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic
from tests.helpers import bf16_bits

pytestmark = pytest.mark.gpu
D = 128
BAD_BF16, BAD_LENGTH, BAD_INT4 = 0x2, 0x4, 0x10


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append --
def rope_table(n):
    a = np.arange(n)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def append_reference(x, w, eps, rope, rot, pairs):
    """float64 [n, heads, 128] and the size of what its rounding errors scale with."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    size = np.abs(x)
    if rope is None:
        return x, size
    y, j = x.copy(), np.arange(rot // 2)
    a, b = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
    c, s = rope[:, None, :rot // 2], rope[:, None, 64:64 + rot // 2]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size = size.copy()
    size[..., a] = size[..., b] = size[..., a] + size[..., b]
    return y, size


def check_rounded(got, ref, size):
    """bf16 output of an fp32 chain: at most 32 operations of 2^-24 (sum of squares 11, root 4, products and the rotation
    the rest) on terms of that size, then half a bf16 step."""
    err = 2.0 ** -19 * size
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)


@pytest.mark.parametrize("n_kv,gqa,page,rot,pairs", [(2, 4, 16, 128, False), (8, 4, 64, 128, True), (1, 8, 32, 64, False),
                                                      (5, 1, 16, 32, True), (3, 2, 64, 16, False), (8, 8, 64, 96, False)])
@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_append_matches_64_bits(n_kv, gqa, page, rot, pairs, tokens):
    rng = np.random.default_rng(tokens * 10 + n_kv)
    L = ob.Layout(n_kv, gqa, page)
    Hq, B, max_pages = n_kv * gqa, 3, 300 // page + 1
    table, n_pages = ic.tables(B, [[(0, 300)]] * B, page, max_pages, rng)
    slots = rng.permutation(B * 300)[:tokens]
    req, pos = slots // 300, slots % 300
    pos[rng.random(tokens) < 0.1] = -1                               # padding tokens anywhere in the batch
    qkv = torch.from_numpy(rng.normal(0, 3, (tokens, (Hq + 2 * n_kv) * D + 8)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = qkv[:, :-8].unflatten(1, (-1, D))
    wq, wk = (torch.from_numpy(rng.normal(1, 0.3, D).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    pool = ob.Bf16Pool(torch.full((n_pages, page, n_kv, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                       torch.full((n_pages, page, n_kv, D), 9.0, dtype=torch.bfloat16, device="cuda"))
    q_out = torch.full((tokens, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    rope, turn = rope_table(400), pos + 100
    ob.oscar_append_kv(L, x[:, :Hq], x[:, Hq:Hq + n_kv], x[:, Hq + n_kv:], pool, i32(table), i32(req), i32(pos), q_out, wq, wk,
                       1e-5, rope, rot, pairs, i32(turn))
    assert ob.oscar_get_device_status() == 0
    on = pos >= 0
    xs = x.double().cpu().numpy()
    angles = rope.double().cpu().numpy()[turn]
    qr, qs = append_reference(xs[:, :Hq], wq.double().cpu().numpy(), 1e-5, angles, rot, pairs)
    kr, ks = append_reference(xs[:, Hq:Hq + n_kv], wk.double().cpu().numpy(), 1e-5, angles, rot, pairs)
    got = q_out.double().cpu().numpy()
    check_rounded(got[on], qr[on], qs[on])
    assert np.all(got[~on] == 5)
    k, v = pool.k.double().cpu().numpy(), pool.v.double().cpu().numpy()
    pg, sl = table[req[on], pos[on] // page], pos[on] % page
    check_rounded(k[pg, sl], kr[on], ks[on])
    assert np.array_equal(v[pg, sl], xs[on][:, Hq + n_kv:])
    rest = np.ones(k.shape[:2], bool)
    rest[pg, sl] = False
    assert np.all(k[rest] == 7) and np.all(v[rest] == 9)


def test_append_without_norm_rotation_or_queries():
    L = ob.Layout(2, 4, 16)
    kv = torch.randn((5, 4, D), device="cuda").to(torch.bfloat16)
    pool = ob.Bf16Pool.empty(L, 4)
    ob.oscar_append_kv(L, None, kv[:, :2], kv[:, 2:], pool, i32([[2, 0, 3, 1]]), i32([0] * 5), i32([0, 17, 33, 50, 63]))
    at = [(2, 0), (0, 1), (3, 1), (1, 2), (1, 15)]
    for i, (p, s) in enumerate(at):
        assert torch.equal(pool.k[p, s], kv[i, :2]) and torch.equal(pool.v[p, s], kv[i, 2:])


def test_append_in_place_and_flags():
    L = ob.Layout(2, 4, 16)
    q = torch.randn((5, 8, D), device="cuda").to(torch.bfloat16)
    kv = torch.randn((5, 4, D), device="cuda").to(torch.bfloat16)
    rope, apart = rope_table(64), torch.empty_like(q)
    args = (kv[:, :2], kv[:, 2:])
    pools = [ob.Bf16Pool.empty(L, 4) for _ in range(2)]
    table, req, pos = i32([[2, 0, 3, 1]]), i32([0] * 5), i32([0, 17, 33, 50, 63])
    ob.oscar_append_kv(L, q, *args, pools[0], table, req, pos, apart, rope=rope)
    same = q.clone()
    ob.oscar_append_kv(L, same, *args, pools[1], table, req, pos, same, rope=rope)
    assert torch.equal(same, apart) and torch.equal(pools[0].k, pools[1].k)
    assert ob.oscar_get_device_status() == 0
    for bad in (dict(req=i32([0, 1, 0, 0, 0])), dict(req=i32([0, -1, 0, 0, 0])), dict(pos=i32([0, 64, 33, 50, 63])),
                dict(pos=i32([0, -2, 33, 50, 63])), dict(rope=rope_table(60), skipped=4)):
        out, skipped = torch.full_like(q, 5.0), bad.get("skipped", 1)
        ob.oscar_append_kv(L, q, *args, pools[1], table, bad.get("req", req), bad.get("pos", pos), out, rope=bad.get("rope", rope))
        assert ob.oscar_get_device_status() == BAD_LENGTH
        assert torch.all(out[skipped] == 5)
        keep = [i for i in range(5) if i != skipped]
        assert torch.equal(out[keep], apart[keep])
    pools[1].k.fill_(3.0)
    out = torch.empty_like(q)
    ob.oscar_append_kv(L, q, *args, pools[1], i32([[2, 4, 3, -1]]), req, pos, out, rope=rope)
    assert ob.oscar_get_device_status() == BAD_BF16
    assert torch.equal(out, apart) and torch.all(pools[1].k[:2] == 3)


# --------------------------------------------------------- demote, promote --
def history_rows(rng, shape):
    """Rows with what a quantizer can trip over: constant, all zero of both signs, one spike, ties, tiny and huge."""
    x = rng.normal(0, 2, shape)
    flat = x.reshape(-1, D)
    flat[0::37] = 1.5
    flat[1::37] = -0.0
    flat[1::37, ::3] = 0.0
    flat[2::37, 5] = 300.0
    flat[3::37] = np.arange(D) % 16 * 0.5 + 0.25 * (np.arange(D) % 2)    # on the borders between two codes
    flat[3::37, 0] = 0
    flat[3::37, 1] = 7.5
    flat[4::37] *= 1e-30
    flat[5::37] *= 1e30
    flat[6::37, 1:] = -6.5
    flat[6::37, 3] = 1e-9                                                # x - zero is not an fp32 number
    flat[6::37, 4] = 8.5
    return ic.bf16(flat.reshape(shape))


RANGES = [[(64, 64), (64, 65), (100, 101)], [(64, 300), (0, 17), (33, 33), (79, 145)], [(0, 320)]]


@pytest.mark.parametrize("n_kv,page,group", [(2, 16, 128), (8, 64, 128), (1, 32, 32), (5, 16, 64), (3, 64, 32)])
@pytest.mark.parametrize("ranges", RANGES)
@pytest.mark.parametrize("clip", [(1.0, 1.0), (0.96, 0.92)])
def test_demote_and_promote_bit_exact(n_kv, page, group, ranges, clip):
    rng = np.random.default_rng(n_kv + len(ranges))
    L = ob.Layout(n_kv, 1, page, group)
    B, max_pages = len(ranges), -(-320 // page)
    tb, nb = ic.tables(B, [[r] for r in ranges], page, max_pages, rng)
    t4, n4 = ic.tables(B, [[r] for r in ranges], page, max_pages, rng)
    rows = [history_rows(rng, (nb, page, n_kv, D)) for _ in range(2)]
    put = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()
    src = ob.Bf16Pool(put(rows[0]), put(rows[1]))
    dst = ob.Int4Pool.empty(L, n4)
    dst.codes_k.fill_(0xAA), dst.codes_v.fill_(0x55), dst.scale_zero.fill_(3.0)
    begin, end = i32([r[0] for r in ranges]), i32([r[1] for r in ranges])
    ob.oscar_demote_int4(L, src, i32(tb), dst, i32(t4), begin, end, *clip)
    back = ob.Bf16Pool(torch.full((nb, page, n_kv, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                       torch.full((nb, page, n_kv, D), 9.0, dtype=torch.bfloat16, device="cuda"))
    ob.oscar_promote_int4(L, dst, i32(t4), back, i32(tb), begin, end)
    assert ob.oscar_get_device_status() == 0
    want_codes = [np.full((n4, n_kv, page, D // 2), f, np.uint8) for f in (0xAA, 0x55)]
    want_sz = np.full((n4, n_kv, page, D // group, 4), 3.0)
    want_back = [np.full((nb, page, n_kv, D), f) for f in (7.0, 9.0)]
    for b, (lo, hi) in enumerate(ranges):
        p = np.arange(lo, hi)
        pb, p4, sl = tb[b, p // page], t4[b, p // page], p % page
        for kind in (0, 1):
            code, scale, zero = ic.quantize(rows[kind][pb, sl], group, clip[kind])     # [n, H, 128]
            c = code.astype(np.uint8)
            want_codes[kind][p4, :, sl] = c[..., 0::2] | (c[..., 1::2] << 4)
            want_sz[p4, :, sl, :, 2 * kind], want_sz[p4, :, sl, :, 2 * kind + 1] = scale, zero
            g = code.reshape(code.shape[:-1] + (D // group, group))
            want_back[kind][pb, sl] = ic.bf16_once((zero[..., None] + g * scale[..., None]).reshape(code.shape))
    assert np.array_equal(dst.codes_k.cpu().numpy(), want_codes[0])
    assert np.array_equal(dst.codes_v.cpu().numpy(), want_codes[1])
    assert np.array_equal(dst.scale_zero.double().cpu().numpy(), want_sz)
    assert np.array_equal(back.k.double().cpu().numpy(), want_back[0])
    assert np.array_equal(back.v.double().cpu().numpy(), want_back[1])


@pytest.mark.parametrize("n_kv,page,group", [(2, 16, 128), (8, 32, 64), (1, 64, 32)])
@pytest.mark.parametrize("ranges", [[(75, 309), (1, 319), (66, 303)], [(7, 318)]])
def test_demote_long_ranges_that_begin_and_end_anywhere(n_kv, page, group, ranges):
    test_demote_and_promote_bit_exact(n_kv, page, group, ranges, (1.0, 0.96))


def test_demote_and_promote_flag_bad_ranges_and_pages():
    L = ob.Layout(2, 1, 16)
    src, dst = ob.Bf16Pool.empty(L, 4), ob.Int4Pool.empty(L, 4)
    src.k.normal_(), src.v.normal_()
    table = i32([[0, 1], [2, 3]])
    for begin, end in (([0, -1], [16, 4]), ([0, 5], [16, 4]), ([0, 0], [16, 33])):
        dst.codes_k.zero_(), dst.scale_zero.zero_()
        ob.oscar_demote_int4(L, src, table, dst, table, i32(begin), i32(end))
        assert ob.oscar_get_device_status() == BAD_LENGTH
        assert dst.codes_k[0].any() and not dst.codes_k[1:].any()
        ob.oscar_promote_int4(L, dst, table, src, table, i32(begin), i32(end))
        assert ob.oscar_get_device_status() == BAD_LENGTH
    bad = i32([[0, 1], [4, -1]])
    dst.codes_k.zero_()
    ob.oscar_demote_int4(L, src, bad, dst, table, i32([0, 0]), i32([32, 32]))
    assert ob.oscar_get_device_status() == BAD_BF16
    assert dst.codes_k[:2].any() and not dst.codes_k[2:].any()
    ob.oscar_demote_int4(L, src, table, dst, bad, i32([0, 0]), i32([32, 32]))
    assert ob.oscar_get_device_status() == BAD_INT4
    ob.oscar_promote_int4(L, dst, bad, src, table, i32([0, 0]), i32([32, 32]))
    assert ob.oscar_get_device_status() == BAD_INT4


# ------------------------------------------------------------------ decode --
def decode(c, splits, fused=True, stream=None):
    part = ob.Partials.empty(c.L, c.B, splits)
    out = torch.full((c.B, c.L.n_q_heads, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out32 = torch.full(out.shape, float("nan"), device="cuda")
    lse = torch.full(out.shape[:2], float("nan"), device="cuda")
    counters = torch.zeros(c.B * c.L.n_kv_heads, dtype=torch.int32, device="cuda") if fused else None
    ob.oscar_decode_attention_int4(*c.attention_args(), part, out, out32, lse, counters, stream)
    torch.cuda.synchronize()
    assert counters is None or not counters.any()
    assert torch.equal(out, out32.to(torch.bfloat16))
    return out32, lse, part


def check_decode(c, splits, fused=True):
    out, lse, part = decode(c, splits, fused)
    ref, ref_lse = c.attention()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    some = c.seq > 0
    assert np.all(got[~some] == 0) and np.all(got_lse[~some] == -np.inf)
    e = c.logit_error()
    # a sum of exponentials of a few roundings each, its logarithm: 2^-20 beside the logits' own error
    assert np.abs(got_lse[some] - ref_lse[some]).max() <= e + 2.0 ** -20 * (1 + np.abs(ref_lse[some]).max())
    assert np.abs(got[some] - ref[some]).max() <= c.output_error()
    return out, lse, part


LENGTHS = [[1], [16, 63, 64], [65, 320, 321], [337, 352, 1], [1000, 400, 700, 337], [2500]]


@pytest.mark.parametrize("seq", LENGTHS)
@pytest.mark.parametrize("n_kv,gqa,page,group", [(2, 4, 16, 128), (8, 4, 64, 128), (1, 8, 32, 32), (5, 1, 16, 64), (2, 2, 64, 32),
                                                  (3, 8, 16, 128)])
def test_decode_matches_64_bits(seq, n_kv, gqa, page, group):
    c = ic.Cache(seq, n_kv=n_kv, gqa=gqa, page=page, group=group, seed=len(seq) + n_kv).upload()
    for splits in (1, 3, 17):
        out, lse, part = check_decode(c, splits)
        again = decode(c, splits)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        two = decode(c, splits, fused=False)
        assert torch.equal(out, two[0]) and torch.equal(lse, two[1])
        merged, mlse = torch.empty_like(out), torch.empty_like(lse)
        ob.oscar_merge(c.L, part, None, None, merged, mlse)
        assert torch.equal(out, merged) and torch.equal(lse, mlse)
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("page,sink", [(16, 64), (16, 16), (16, 48), (32, 32), (64, 64), (16, 0)])
@pytest.mark.parametrize("seq,hist", [([500], [500]), ([500, 500], [64, 65]), ([500, 500, 500], [479, 480, 481]), ([300, 97], [96, 97]),
                                      ([100, 0, 70], [100, 0, 70])])
def test_decode_history_ends(page, sink, seq, hist):
    """History ends on and around page and block borders, none at all, all of it; no recent rows; no sink."""
    c = ic.Cache(seq, hist, page=page, sink=sink, group=64, seed=page + sink).upload()
    check_decode(c, 4)
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("gqa,group", [(4, 128), (8, 32)])
@pytest.mark.parametrize("scale_k,scale_v,q_size", [(1, 1e-30, 1), (1, 1e28, 1), (1, 1, 40), (30, 300, 1), (1e-3, 1e-3, 1e3), (0, 0, 1)])
def test_decode_extreme_scales(gqa, group, scale_k, scale_v, q_size):
    """Value scales far from 1, one dominant logit, all logits alike, rows that are all zero."""
    c = ic.Cache([900, 350], gqa=gqa, group=group, scale_k=scale_k, scale_v=scale_v, q_size=q_size, seed=3).upload()
    check_decode(c, 2)


def test_decode_value_scales_that_grow_and_fall():
    """Along the history the value scale runs over 2^-60 .. 2^60: what a running scale must follow both ways."""
    for order in (1, -1):
        c = ic.Cache([1344], n_kv=1, page=16, seed=5)
        for p in range(64, int(c.hist[0])):
            e = (p - 64) / (c.hist[0] - 64) * 120 - 60
            pg = c.t4[0, p // 16]
            c.sz[pg, 0, p % 16, :, 2:] = ic.bf16(c.sz[pg, 0, p % 16, :, 2:] * 2.0 ** (order * e))
        check_decode(c.upload(), 1)


def test_decode_sink_logit_far_above_the_rest():
    """One history token with nearly all the weight and a long flat tail whose sum still counts."""
    c = ic.Cache([3000], n_kv=1, gqa=4, page=16, seed=9)
    pg = c.t4[0, 80 // 16]
    c.sz[pg, 0, 0, :, :2] *= 12
    c.sz = ic.bf16(c.sz)
    check_decode(c.upload(), 2)


def test_decode_many_splits_and_long_history():
    c = ic.Cache([30000, 9000], n_kv=2, page=64, seed=2, rubbish=False).upload()
    check_decode(c, 1024)
    check_decode(c, ob.oscar_suggest_splits_int4(c.L, 2, 30000, 152))


@pytest.mark.parametrize("splits", [15, 16, 31, 32, 33, 48, 65, 100, 1024])
@pytest.mark.parametrize("gqa", [1, 8])
def test_decode_merge_of_any_number_of_splits(splits, gqa):
    """The merge inside the launch has the separate merge's bits: full ones, part ones, empty ones, none."""
    c = ic.Cache([3300, 0, 500, 70], n_kv=2, gqa=gqa, page=16, seed=splits).upload()
    out, lse, _ = check_decode(c, splits)
    two = decode(c, splits, fused=False)
    assert torch.equal(out, two[0]) and torch.equal(lse, two[1])


def test_decode_bad_pages_and_lengths_are_flagged():
    c = ic.Cache([600, 600], seed=4).upload()
    good = decode(c, 3)[0]
    c.d4[1, 6] = -1
    out = decode(c, 3)[0]
    assert ob.oscar_get_device_status() == BAD_INT4
    assert torch.equal(out[0], good[0]) and torch.isfinite(out[1]).all() and not torch.equal(out[1], good[1])
    c.d4[1, 6] = c.int4.n_pages
    assert torch.equal(decode(c, 3)[0], out)
    assert ob.oscar_get_device_status() == BAD_INT4
    c.upload()
    c.db[1, 0] = c.bfp.n_pages
    out = decode(c, 3)[0]
    assert ob.oscar_get_device_status() == BAD_BF16
    assert torch.equal(out[0], good[0]) and torch.isfinite(out[1]).all()
    c.upload()
    c.dh[1] = 601
    decode(c, 3)
    assert ob.oscar_get_device_status() & BAD_LENGTH


def test_decode_far_offsets():
    """Pages beyond 2^32 bytes of codes."""
    n_pages, H, ps = (1 << 32) // (8 * 64 * 64) + 40, 8, 64
    c = ic.Cache([2000], n_kv=H, page=ps, seed=6)
    c.upload()
    ref = decode(c, 5)
    big = ob.Int4Pool(torch.empty((n_pages, H, ps, 64), dtype=torch.uint8, device="cuda"),
                      torch.empty((n_pages, H, ps, 64), dtype=torch.uint8, device="cuda"),
                      torch.empty((n_pages, H, ps, 1, 4), dtype=torch.bfloat16, device="cuda"))
    n = c.int4.n_pages
    for name in ("codes_k", "codes_v", "scale_zero"):
        getattr(big, name)[-n:] = getattr(c.int4, name)
    c.int4 = big
    c.d4 = torch.where(c.d4 >= 0, c.d4 + (n_pages - n), c.d4)
    got = decode(c, 5)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    mass = torch.zeros((1, H, c.max_pages * ps), device="cuda")
    ob.oscar_attention_mass_int4(*c.attention_args(), got[1], mass)
    assert abs(float(mass.sum()) - 32) < 1e-3


def test_decode_captured_and_on_another_stream():
    c = ic.Cache([900, 333], seed=8).upload()
    ref = decode(c, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = decode(c, 4, stream=side)
    assert torch.equal(ref[0], got[0])
    part = ob.Partials.empty(c.L, c.B, 4)
    out, lse = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    mass = torch.zeros((c.B, c.L.n_kv_heads, c.max_pages * c.L.page_size), device="cuda")
    counters = torch.zeros(c.B * c.L.n_kv_heads, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ob.oscar_decode_attention_int4(*c.attention_args(), part, None, out, lse, counters)
        ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
    for i in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        assert abs(float(mass.sum()) - (i + 1) * c.B * c.L.n_q_heads) < 1e-2
    c2 = ic.Cache([900, 333], seed=18).upload()
    c.dq.copy_(c2.dq), c.dT.copy_(i32([800, 333]))                  # a captured call reads its inputs anew
    c.dh.copy_(i32([600, 77]))
    want = decode(c, 4)[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# -------------------------------------------------------------------- mass --
@pytest.mark.parametrize("seq", LENGTHS)
@pytest.mark.parametrize("n_kv,gqa,page,group", [(2, 4, 16, 128), (8, 4, 64, 128), (1, 8, 32, 32), (5, 1, 16, 64), (2, 2, 64, 32)])
def test_mass_matches_64_bits(seq, n_kv, gqa, page, group):
    c = ic.Cache(seq, n_kv=n_kv, gqa=gqa, page=page, group=group, seed=len(seq) + n_kv, extra_pages=1).upload()
    _, ref_lse = c.attention()
    lse = torch.from_numpy(ref_lse).float().cuda()
    N = c.max_pages * page
    start = c.rng.uniform(0, 1, (c.B, n_kv, N)).astype(np.float32)
    mass = torch.from_numpy(start.copy()).cuda()
    ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
    assert ob.oscar_get_device_status() == 0
    got = mass.double().cpu().numpy()
    lse64 = lse.double().cpu().numpy()
    for b in range(c.B):
        T = int(c.seq[b])
        assert np.array_equal(got[b, :, T:], start[b, :, T:].astype(np.float64))
        for h in range(n_kv):
            add = sum(np.exp(c.logits(b, hq) - lse64[b, hq]) for hq in range(h * gqa, (h + 1) * gqa))
            # each weight is off by its logit's error and a few roundings, the sum by half a step
            tol = (2 * c.logit_error() + 2.0 ** -19 * (1 + np.abs(ref_lse[b]).max())) * add + 2.0 ** -23 * (add + start[b, h, :T])
            assert np.all(np.abs(got[b, h, :T] - start[b, h, :T] - add) <= tol)


def test_mass_of_an_empty_head_and_bad_pages():
    c = ic.Cache([600, 600], seed=4).upload()
    lse = decode(c, 3)[1]
    mass = torch.zeros((2, 2, c.max_pages * 16), device="cuda")
    lse[0, :4] = -float("inf")
    ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
    assert not mass[0, 0].any() and mass[0, 1].any() and torch.isfinite(mass).all()
    ref = mass.clone()
    mass.zero_()
    c.d4[1, 6] = -1
    c.db[0, 0] = -1
    ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
    assert ob.oscar_get_device_status() == BAD_INT4 | BAD_BF16
    ref[1, :, 96:112] = 0
    ref[0, :, :16] = 0
    assert torch.equal(mass, ref)


# ------------------------------------------------------------------- evict --
def evict_reference(mass, sink, he, k):
    m = mass[sink:he].astype(np.float64)
    m = np.where(np.isnan(m), np.inf, m)
    nan = np.isnan(mass[sink:he])
    order = np.lexsort((np.arange(he - sink), -m, ~nan))
    return np.sort(order[:k]) + sink


def run_evict(c, keep, mass, stride=None, fill=-7):
    L, ps = c.L, c.L.page_size
    keep = np.asarray(keep)
    spans = [[(L.sink, L.sink + max(int(k), 0))] for k in keep]
    tn, nn = ic.tables(c.B, spans, ps, c.max_pages, c.rng)
    new = ob.Int4Pool(torch.full((nn, L.n_kv_heads, ps, 64), 0xEE, dtype=torch.uint8, device="cuda"),
                      torch.full((nn, L.n_kv_heads, ps, 64), 0xDD, dtype=torch.uint8, device="cuda"),
                      torch.full((nn, L.n_kv_heads, ps, D // L.group, 4), 3.0, dtype=torch.bfloat16, device="cuda"))
    dm = torch.from_numpy(mass).cuda()
    out = torch.full_like(dm, 11.0)
    kept = torch.full((c.B, L.n_kv_heads, stride or max(1, int(keep.max()))), fill, dtype=torch.int32, device="cuda")
    ob.oscar_evict_int4(L, c.int4, c.d4, new, i32(tn), c.dT, c.dh, i32(keep), dm, out, kept)
    torch.cuda.synchronize()
    return tn, new, out.cpu().numpy(), kept.cpu().numpy()


def check_evict(c, keep, mass, stride=None):
    L, ps = c.L, c.L.page_size
    tn, new, out, kept = run_evict(c, keep, mass, stride)
    nck, ncv, nsz = new.codes_k.cpu().numpy(), new.codes_v.cpu().numpy(), bf16_bits(new.scale_zero)
    osz = bf16_bits(c.int4.scale_zero)
    written = np.zeros((new.n_pages, L.n_kv_heads, ps), bool)
    for b in range(c.B):
        T, he, k = int(c.seq[b]), int(c.hist[b]), int(keep[b])
        if k < 0 or k > max(0, he - L.sink):                         # left alone, or refused
            assert np.all(kept[b] == -7) and np.all(out[b] == 11)
            continue
        for h in range(L.n_kv_heads):
            want = evict_reference(mass[b, h], L.sink, he, k)
            assert np.array_equal(kept[b, h, :k], want)
            assert np.all(kept[b, h, k:] == -7)
            lo = min(L.sink, T)
            m = np.concatenate([mass[b, h, :lo], mass[b, h, want], mass[b, h, max(he, lo):T]])
            assert np.array_equal(out[b, h, :len(m)], m, equal_nan=True) and np.all(out[b, h, len(m):] == 0)
            to = L.sink + np.arange(k)
            src, dst = (c.t4[b, want // ps], h, want % ps), (tn[b, to // ps], h, to % ps)
            assert np.array_equal(nck[dst], c.ck[src]) and np.array_equal(ncv[dst], c.cv[src])
            assert np.array_equal(nsz[dst], osz[src])
            written[dst] = True
    assert np.all(nck[~written] == 0xEE) and np.all(ncv[~written] == 0xDD) and np.all(nsz[~written] == 0x4040)


def weights(rng, shape, kind):
    m = np.exp(rng.normal(0, 2, shape)).astype(np.float32)
    if kind == "ties":
        m = np.round(m).astype(np.float32)
    elif kind == "same":
        m[:] = 0.25
    elif kind == "odd":
        m[rng.random(shape) < 0.2] = 0
        m[rng.random(shape) < 0.2] *= -1
        m[rng.random(shape) < 0.2] = -0.0
        m[rng.random(shape) < 0.02] = np.nan
        m[rng.random(shape) < 0.05] = np.inf
        m[rng.random(shape) < 0.05] = -np.inf
        m[rng.random(shape) < 0.1] = 1e-42
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "same", "odd"])
@pytest.mark.parametrize("n_kv,page,group", [(2, 16, 128), (8, 64, 128), (1, 32, 32), (5, 16, 64)])
def test_evict_matches_a_full_sort(kind, n_kv, page, group):
    c = ic.Cache([1000, 337, 64, 2500, 400, 321], n_kv=n_kv, gqa=1, page=page, group=group, seed=n_kv, extra_pages=1).upload()
    mass = weights(c.rng, (c.B, n_kv, c.max_pages * page), kind)
    n = np.maximum(0, c.hist - 64)
    check_evict(c, [400, 17, 0, 1024, -1, 1], mass)
    check_evict(c, n, mass, int(n.max()) + 3)                        # everything kept: a move
    check_evict(c, np.minimum(n, 1), mass)
    check_evict(c, n // 2, mass)
    assert ob.oscar_get_device_status() == 0


@pytest.mark.parametrize("T", [4500, 40000, 140000])
def test_evict_long_histories(T):
    c = ic.Cache([T], n_kv=2, gqa=1, page=64, seed=1, rubbish=False).upload()
    for kind in ("plain", "ties"):
        mass = weights(c.rng, (1, 2, c.max_pages * 64), kind)
        for k in (1, T // 3, int(c.hist[0]) - 64 - 1):
            check_evict(c, [k], mass)


def test_evict_many_heads_with_long_histories():
    """One CTA a head, with more keys than it holds in shared memory; a request without a history to keep 3 of."""
    c = ic.Cache([20000, 300, 18000], n_kv=64, gqa=1, page=64, seed=1, rubbish=False).upload()
    mass = weights(c.rng, (3, 64, c.max_pages * 64), "ties")
    check_evict(c, [700, 3, 17680], mass)
    assert ob.oscar_get_device_status() == BAD_LENGTH


def test_evict_flags_and_shared_pages():
    c = ic.Cache([600, 600, 600], seed=4)
    c.t4[1], c.t4[2] = c.t4[0], c.t4[0]                              # three requests on the same source pages
    c.upload()
    mass = weights(c.rng, (3, 2, c.max_pages * 16), "plain")
    check_evict(c, [100, 7, 280], mass)
    assert ob.oscar_get_device_status() == 0
    for bad in (281, -2):
        tn, new, out, kept = run_evict(c, [100, bad, 280], mass, 300)
        assert ob.oscar_get_device_status() == BAD_LENGTH
        assert np.all(kept[1] == -7) and np.all(out[1] == 11)
        assert np.array_equal(kept[2, 0, :280], np.arange(64, 344))
    run_evict(c, [100, 7, 280], mass, 200)                           # kept_stride below keep
    assert ob.oscar_get_device_status() == BAD_LENGTH
    c.d4[0, 5] = c.int4.n_pages
    tn, new, out, kept = run_evict(c, [280, 0, 0], mass)
    assert ob.oscar_get_device_status() == BAD_INT4
    assert np.array_equal(kept[0, 1, :280], np.arange(64, 344))


def test_evict_within_one_pool_and_a_kept_view():
    """Source and destination pages of the same pool, apart; kept a larger array than any keep."""
    c = ic.Cache([900], n_kv=2, gqa=1, page=16, seed=3, extra_pages=0)
    n = c.ck.shape[0]
    grow = lambda a: np.concatenate([a, np.zeros((40,) + a.shape[1:], a.dtype)])
    c.ck, c.cv, c.sz = grow(c.ck), grow(c.cv), grow(c.sz)
    c.upload()
    L, mass = c.L, weights(c.rng, (1, 2, c.max_pages * 16), "plain")
    tn = np.full_like(c.t4, -1)
    tn[0, 4:4 + 20] = n + c.rng.permutation(40)[:20]
    dm = torch.from_numpy(mass).cuda()
    out, kept = torch.empty_like(dm), torch.full((1, 2, 500), -7, dtype=torch.int32, device="cuda")
    before = c.int4.codes_k[:n].clone()
    ob.oscar_evict_int4(L, c.int4, c.d4, c.int4, i32(tn), c.dT, c.dh, i32([313]), dm, out, kept)
    assert torch.equal(before, c.int4.codes_k[:n])
    for h in range(2):
        want = evict_reference(mass[0, h], 64, 644, 313)
        assert np.array_equal(kept[0, h, :313].cpu().numpy(), want) and torch.all(kept[0, h, 313:] == -7)
        to = 64 + np.arange(313)
        assert np.array_equal(c.int4.codes_v.cpu().numpy()[tn[0, to // 16], h, to % 16], c.cv[c.t4[0, want // 16], h, want % 16])
    assert ob.oscar_get_device_status() == 0


# ------------------------------------------------------------ order of work --
def test_calls_follow_the_kernels_copies_and_fills_before_them():
    """Each call is launched ahead of its predecessor's end: it still sees what that one wrote, in a stream and in a graph,
    after kernels, copies and fills, and what follows sees what it wrote."""
    c = ic.Cache([900, 340], n_kv=2, gqa=4, page=16, seed=12, rubbish=False).upload()
    L, B = c.L, c.B
    want, want_lse, _ = decode(c, 3)
    N = c.max_pages * 16
    src = [t.clone() for t in (c.int4.codes_k, c.int4.codes_v, c.int4.scale_zero, c.dq)]
    dst = (c.int4.codes_k, c.int4.codes_v, c.int4.scale_zero, c.dq)
    part, counters = ob.Partials.empty(L, B, 3), torch.zeros(B * 2, dtype=torch.int32, device="cuda")
    out, lse, mass, copy = torch.empty_like(want), torch.empty_like(want_lse), torch.zeros((B, 2, N), device="cuda"), torch.empty_like(want)
    big = torch.empty(1 << 26, device="cuda")

    def step():
        for t in dst:                                   # fills, then late copies of the real inputs
            t.zero_()
        big.normal_()
        for t, s in zip(dst, src):
            t.copy_(s)
        mass.zero_()
        ob.oscar_decode_attention_int4(*c.attention_args(), part, None, out, lse, counters)
        ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
        copy.copy_(out)

    ref_mass = torch.zeros_like(mass)
    ob.oscar_attention_mass_int4(*c.attention_args(), want_lse, ref_mass)
    for _ in range(5):
        step()
        torch.cuda.synchronize()
        assert torch.equal(copy, want) and torch.equal(lse, want_lse) and torch.equal(mass, ref_mass)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        copy.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(copy, want) and torch.equal(lse, want_lse) and torch.equal(mass, ref_mass)


def test_a_chain_of_calls_many_times_over():
    """append -> demote -> promote -> append ... back to back on the same pages: every call reads the one before."""
    L = ob.Layout(2, 4, 16)
    a, b, q4 = ob.Bf16Pool.empty(L, 4), ob.Bf16Pool.empty(L, 4), ob.Int4Pool.empty(L, 4)
    t, lo, hi, req, pos = i32([[2, 0, 3, 1]]), i32([0]), i32([64]), i32([0] * 64), i32(np.arange(64))
    x = torch.randn((64, 4, D), device="cuda").to(torch.bfloat16)
    ob.oscar_append_kv(L, None, x[:, :2], x[:, 2:], a, t, req, pos)
    ob.oscar_demote_int4(L, a, t, q4, t, lo, hi)
    ob.oscar_promote_int4(L, q4, t, b, t, lo, hi)
    torch.cuda.synchronize()
    want = b.k.clone(), b.v.clone(), q4.codes_k.clone()
    for _ in range(300):
        a.k.zero_(), q4.codes_k.zero_(), b.k.zero_()
        ob.oscar_append_kv(L, None, x[:, :2], x[:, 2:], a, t, req, pos)
        ob.oscar_demote_int4(L, a, t, q4, t, lo, hi)
        ob.oscar_promote_int4(L, q4, t, b, t, lo, hi)
        assert bool((b.k == want[0]).all() & (b.v == want[1]).all() & (q4.codes_k == want[2]).all())


def test_two_calls_at_once_on_two_streams():
    cs = [ic.Cache([2000, 700], n_kv=2, gqa=4, page=16, seed=s).upload() for s in (1, 2)]
    want = [decode(c, 5) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    work = [(ob.Partials.empty(c.L, c.B, 5), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.empty_like(w[0]), torch.empty_like(w[1]))
            for c, w in zip(cs, want)]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, s, (p, n, o, l) in zip(cs, streams, work):
            ob.oscar_decode_attention_int4(*c.attention_args(), p, None, o, l, n, s)
    torch.cuda.synchronize()
    for (p, n, o, l), w in zip(work, want):
        assert torch.equal(o, w[0]) and torch.equal(l, w[1]) and not n.any()


# ----------------------------------------------------------------- binding --
def test_the_binding_refuses_types_shapes_strides_and_places():
    c = ic.Cache([400], seed=1).upload()
    L, cpu = c.L, lambda t: t.cpu()
    lo, hi = i32([64]), i32([144])
    demote = lambda **k: ob.oscar_demote_int4(L, k.get("src", c.bfp), k.get("bt", c.db), k.get("dst", c.int4), k.get("it", c.d4),
                                              k.get("lo", lo), k.get("hi", hi))
    cases = [(dict(lo=lo.long()), "pos_begin must be torch.int32, not Long"), (dict(hi=i32([1, 2])), "pos_end must have shape .1,., not .2,."),
             (dict(lo=cpu(lo)), "pos_begin is on cpu, not on the current CUDA device"), (dict(it=c.d4[0]), "page tables must be"),
             (dict(bt=c.db[:, :5]), "bf16_page_table must have shape"), (dict(src=ob.Bf16Pool(c.bfp.k.float(), c.bfp.v)), "pool k must be torch.bfloat16"),
             (dict(src=ob.Bf16Pool(c.bfp.k, c.bfp.v[:1])), "pool v must have shape"), (dict(lo=7), "pos_begin must be a tensor"),
             (dict(bt=c.db.t().contiguous().t()), "bf16_page_table must be contiguous" if c.db.shape[0] > 1 else None),
             (dict(dst=ob.Int4Pool(c.int4.codes_k, c.int4.codes_v.view(torch.int8), c.int4.scale_zero)), "codes_v must be torch.uint8"),
             (dict(dst=ob.Int4Pool(c.int4.codes_k, c.int4.codes_v, c.int4.scale_zero[..., :2])), "scale_zero must have shape")]
    before = c.int4.codes_k.clone()
    for kw, text in cases:
        if text:
            with pytest.raises(ob.OscarError, match=text):
                demote(**kw)
    x = torch.zeros((2, 2, D), dtype=torch.bfloat16, device="cuda")
    for bad in (x.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros((2, 2, 2 * D), dtype=torch.bfloat16, device="cuda")[..., ::2]):
        with pytest.raises(ob.OscarError, match="lie together"):
            ob.oscar_append_kv(L, None, bad, x, c.bfp, c.db, i32([0, 0]), i32([0, 1]))
    with pytest.raises(ob.OscarError, match="failed .1.: .*both or neither"):
        ob.oscar_append_kv(L, None, x, x, c.bfp, c.db, i32([0, 0]), i32([0, 1]), q_out=torch.zeros((2, 8, D), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ob.OscarError, match="clip"):
        ob.oscar_demote_int4(L, c.bfp, c.db, c.int4, c.d4, lo, hi, 0.0)
    with pytest.raises(AttributeError):
        demote(src=None)
    with pytest.raises(TypeError):
        ob.oscar_demote_int4(L, c.bfp, c.db, c.int4, c.d4, lo, hi, "1")
    torch.cuda.synchronize()
    assert torch.equal(before, c.int4.codes_k) and ob.oscar_get_device_status() == 0


# ---------------------------------------------------------------- together --
@pytest.mark.parametrize("n_kv,gqa,page,group", [(2, 4, 16, 128), (1, 8, 32, 32)])
def test_a_conversation(n_kv, gqa, page, group):
    """Prompt appended, its history demoted, steps decoded with their weights summed and the leaving token demoted, the
    history evicted to half, its recent pages moved in the table, and more steps decoded: against 64 bits throughout."""
    rng = np.random.default_rng(0)
    L = ob.Layout(n_kv, gqa, page, group)
    Hq, B, prompt, max_pages = n_kv * gqa, 2, np.array([700, 530]), 1024 // page
    rope = rope_table(1100)
    bf = ob.Bf16Pool.empty(L, B * max_pages)
    pools = [ob.Int4Pool.empty(L, B * max_pages) for _ in range(2)]
    db = i32(rng.permutation(B * max_pages).reshape(B, max_pages))
    d4 = [i32(rng.permutation(B * max_pages).reshape(B, max_pages)) for _ in range(2)]
    weight = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    mass = torch.zeros((B, n_kv, max_pages * page), device="cuda")

    def put(tokens, cache_pos, text_pos, req):
        x = torch.from_numpy(rng.normal(0, 1, (tokens, Hq + 2 * n_kv, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        q = torch.empty((tokens, Hq, D), dtype=torch.bfloat16, device="cuda")
        ob.oscar_append_kv(L, x[:, :Hq], x[:, Hq:Hq + n_kv], x[:, Hq + n_kv:], bf, db, i32(req), i32(cache_pos), q, weight, weight,
                           1e-6, rope, 128, False, i32(text_pos))
        return q

    def view(q, T, he, pool, table):
        c = ic.Cache.__new__(ic.Cache)
        c.L, c.B, c.seq, c.hist, c.sm_scale = L, B, np.asarray(T), np.asarray(he), D ** -0.5
        c.t4, c.tb = table.cpu().numpy(), db.cpu().numpy()
        c.ck, c.cv, c.sz = pool.codes_k.cpu().numpy(), pool.codes_v.cpu().numpy(), pool.scale_zero.double().cpu().numpy()
        c.bk, c.bv, c.q = bf.k.double().cpu().numpy(), bf.v.double().cpu().numpy(), q.double().cpu().numpy()
        c.int4, c.bfp, c.d4, c.db, c.dT, c.dh, c.dq = pool, bf, table, db, i32(T), i32(he), q
        return c

    T = prompt.copy()
    put(int(T.sum()), np.concatenate([np.arange(t) for t in T]), np.concatenate([np.arange(t) for t in T]), np.repeat(np.arange(B), T))
    he = T - 256
    ob.oscar_demote_int4(L, bf, db, pools[0], d4[0], i32([64] * B), i32(he))
    text, cur, total = T.copy(), 0, np.zeros((B, n_kv, max_pages * page))
    for step in range(6):
        q = put(B, T, text, np.arange(B))
        T, text = T + 1, text + 1
        c = view(q, T, he, pools[cur], d4[cur])
        out, lse, _ = check_decode(c, 3)
        ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
        for b in range(B):
            for hq in range(Hq):
                total[b, hq // gqa, :T[b]] += np.exp(c.logits(b, hq) - float(lse[b, hq]))
        ob.oscar_demote_int4(L, bf, db, pools[cur], d4[cur], i32(he), i32(he + 1))
        he = he + 1
        if step == 2:
            gone = (he - 64) // 2 // page * page                     # whole pages leave: the recent rows stay where they are
            keep = he - 64 - gone
            new_mass, kept = torch.empty_like(mass), torch.empty((B, n_kv, int(keep.max())), dtype=torch.int32, device="cuda")
            assert np.allclose(mass.double().cpu().numpy(), total, rtol=1e-4, atol=1e-7)
            ob.oscar_evict_int4(L, pools[0], d4[0], pools[1], d4[1], i32(T), i32(he), i32(keep), mass, new_mass, kept)
            before = mass.cpu().numpy()
            rows = kept.cpu().numpy()
            moved = np.zeros_like(total)
            tb = db.cpu().numpy()
            for b in range(B):
                k, g = int(keep[b]), int(gone[b])
                for h in range(n_kv):
                    assert np.array_equal(rows[b, h, :k], evict_reference(before[b, h], 64, int(he[b]), k))
                    moved[b, h, :T[b] - g] = np.concatenate([total[b, h, :64], total[b, h, rows[b, h, :k]], total[b, h, he[b]:T[b]]])
                first = 64 // page
                tb[b, first:max_pages - g // page] = tb[b, first + g // page:].copy()
            total, mass, cur = moved, new_mass, 1
            db.copy_(torch.from_numpy(tb))
            T, he = T - gone, he - gone
    assert np.allclose(mass.double().cpu().numpy(), total, rtol=1e-4, atol=1e-7)
    assert ob.oscar_get_device_status() == 0
