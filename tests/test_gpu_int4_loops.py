"""The 4-bit history's bulk loops past their first turn: sizes chosen from what a launch covers at once."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic
from tests.test_gpu_int4 import append_reference, check_rounded, decode, history_rows, i32, rope_table

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True)
def clean_status():
    ob.oscar_get_device_status()
    yield
    assert ob.oscar_get_device_status() == 0


# One request of 8 kv heads: the demotion's CTAs take 38·64 = 2,432 positions at once in runs of eight, 38·16 = 608 a step at a
# time (ranges up to 1,216), the promotion's 152·16 = 2,432; 64 heads: 256, 64 (up to 128) and 304; two requests half of it.
@pytest.mark.parametrize("n_kv,page,group,ranges", [(8, 64, 128, [(64, 6001)]), (8, 64, 32, [(71, 5990)]), (8, 16, 64, [(3, 1100)]),
                                                     (8, 32, 128, [(65, 1281)]), (8, 64, 64, [(64, 3003), (5, 4999)]), (64, 64, 128, [(7, 1030)]),
                                                     (64, 16, 32, [(1, 128)]), (64, 32, 64, [(64, 64), (33, 1000)])])
def test_demotion_and_promotion_of_many_runs(n_kv, page, group, ranges):
    rng = np.random.default_rng(n_kv + group)
    L, B = ob.Layout(n_kv, 1, page, group), len(ranges)
    max_pages = -(-max(hi for _, hi in ranges) // page)
    tb, nb = ic.tables(B, [[r] for r in ranges], page, max_pages, rng)
    t4, n4 = ic.tables(B, [[r] for r in ranges], page, max_pages, rng)
    rows = [history_rows(rng, (nb, page, n_kv, D)) for _ in range(2)]
    src = ob.Bf16Pool(*(torch.from_numpy(r).to(torch.bfloat16).cuda() for r in rows))
    dst = ob.Int4Pool.empty(L, n4)
    dst.codes_k.fill_(0xAA), dst.codes_v.fill_(0x55), dst.scale_zero.fill_(3.0)
    back = ob.Bf16Pool(torch.full_like(src.k, 7.0), torch.full_like(src.v, 9.0))
    begin, end = i32([r[0] for r in ranges]), i32([r[1] for r in ranges])
    clip = (0.96, 1.0)
    ob.oscar_demote_int4(L, src, i32(tb), dst, i32(t4), begin, end, *clip)
    ob.oscar_promote_int4(L, dst, i32(t4), back, i32(tb), begin, end)
    sz, want_sz = dst.scale_zero.double().cpu().numpy(), np.full((n4, n_kv, page, D // group, 4), 3.0)
    for kind, (codes, fill, restored, rest) in enumerate(((dst.codes_k, 0xAA, back.k, 7.0), (dst.codes_v, 0x55, back.v, 9.0))):
        want, want_back = np.full(codes.shape, fill, np.uint8), np.full(restored.shape, rest)
        for b, (lo, hi) in enumerate(ranges):
            p = np.arange(lo, hi)
            pb, p4, sl = tb[b, p // page], t4[b, p // page], p % page
            code, scale, zero = ic.quantize(rows[kind][pb, sl], group, clip[kind])
            c = code.astype(np.uint8)
            want[p4, :, sl] = c[..., 0::2] | (c[..., 1::2] << 4)
            want_sz[p4, :, sl, :, 2 * kind], want_sz[p4, :, sl, :, 2 * kind + 1] = scale, zero
            g = code.reshape(code.shape[:-1] + (D // group, group))
            want_back[pb, sl] = ic.bf16_once((zero[..., None] + g * scale[..., None]).reshape(code.shape))
        assert np.array_equal(codes.cpu().numpy(), want)
        assert np.array_equal(restored.double().cpu().numpy(), want_back)
    assert np.array_equal(sz, want_sz)


# 16 warps an SM and 152 SMs: 300 tokens leave a warp 3 or 4 pairs of rows, 700 up to 14, 1,300 and more a whole token (24 pairs of
# 32 + 8 + 8 rows, 40 of 64 + 8 + 8); four pairs are in flight.
@pytest.mark.parametrize("tokens", [300, 700, 1300, 3001])
@pytest.mark.parametrize("n_kv,gqa,rot,pairs", [(8, 4, 128, False), (8, 8, 64, True), (8, 8, 128, False), (5, 1, 96, False)])
def test_append_of_many_tokens(tokens, n_kv, gqa, rot, pairs):
    rng = np.random.default_rng(tokens)
    L, Hq, B, most, page = ob.Layout(n_kv, gqa, 64), n_kv * gqa, 3, 1100, 64
    table, n_pages = ic.tables(B, [[(0, most)]] * B, page, -(-most // page), rng)
    slots = rng.permutation(B * most)[:tokens]
    req, pos = slots // most, slots % most
    pos[rng.random(tokens) < 0.05] = -1
    x = torch.from_numpy(rng.normal(0, 3, (tokens, Hq + 2 * n_kv, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    wq, wk = (torch.from_numpy(rng.normal(1, 0.3, D).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    pool = ob.Bf16Pool(*(torch.full((n_pages, page, n_kv, D), f, dtype=torch.bfloat16, device="cuda") for f in (7.0, 9.0)))
    q_out, rope, turn = torch.full((tokens, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda"), rope_table(1200), pos + 100
    ob.oscar_append_kv(L, x[:, :Hq], x[:, Hq:Hq + n_kv], x[:, Hq + n_kv:], pool, i32(table), i32(req), i32(pos), q_out, wq, wk,
                       1e-5, rope, rot, pairs, i32(turn))
    on, xs, angles = pos >= 0, x.double().cpu().numpy(), rope.double().cpu().numpy()[turn]
    got = q_out.double().cpu().numpy()
    qr, qs = append_reference(xs[:, :Hq], wq.double().cpu().numpy(), 1e-5, angles, rot, pairs)
    kr, ks = append_reference(xs[:, Hq:Hq + n_kv], wk.double().cpu().numpy(), 1e-5, angles, rot, pairs)
    check_rounded(got[on], qr[on], qs[on])
    assert np.all(got[~on] == 5)
    k, v = pool.k.double().cpu().numpy(), pool.v.double().cpu().numpy()
    pg, sl = table[req[on], pos[on] // page], pos[on] % page
    check_rounded(k[pg, sl], kr[on], ks[on])
    assert np.array_equal(v[pg, sl], xs[on][:, Hq + n_kv:])
    rest = np.ones(k.shape[:2], bool)
    rest[pg, sl] = False
    assert np.all(k[rest] == 7) and np.all(v[rest] == 9)


def reference(c):
    """Output and log-sum-exp in float64, and logits by (request, query head), each kv head's rows formed once."""
    out, lse, logits = np.zeros(c.q.shape), np.full(c.q.shape[:2], -np.inf), {}
    for b in range(c.B):
        for h in range(c.L.n_kv_heads if c.seq[b] else 0):
            k, v = c.rows(b, h, 0), c.rows(b, h, 1)
            for hq in range(h * c.L.gqa, (h + 1) * c.L.gqa):
                z = logits[b, hq] = k @ c.q[b, hq] * c.sm_scale
                p = np.exp(z - z.max())
                lse[b, hq], out[b, hq] = z.max() + np.log(p.sum()), p @ v / p.sum()
    return out, lse, logits


def check(c, splits):
    out, lse, _ = decode(c, splits)
    ref, ref_lse, logits = reference(c)
    got, got_lse, some = out.double().cpu().numpy(), lse.double().cpu().numpy(), c.seq > 0
    # a lane adds up to 400 probabilities before lanes and warps are joined: 2^-24 each
    assert np.abs(got_lse[some] - ref_lse[some]).max() <= c.logit_error() + 400 * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(ref_lse[some]).max())
    assert np.abs(got[some] - ref[some]).max() <= c.output_error()
    return ref_lse, logits


# One split, 16 warps a CTA (a CTA for each SM at most): a warp loads the page ids of 32 blocks of 32 tokens, 16,384 tokens in all.
@pytest.mark.parametrize("n_kv,gqa,page,group", [(2, 4, 64, 128), (1, 8, 32, 32), (3, 2, 16, 64), (1, 8, 64, 128)])
def test_decode_of_one_split_and_a_long_history(n_kv, gqa, page, group):
    check(ic.Cache([36000 if n_kv == 1 else 20001], n_kv=n_kv, gqa=gqa, page=page, group=group, seed=gqa, rubbish=False).upload(), 1)


# More CTAs than SMs, 8 warps each: page ids last 8,192 tokens.
@pytest.mark.parametrize("n_kv,gqa,page,group,seq", [(40, 1, 64, 128, [9001, 700, 2500, 100]), (20, 8, 64, 32, [9500, 300, 0, 1, 64, 900, 33, 321]),
                                                      (20, 8, 16, 128, [8900] + 7 * [330]), (40, 4, 32, 64, [17000, 320, 500, 65])])
def test_decode_of_a_batch_with_a_long_history(n_kv, gqa, page, group, seq):
    check(ic.Cache(seq, n_kv=n_kv, gqa=gqa, page=page, group=group, seed=n_kv, rubbish=False).upload(), 1)


# Weights: a ring of four blocks a warp, page ids of 32.  24 heads: CTAs of 16 warps, 6 splits, 10 blocks a warp; 80 heads: of 4 warps,
# 7 splits, 13 blocks; 640 heads: two splits of the longest request, 35 blocks.
@pytest.mark.parametrize("n_kv,gqa,page,group,seq", [(8, 4, 64, 128, [30000, 17, 12000]), (8, 2, 32, 32, [30001, 400, 9000]), (40, 1, 64, 64, [12000, 5000]),
                                                      (40, 2, 16, 128, [12001, 2]), (64, 1, 64, 128, [9100] + 9 * [40]), (64, 1, 64, 32, [9100, 0] + 8 * [70])])
def test_weights_of_long_histories(n_kv, gqa, page, group, seq):
    c = ic.Cache(seq, n_kv=n_kv, gqa=gqa, page=page, group=group, seed=group, rubbish=False).upload()
    _, ref_lse, logits = reference(c)
    lse = torch.from_numpy(ref_lse).float().cuda()
    mass = torch.from_numpy(c.rng.uniform(0, 1, (c.B, n_kv, c.max_pages * page)).astype(np.float32)).cuda()
    start = mass.double().cpu().numpy()
    ob.oscar_attention_mass_int4(*c.attention_args(), lse, mass)
    got, lse64, e = mass.double().cpu().numpy(), lse.double().cpu().numpy(), c.logit_error()
    for b in range(c.B):
        T = int(c.seq[b])
        assert np.array_equal(got[b, :, T:], start[b, :, T:])
        for h in range(n_kv if T else 0):
            add = sum(np.exp(logits[b, hq] - lse64[b, hq]) for hq in range(h * gqa, (h + 1) * gqa))
            # as for short histories: the logit's error, a few roundings, half a step of the sum
            tol = (2 * e + 2.0 ** -19 * (1 + np.abs(ref_lse[b]).max())) * add + 2.0 ** -23 * (add + start[b, h, :T])
            assert np.all(np.abs(got[b, h, :T] - start[b, h, :T] - add) <= tol)


def test_page_tables_of_several_requests_must_be_contiguous():
    c = ic.Cache([400, 500], seed=1).upload()
    turned = c.db.t().contiguous().t()
    assert turned.shape == c.db.shape and not turned.is_contiguous()
    with pytest.raises(ob.OscarError, match="bf16_page_table must be contiguous"):
        ob.oscar_demote_int4(c.L, c.bfp, turned, c.int4, c.d4, i32([64, 64]), i32([65, 65]))
    with pytest.raises(ob.OscarError, match="int4_page_table must be contiguous"):
        ob.oscar_promote_int4(c.L, c.int4, c.d4.t().contiguous().t(), c.bfp, c.db, i32([64, 64]), i32([65, 65]))
