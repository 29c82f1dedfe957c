"""Decode attention over the INT4 history held to the accuracy of fp32 sums, and rows of any scale beside each other.

Keys are zero + code·scale with zero 0 and a power of two as scale in the one channel that the queries read, so a logit
is one product and its error does not hide the value product's."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic
from tests.test_gpu_int4 import decode

pytestmark = pytest.mark.gpu
D, CH = 128, 5


def cache(T, hist=None, sink=0, gqa=4, group=128, n_kv=1, page=16, seed=0):
    c = ic.Cache([T], [T if hist is None else hist], n_kv=n_kv, gqa=gqa, page=page, group=group, sink=sink, seed=seed)
    on = np.isfinite(c.sz)
    c.sz[..., 0] = np.where(on[..., 0], 2.0 ** -4, c.sz[..., 0])
    c.sz[..., 1] = np.where(on[..., 1], 0.0, c.sz[..., 1])
    c.q[:] = 0
    c.q[..., CH] = ic.bf16(np.linspace(1, 3, c.q.shape[1]))[None]        # logits 0 .. 2.8 at code 15
    c.sm_scale = 1.0
    return c


def at(c, p):
    """Index of position p's rows in the INT4 arrays (one kv head)."""
    return c.t4[0, p // c.L.page_size], 0, p % c.L.page_size


def check(c, splits):
    """fp32 throughout but for p·scale in two fp16 parts.  Relative to a weight and the size of its value (15 scale + |zero|,
    or the BF16 value): 2^-21 for the parts; for p five roundings of 2^-24 on its logit and its distance from the maximum, and
    2^-22 for the exponential, once for itself and once for the sum it is divided by; 32 steps of 2^-23 for the sums, the join
    and the division; the BF16 rows' p in two bf16 parts 2^-17.  Parts that are fp16 subnormals: 2^-24 absolute, where the
    largest p·scale is brought to 2^11, of which ten raises of the maximum may each lose a factor of sqrt(2): 2^-30 of it a
    token, times the code."""
    out, lse, _ = decode(c, splits)
    got = out.double().cpu().numpy()
    for hq in range(c.L.n_q_heads):
        h = hq // c.L.gqa
        z = c.logits(0, hq)
        w = np.exp(z - z.max())
        w /= w.sum()
        v = c.rows(0, h, 1)
        T, he, sink, ps = len(z), int(c.hist[0]), c.L.sink, c.L.page_size
        p = np.arange(T)
        far = (p >= sink) & (p < he)
        rec = c.sz[c.t4[0, p[far] // ps], h, p[far] % ps]                # [n, groups, 4]
        size, scale = np.abs(v), np.zeros((T, D))
        size[far] = np.repeat(15 * rec[..., 2] + np.abs(rec[..., 3]), c.L.group, 1)
        scale[far] = np.repeat(rec[..., 2], c.L.group, 1)
        of_p = 2.0 ** -22 + 5 * 2.0 ** -24 * (np.abs(z) + z.max() - z)
        rel = 2.0 ** -21 + of_p + w @ of_p + 2.0 ** -18 + np.where(far, 0, 2.0 ** -17)
        err = (w * rel) @ size + 2.0 ** -30 * 15 * T * (w[:, None] * scale).max(0)
        assert np.all(np.abs(got[0, hq] - w @ v) <= err), (hq, (np.abs(got[0, hq] - w @ v) / err).max())
    assert ob.oscar_get_device_status() == 0


SHAPES = [(4, 128), (8, 128), (8, 32), (4, 32), (2, 64), (1, 128)]


@pytest.mark.parametrize("gqa,group", SHAPES)
@pytest.mark.parametrize("T", [31, 700, 3001])
def test_equal_values_come_back_as_they_are(gqa, group, T):
    """Every row's value is 15 in every channel: a weighted mean of equal numbers, whatever the weights' last bits."""
    c = cache(T, gqa=gqa, group=group, seed=T)
    c.cv[:] = 0xFF
    on = np.isfinite(c.sz)
    c.sz[..., 2], c.sz[..., 3] = np.where(on[..., 2], 1.0, c.sz[..., 2]), np.where(on[..., 3], 0.0, c.sz[..., 3])
    check(c.upload(), 1)
    check(c, 3)


@pytest.mark.parametrize("gqa,group", SHAPES)
def test_values_of_any_row(gqa, group):
    c = cache(2600, gqa=gqa, group=group, seed=gqa).upload()
    check(c, 1)
    check(c, 7)


@pytest.mark.parametrize("gqa,group", SHAPES)
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("power", [8, 16, 30, 60])
def test_a_row_of_huge_scale_and_no_weight(gqa, group, first, power):
    """One history row with value scale and zero 2^power times the others' and a weight of e^-120 to e^-40: nothing of it is
    left in the output, and nothing of the others is lost to its scale."""
    c = cache(1500, gqa=gqa, group=group, seed=power)
    row = at(c, 3 if first else 1111)
    c.sz[row][:, 0], c.sz[row][:, 1] = 0.0, -40.0
    c.sz[row][:, 2:] *= 2.0 ** power
    check(c.upload(), 1)
    check(c, 3)


@pytest.mark.parametrize("gqa,group", SHAPES)
@pytest.mark.parametrize("size", [1e3, 1e9, 1e20])
def test_bf16_rows_of_huge_values_and_no_weight(gqa, group, size):
    """The same for the sink's BF16 rows, which are summed before the history."""
    c = cache(1200, sink=16, gqa=gqa, group=group, seed=2)
    used = np.isfinite(c.bk)
    c.bk = np.where(used, 0.0, c.bk)
    c.bk[..., CH] = np.where(used[..., CH], -40.0, c.bk[..., CH])
    c.bv = ic.bf16(np.where(np.isfinite(c.bv), c.bv * size, c.bv))
    check(c.upload(), 1)
    check(c, 2)


@pytest.mark.parametrize("gqa,group", [(4, 128), (8, 32)])
def test_a_flat_tail_behind_one_row(gqa, group):
    """One row of weight 1 and 20,000 of 2^-16 whose sum counts."""
    c = cache(20000, gqa=gqa, group=group, page=64, seed=1)
    c.ck[:] = 0
    c.sz[..., 0] = np.where(np.isfinite(c.sz[..., 0]), 0.75, c.sz[..., 0])
    c.q[..., CH] = np.where(c.q[..., CH] > 0, 1.0, 0.0)
    row = at(c, 777)
    c.ck[row] = 0xFF
    check(c.upload(), 8)


@pytest.mark.parametrize("gqa,group", [(4, 128), (8, 32), (8, 64)])
@pytest.mark.parametrize("order", [1, -1])
def test_weights_that_rise_along_the_history_while_scales_run_over_the_range(gqa, group, order):
    """Logits rise by 60 from the first row to the last while value scales fall from 2^50 to 2^-50, or rise."""
    c = cache(1024, gqa=gqa, group=group, seed=4)
    c.ck[:] = 0
    c.q[..., CH] = 1.0
    for p in range(1024):
        x = p / 1023
        row = at(c, p)
        c.sz[row][:, 1] = ic.bf16(np.float32(60 * x))
        c.sz[row][:, 2:] = ic.bf16(c.sz[row][:, 2:] * 2.0 ** (order * (100 * x - 50)))
    check(c.upload(), 1)


@pytest.mark.parametrize("gqa,group", [(4, 128), (8, 128), (8, 32), (4, 32), (2, 64)])
@pytest.mark.parametrize("splits", [1, 3])
def test_long_sums_are_not_biased(gqa, group, splits):
    """40,001 rows of codes 0 .. 15, zero 0, scale 1: sums that only grow.  The mean relative error over all heads and channels
    is what does not average out.  A sum in the tensor cores may be truncated (2^-23 each); four in a row at most are, one lower
    and one upper part of two tiles, before a rounded addition.  Rounded operations leave 2^-24 sqrt(n) an output for n below
    2^9 additions a lane, over more than 2^6 lanes and outputs together: 2^-24 sqrt(2^9 / 2^6) < 2^-22, and 2^-23 for the
    exponentials."""
    T = 40001
    c = cache(T, gqa=gqa, group=group, n_kv=2, page=64, seed=splits)
    c.sz[..., 2], c.sz[..., 3] = 1.0, 0.0
    c.upload()
    out = decode(c, splits)[0].double().cpu().numpy()
    for_all = []
    for h in range(2):
        v = c.rows(0, h, 1)
        for hq in range(h * gqa, (h + 1) * gqa):
            z = c.logits(0, hq)
            w = np.exp(z - z.max())
            for_all.append(out[0, hq] / (w @ v / w.sum()) - 1)
    assert np.abs(np.mean(for_all)) <= 4 * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23, np.mean(for_all)


@pytest.mark.parametrize("gqa,group", [(4, 128), (8, 32)])
@pytest.mark.parametrize("splits", [1, 9])
def test_a_long_history_of_values_around_zero(gqa, group, splits):
    """131,072 rows whose values are random around zero: the output is the small rest of two sums, codes and zero points, each
    hundreds of times as large.  Their relative error of at most 2^-21 (see above, with 2^-24 sqrt(2^10 / 2^7) for 2^10 additions
    a lane) meets 7.5, the mean code."""
    c = cache(131072, gqa=gqa, group=group, n_kv=1, page=64, seed=9)
    c.sz[..., 2], c.sz[..., 3] = 1.0, -7.5
    c.upload()
    out = decode(c, splits)[0].double().cpu().numpy()
    k, v = c.rows(0, 0, 0), c.rows(0, 0, 1)
    for hq in range(gqa):
        w = np.exp(k @ c.q[0, hq])
        assert np.sqrt(np.mean((out[0, hq] - w @ v / w.sum()) ** 2)) <= 2.0 ** -21 * 7.5


@pytest.mark.parametrize("gqa,group", SHAPES)
@pytest.mark.parametrize("large", [3, 20])
def test_weights_far_below_their_tile_s_largest(gqa, group, large):
    """One row of weight 1 whose codes are 0 and 31 of about 2^-10 with codes 15: the output is theirs.  The tensor cores cut a
    sum's terms off 25 bits below the largest one's exponents, 2^-17 of the largest p·scale for a unit of code at 2^-22 (half of
    the channels; 2^-21 for the others): once for each of the 15 rows of the same tile, and the sum before it."""
    c = cache(32, gqa=gqa, group=group, page=16, seed=large)
    c.q[..., CH] = 1.0
    c.sz[..., 0], c.sz[..., 2], c.sz[..., 3] = ic.bf16(np.float32(0.47)), 1.0, 0.0
    c.ck[:], c.cv[:] = 0, 0xFF
    c.ck[at(c, large)], c.cv[at(c, large)] = 0xFF, 0
    c.upload()
    out = decode(c, 1)[0].double().cpu().numpy()
    z = c.logits(0, 0)
    w = np.exp(z - z.max())
    ref = (w @ c.rows(0, 0, 1) / w.sum())[None]
    cut = np.where(np.arange(D) % 2 == 0, 2.0 ** -17, 2.0 ** -21) * 16 / w.sum()
    assert np.all(np.abs(out[0] - ref) <= cut + 2.0 ** -18 * ref)


@pytest.mark.parametrize("gqa,group", SHAPES)
@pytest.mark.parametrize("scale", [1.0, 2.0, 4.0, 8.0, 16.0, 64.0])
def test_logits_whose_last_bit_is_8(gqa, group, scale):
    """Logits of 2^26 and, from every warp's second block on, 2^26 + 8 in base 2, each an fp32 number: weights of 1 and 2^8, which
    the running maximum need not follow but the scaling of p·scale must."""
    T = 32 * 16 * 3
    c = cache(T, gqa=gqa, group=group, page=16, seed=1)
    c.sm_scale = float(np.log(2))
    assert np.float32(c.sm_scale) * np.float32(1.4426950408889634) == 1
    c.q[..., CH] = 2.0 ** 16
    c.ck[:] = 0
    c.sz[..., 0], c.sz[..., 1], c.sz[..., 2], c.sz[..., 3] = 2.0 ** -13, 2.0 ** 10, scale, -7.5 * scale
    late = np.arange(512, T)
    c.ck[c.t4[0, late // 16], 0, late % 16, CH // 2] = 0x11
    c.upload()
    out = decode(c, 1)[0].double().cpu().numpy()
    w, v = np.where(np.arange(T) < 512, 1.0, 256.0), c.rows(0, 0, 1)
    ref = w @ v / w.sum()
    assert np.all(np.abs(out[0] - ref[None]) <= 2.0 ** -18 * 15 * scale)
