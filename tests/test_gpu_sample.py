"""Sampling on the GPU: tokens equal to those of 64-bit arithmetic from the definition."""
import math

import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def reference(x, temp, u, k=None, p=None, m=None):
    """x [rows, vocab] in float64."""
    got = []
    for r in range(len(x)):
        row = np.where(np.isnan(x[r]), -np.inf, x[r])
        top = row.max()
        if top == -np.inf:
            got.append(-1)
            continue
        t = float(temp[r])
        if not t > 0:
            got.append(int(np.argmax(row)))
            continue
        order = np.argsort(-row, kind="stable")
        with np.errstate(invalid="ignore"):
            w = np.where(row == top, 1.0, np.where(row == -np.inf, 0.0, np.exp((row - top) / t)))
        ws = w[order]
        n = len(ws)
        if k is not None and k[r] > 0:
            n = min(n, int(k[r]))
        if p is not None and p[r] < 1:
            sums = np.cumsum(ws[:n])
            n = min(n, int(np.searchsorted(sums, max(0.0, float(p[r])) * sums[-1], side="left")) + 1)
        if m is not None and m[r] > 0:
            n = min(n, int((ws >= float(m[r])).sum()))
        ids = np.sort(order[:max(1, n)])
        sums = np.cumsum(w[ids])
        got.append(int(ids[min(int(np.searchsorted(sums, float(u[r]) * sums[-1], side="right")), len(ids) - 1)]))
    return np.array(got)


def run(x, temp, u, k=None, p=None, m=None, stream=None):
    put = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t, device="cuda")  # noqa: E731
    tokens = torch.full((x.shape[0],), -7, dtype=torch.int32, device="cuda")
    f = torch.float32
    ob.oscar_sample(x, put(temp, f), put(u, f), tokens, put(k, torch.int32), put(p, f), put(m, f), stream=stream)
    return tokens


def check(x, temp, u, **kw):
    got = run(x, temp, u, **kw).cpu().numpy()
    f32 = {n: None if a is None else np.asarray(a, np.float32).astype(np.float64) if n != "k" else a for n, a in kw.items()}
    want = reference(x.double().cpu().numpy(), np.asarray(temp, np.float32), np.asarray(u, np.float32), **f32)
    assert np.array_equal(got, want), (got[got != want][:5], want[got != want][:5], np.flatnonzero(got != want)[:5])


def logits(rows, vocab, dtype, rng, kind="mixed"):
    x = rng.normal(0, 2, (rows, vocab))
    if kind == "mixed":
        x += (rng.random((rows, vocab)) < 0.002) * rng.uniform(0, 14, (rows, vocab))
    elif kind == "flat":
        x *= 0.02
    elif kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "peak":
        x[np.arange(rows), rng.integers(0, vocab, rows)] = 60
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 255, 2049, 32000, 151936, 262144])
@pytest.mark.parametrize("kind", ["mixed", "flat", "ties", "equal", "peak"])
def test_tokens_match_64_bits(dtype, vocab, kind):
    rng = np.random.default_rng(vocab + len(kind))
    rows = 12
    x = logits(rows, vocab, dtype, rng, kind)
    temp, u = rng.uniform(0.2, 1.6, rows), rng.random(rows)
    k, p, m = rng.integers(1, max(2, vocab), rows), rng.uniform(0.05, 0.999, rows), 10.0 ** rng.uniform(-5, -0.3, rows)
    small = np.minimum(k, rng.integers(1, 300, rows))
    check(x, temp, u)
    check(x, temp, u, k=k)
    check(x, temp, u, k=small)
    check(x, temp, u, p=p)
    check(x, temp, u, m=m)
    check(x, temp, u, k=small, p=p, m=m)
    check(x, temp, u, k=k, p=p, m=m)


@pytest.mark.parametrize("rows", [1, 5, 100, 400])
def test_rows_of_every_count(rows):
    rng = np.random.default_rng(rows)
    x = logits(rows, 5000, torch.bfloat16, rng)
    check(x, np.full(rows, 0.8), rng.random(rows), k=np.full(rows, 40), p=np.full(rows, 0.95))


def test_values_that_switch_a_filter_off():
    rng = np.random.default_rng(1)
    x = logits(8, 3000, torch.float32, rng)
    temp, u = np.full(8, 0.9), rng.random(8)
    plain = run(x, temp, u)
    for kw in (dict(k=[0] * 8), dict(k=[-3] * 8), dict(k=[3000] * 8), dict(k=[2 ** 31 - 1] * 8), dict(p=[1.0] * 8), dict(p=[7.0] * 8),
               dict(p=[math.nan] * 8), dict(m=[0.0] * 8), dict(m=[-1.0] * 8), dict(m=[math.nan] * 8)):
        assert torch.equal(run(x, temp, u, **kw), plain), kw
    first = x.argmax(1).int()
    for kw in (dict(k=[1] * 8), dict(p=[0.0] * 8), dict(p=[-2.0] * 8), dict(m=[1.0] * 8), dict(m=[5.0] * 8), dict(m=[math.inf] * 8)):
        assert torch.equal(run(x, temp, u, **kw), first), kw


def test_temperatures():
    rng = np.random.default_rng(2)
    x = logits(7, 4000, torch.bfloat16, rng)
    x[:, 9] = x[:, 1234] = x.amax(1)                             # ties of the largest: the lowest index
    u = rng.random(7)
    for t in (0.0, -1.0, math.nan, -math.inf):
        assert torch.equal(run(x, [t] * 7, u, k=[50] * 7, p=[0.9] * 7), (x == x.amax(1, keepdim=True)).int().argmax(1).int()), t
    check(x, [1e-3] * 7, u)
    check(x, [1e-30] * 7, u)
    check(x, [100.0] * 7, u, p=[0.5] * 7)
    x[:, 100:200] = -math.inf
    check(x, [math.inf] * 7, u)
    check(x, [math.inf] * 7, u, k=[17] * 7, m=[0.5] * 7)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(dtype):
    rng = np.random.default_rng(3)
    x = logits(6, 2500, dtype, rng)
    x[0, 1000:] = -math.inf
    x[1] = -math.inf
    x[2] = math.nan
    x[3, ::2] = math.nan
    x[4, [5, 77, 2000]] = math.inf
    x[5, :] = -math.inf
    x[5, 2499] = -60000.0
    u = rng.random(6)
    check(x, [0.7] * 6, u)
    check(x, [0.7] * 6, u, k=[2] * 6, p=[0.6] * 6, m=[0.01] * 6)
    check(x, [0.0] * 6, u)


def test_uniform_numbers_at_the_ends():
    rng = np.random.default_rng(4)
    x = logits(5, 1000, torch.float32, rng, "equal")
    u = [0.0, 1.0 - 2.0 ** -24, 0.5, 2.0 ** -60, 0.25]
    check(x, [1.0] * 5, u)
    assert run(x, [1.0] * 5, [-1.0, 1.0, 2.0, math.inf, 0.0]).tolist() == [0, 999, 999, 999, 0]
    check(x, [1.0] * 5, u, k=[10] * 5)


def test_every_token_at_its_share():
    """A row whose weights are known: u steps through it, each token for as many steps as its weight."""
    x = torch.tensor([[math.log(1), math.log(2), -math.inf, math.log(5)]], device="cuda").repeat(800, 1)
    u = (np.arange(800) + 0.5) / 800
    assert torch.bincount(run(x, np.ones(800), u).long(), minlength=4).tolist() == [100, 200, 0, 500]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift,extra", [(1, 3), (3, 8), (7, 1), (8, 16)])
def test_strides_and_alignments(dtype, shift, extra):
    rng = np.random.default_rng(5)
    wide = logits(9, 1500 + shift + extra, dtype, rng)
    x = wide[:, shift:shift + 1500]
    check(x, np.full(9, 0.9), rng.random(9), k=np.full(9, 30))
    check(x, np.full(9, 0.9), rng.random(9))


def test_what_lies_between_rows_is_not_read():
    x = torch.full((4, 64), math.nan, device="cuda")
    x[:, :33] = 0.0
    assert torch.all(run(x[:, :33], [1.0] * 4, [0.999] * 4) == 32)


def test_many_draws_without_a_miss():
    """What fp32 sums would miss by: 2,000 draws from a nearly flat row of a large vocabulary."""
    rng = np.random.default_rng(6)
    x = logits(1, 151936, torch.float32, rng, "flat")
    u = rng.random(2000).astype(np.float32)
    got = np.concatenate([run(x.expand(200, -1), np.ones(200), u[i:i + 200]).cpu().numpy() for i in range(0, 2000, 200)])
    w = np.exp(x.double().cpu().numpy()[0])
    sums = np.cumsum(w)
    assert np.array_equal(got, np.searchsorted(sums, u.astype(np.float64) * sums[-1], side="right"))


def test_captured_and_on_other_streams():
    rng = np.random.default_rng(7)
    x = logits(20, 32000, torch.bfloat16, rng)
    temp, u, k = (torch.as_tensor(a, dtype=t, device="cuda") for a, t in ((np.full(20, 0.8), torch.float32), (rng.random(20), torch.float32),
                                                                         (np.full(20, 50), torch.int32)))
    want = run(x, temp.cpu(), u.cpu(), k=k.cpu())
    tokens = torch.zeros(20, dtype=torch.int32, device="cuda")
    ob.oscar_sample(x, temp, u, tokens, top_k=k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ob.oscar_sample(x, temp, u, tokens, top_k=k)
    tokens.zero_()
    g.replay()
    assert torch.equal(tokens, want)
    keep = u.clone()
    u.copy_(1 - u)
    g.replay()
    assert torch.equal(tokens, run(x, temp.cpu(), u.cpu(), k=k.cpu()))
    u.copy_(keep)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], [torch.zeros_like(tokens) for _ in range(3)]
    for _ in range(10):
        for s, o in zip(streams, outs):
            ob.oscar_sample(x, temp, u, o, top_k=k, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
