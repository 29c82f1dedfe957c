"""oscar_append_kv leaves what it neither normalises nor rotates as it is: every bit pattern, beside any neighbour."""
import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests.test_gpu_int4 import append_reference, check_rounded, i32, rope_table

pytestmark = pytest.mark.gpu
D = 128
ODD = [0x7F80, 0xFF80, 0x8000, 0x0001, 0x8001, 0x7F7F, 0xFF7F, 0x7FC0, 0xFFC1, 0x0080]     # +-inf, -0, subnormals, largest, NaN


def rows(rng, n, heads, first):
    """Random bf16 rows as int16 bits; odd values at random in channels from `first` on."""
    x = torch.from_numpy(rng.normal(0, 2, (n, heads, D)).astype(np.float32)).to(torch.bfloat16)
    bits = x.view(torch.int16).numpy().copy()
    at = rng.random(bits.shape) < 0.2
    at[..., :first] = False
    bits[at] = rng.choice(np.array(ODD, np.uint16).view(np.int16), int(at.sum()))
    return torch.from_numpy(bits).cuda()


def append(L, q, k, v, **kw):
    n = k.shape[0]
    pool = ob.Bf16Pool.empty(L, -(-n // L.page_size))
    table = i32(np.arange(pool.n_pages)[None])
    out = torch.zeros_like(q)
    bf = lambda t: t.view(torch.bfloat16)
    ob.oscar_append_kv(L, bf(q), bf(k), bf(v), pool, table, i32([0] * n), i32(np.arange(n)), bf(out), **kw)
    assert ob.oscar_get_device_status() == 0
    flat = lambda t: t.view(torch.int16).flatten(0, 1)[:n]
    return out, flat(pool.k), flat(pool.v)


@pytest.mark.parametrize("n_kv,gqa", [(2, 4), (1, 1), (5, 2), (8, 8)])
@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("pairs", [False, True])
def test_nothing_to_do_moves_every_bit(n_kv, gqa, tokens, pairs):
    rng = np.random.default_rng(n_kv)
    L = ob.Layout(n_kv, gqa, 16)
    q, k, v = (rows(rng, tokens, h, 0) for h in (n_kv * gqa, n_kv, n_kv))
    got = append(L, q, k, v, interleaved=pairs)
    assert all(torch.equal(a, b) for a, b in zip(got, (q, k, v)))


@pytest.mark.parametrize("rot", [16, 48, 64, 112])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens", [1, 40])
def test_channels_beyond_the_rotation(rot, pairs, tokens):
    rng = np.random.default_rng(rot)
    L = ob.Layout(2, 4, 16)
    q, k, v = (rows(rng, tokens, h, rot) for h in (8, 2, 2))
    rope = rope_table(64)
    got = append(L, q, k, v, rope=rope, rot_dim=rot, interleaved=pairs)
    angles = rope.double().cpu().numpy()[:tokens]
    for a, x in zip(got[:2], (q, k)):
        assert torch.equal(a[..., rot:], x[..., rot:])
        f = lambda t: np.nan_to_num(t.view(torch.bfloat16).double().cpu().numpy(), posinf=0, neginf=0)
        ref, size = append_reference(f(x), None, 0.0, angles, rot, pairs)
        check_rounded(f(a)[..., :rot], ref[..., :rot], size[..., :rot])
    assert torch.equal(got[2], v)


@pytest.mark.parametrize("pairs", [False, True])
def test_one_of_queries_and_keys_normalised(pairs):
    rng = np.random.default_rng(3)
    L = ob.Layout(2, 4, 16)
    w = torch.from_numpy(rng.normal(1, 0.3, D).astype(np.float32)).to(torch.bfloat16).cuda()
    for which in (0, 1):
        x = [rows(rng, 40, h, D if i == which else 0) for i, h in enumerate((8, 2, 2))]
        got = append(L, *x, interleaved=pairs, **{("q_weight", "k_weight")[which]: w})
        f = lambda t: t.view(torch.bfloat16).double().cpu().numpy()
        check_rounded(f(got[which]), *append_reference(f(x[which]), w.double().cpu().numpy(), 1e-6, None, 0, pairs))
        assert torch.equal(got[1 - which], x[1 - which]) and torch.equal(got[2], x[2])
