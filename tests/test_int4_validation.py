"""Host-side argument checks of the INT4 entry points, without a GPU: every call here is refused (or, with no work,
accepted) before the library makes a CUDA call."""
import ctypes
import os
import re

import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from bit_kv_cache_oscar_gb300 import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x7F0000000000          # 16-byte aligned placeholder address (never dereferenced)
OFF = FAKE + 8

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder addresses: host-only case")


@pytest.fixture(scope="module")
def L():
    build.build()
    return ob.lib()


def test_the_header_is_exported_and_bound(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "oscar_int4.h")).read()
    names = sorted(set(re.findall(r"OSCAR_API\s+[\w\s\*]*?\b(oscar_\w+)\s*\(", text)))
    assert names == sorted(ob.EXPORTS_INT4) and all(hasattr(L, n) and hasattr(ob, n) for n in names)


def layout(**kw):
    lay = ob.LayoutC(128, 8, 4, 64, 128, 64, 256)
    for k, v in kw.items():
        setattr(lay, k, v)
    return lay


def bf16_pool(n_pages=4, addr=FAKE):
    return ob.Bf16PoolC(addr, addr, n_pages)


def int4_pool(n_pages=4, addr=FAKE, sz=FAKE):
    return ob.Int4PoolC(addr, addr, sz, n_pages)


def err(L):
    return L.oscar_last_error_string().decode()


def append(L, lay=None, q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, n=1, wq=FAKE, wk=FAKE, eps=1e-6, rope=FAKE, rows=8,
           rot=128, pool=None, pt=FAKE, max_pages=4, batch=1, req=FAKE, pos=FAKE, q_out=FAKE):
    return L.oscar_append_kv(ctypes.byref(lay or layout()), q, qs, k, ks, v, vs, n, wq, wk, eps, rope, rows, rot, 0,
                             ctypes.byref(pool or bf16_pool()), pt, max_pages, batch, req, pos, None, q_out, None)


def demote(L, lay=None, src=None, dst=None, bpt=FAKE, ipt=FAKE, max_pages=4, batch=1, lo=FAKE, hi=FAKE, cK=1.0, cV=1.0):
    return L.oscar_demote_int4(ctypes.byref(lay or layout()), ctypes.byref(src or bf16_pool()), bpt, ctypes.byref(dst or int4_pool()),
                               ipt, max_pages, batch, lo, hi, cK, cV, None)


def promote(L, lay=None, src=None, dst=None, bpt=FAKE, ipt=FAKE, max_pages=4, batch=1, lo=FAKE, hi=FAKE):
    return L.oscar_promote_int4(ctypes.byref(lay or layout()), ctypes.byref(src or int4_pool()), ipt, ctypes.byref(dst or bf16_pool()),
                                bpt, max_pages, batch, lo, hi, None)


def decode(L, lay=None, q=FAKE, bf=None, i4=None, bpt=FAKE, ipt=FAKE, max_pages=4, T=FAKE, he=FAKE, batch=1, splits=4, out=FAKE,
           lse=FAKE, part=None):
    part = part or ob.PartialsC(FAKE, FAKE, FAKE, splits)
    return L.oscar_decode_attention_int4(ctypes.byref(lay or layout()), q, ctypes.byref(bf or bf16_pool()), bpt,
                                         ctypes.byref(i4 or int4_pool()), ipt, max_pages, T, he, batch, 0.1, ctypes.byref(part), out,
                                         None, lse, None, None)


def mass(L, lay=None, q=FAKE, i4=None, max_pages=4, T=FAKE, batch=1, lse=FAKE, m=FAKE):
    return L.oscar_attention_mass_int4(ctypes.byref(lay or layout()), q, ctypes.byref(bf16_pool()), FAKE, ctypes.byref(i4 or int4_pool()),
                                       FAKE, max_pages, T, FAKE, batch, 0.1, lse, m, None)


def evict(L, lay=None, src=None, spt=FAKE, dst=None, dpt=FAKE + 64, max_pages=4, batch=1, keep=FAKE, m=FAKE, mo=FAKE + (1 << 20),
          kept=FAKE, stride=4):
    return L.oscar_evict_int4(ctypes.byref(lay or layout()), ctypes.byref(src or int4_pool()), spt, ctypes.byref(dst or int4_pool()), dpt,
                              max_pages, batch, FAKE, FAKE, keep, m, mo, kept, stride, None)


ALL = [append, demote, promote, decode, mass, evict]


@no_gpu
@pytest.mark.parametrize("call", ALL)
def test_layout_tables_and_batch(L, call):
    assert call(L, lay=layout(head_dim=64)) == UNSUPPORTED
    assert call(L, lay=layout(gqa=3)) == UNSUPPORTED
    assert call(L, max_pages=0) == INVALID and "max_pages" in err(L)
    assert call(L, max_pages=(1 << 31) // 64) == INVALID and "int32" in err(L)
    assert call(L, batch=65536) == INVALID and "batch" in err(L)
    assert call(L, batch=-1) == INVALID
    if call is not append:
        assert call(L, batch=0) == OK
    else:
        assert call(L, n=0) == OK and call(L, batch=0) == INVALID


@no_gpu
@pytest.mark.parametrize("call,which", [(demote, "dst"), (promote, "src"), (decode, "i4"), (mass, "i4"), (evict, "src"), (evict, "dst")])
def test_int4_pool(L, call, which):
    for pool, text in ((int4_pool(addr=None), "NULL"), (int4_pool(sz=None), "NULL"), (int4_pool(addr=OFF), "aligned"), (int4_pool(sz=OFF), "aligned"),
                       (int4_pool(n_pages=0), "n_pages"), (int4_pool(n_pages=(1 << 31) // 512), "2^31")):
        assert call(L, **{which: pool}) == INVALID and text in err(L), text


@no_gpu
def test_append_arguments(L):
    assert append(L, q=None) == INVALID and "both or neither" in err(L)
    assert append(L, q_out=None) == INVALID
    for name in ("k", "v", "pt", "req", "pos"):
        assert append(L, **{name: None}) == INVALID and "NULL" in err(L)
    for name in ("q", "k", "v", "q_out", "wq", "wk", "rope"):
        assert append(L, **{name: OFF}) == INVALID and "aligned" in err(L)
    for kw in (dict(qs=4095), dict(qs=4088), dict(ks=1016), dict(vs=1028)):
        assert append(L, **kw) == INVALID and "strides" in err(L)
    assert append(L, qs=6144) == INVALID and "q_out may be q" in err(L)
    for rot in (0, 8, 24, 144):
        assert append(L, rot=rot) == INVALID and "rot_dim" in err(L)
    assert append(L, rows=0) == INVALID and "rope_rows" in err(L)
    for eps in (-1e-6, float("nan"), float("inf")):
        assert append(L, eps=eps) == INVALID and "eps" in err(L)
    assert append(L, n=-1) == INVALID and append(L, n=65535 * 256 + 1) == INVALID


@no_gpu
def test_other_arguments(L):
    for name in ("bpt", "ipt", "lo", "hi"):
        assert demote(L, **{name: None}) == INVALID and promote(L, **{name: None}) == INVALID
    assert demote(L, cK=0.0) == INVALID and demote(L, cV=float("nan")) == INVALID and "clip" in err(L)
    for name in ("q", "bpt", "ipt", "T", "he"):
        assert decode(L, **{name: None}) == INVALID and "NULL" in err(L)
    assert decode(L, q=OFF) == INVALID and mass(L, q=OFF) == INVALID and "aligned" in err(L)
    assert decode(L, splits=0) == INVALID and decode(L, splits=1025) == INVALID
    assert decode(L, out=None) == INVALID and "lse" in err(L)
    assert decode(L, part=ob.PartialsC(FAKE, FAKE, None, 4)) == INVALID
    for name in ("q", "T", "lse", "m"):
        assert mass(L, **{name: None}) == INVALID
    for name in ("spt", "dpt", "keep", "m", "mo", "kept"):
        assert evict(L, **{name: None}) == INVALID
    assert evict(L, stride=0) == INVALID and "kept_stride" in err(L)
    assert evict(L, dpt=FAKE) == INVALID and "pages of their own" in err(L)
    assert evict(L, mo=FAKE) == INVALID and "overlap" in err(L)
    assert evict(L, mo=FAKE + 4 * (8 * 256 - 1)) == INVALID and "overlap" in err(L)


def test_suggested_splits(L):
    lay = ob.Layout(8, 4, 64)
    for batch in (1, 2, 32, 1000):
        for tokens in (1, 32, 33, 5000, 131072, 10 ** 9):
            s = ob.oscar_suggest_splits_int4(lay, batch, tokens, 152)
            assert 1 <= s <= min(1024, -(-tokens // 32))
    assert ob.oscar_suggest_splits_int4(lay, 0, 100, 152) == 1 and ob.oscar_suggest_splits_int4(lay, 1, 0, 152) == 1


def test_the_binding_needs_a_device():
    lay = ob.Layout(2, 4, 16)
    i4, bf = ob.Int4Pool.empty(lay, 3, "cpu"), ob.Bf16Pool.empty(lay, 3, "cpu")
    pt, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ob.OscarError, match="current CUDA device"):      # CPU tensors, with and without a GPU
        ob.oscar_demote_int4(lay, bf, pt, i4, pt, one, one)
