"""Host-side argument checks of the speculative decoding calls, without a GPU: every call here is refused (or, with no work,
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

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder addresses: host-only case")


@pytest.fixture(scope="module")
def L():
    build.build()
    return ob.lib()


def test_the_header_is_exported_and_bound(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "oscar_tree.h")).read()
    names = sorted(set(re.findall(r"OSCAR_API\s+[\w\s\*]*?\b(oscar_\w+)\s*\(", text)))
    assert names == sorted(ob.EXPORTS_TREE) and all(hasattr(L, n) and hasattr(ob, n) for n in names)


def layout(**kw):
    lay = ob.LayoutC(128, 8, 4, 64, 128, 64, 256)
    for k, v in kw.items():
        setattr(lay, k, v)
    return lay


def bf16_pool(n_pages=4, addr=FAKE):
    return ob.Bf16PoolC(addr, addr, n_pages)


def tree(L, lay=None, q=FAKE, n=3, begin=FAKE, mask=FAKE, words=1, nodes=3, bf=None, bpt=FAKE, i4=None, ipt=FAKE, max_pages=4, T=FAKE, he=FAKE, batch=1,
         splits=4, out=FAKE, lse=FAKE):
    part = ob.PartialsC(FAKE, FAKE, FAKE, splits)
    return L.oscar_tree_attention_int4(ctypes.byref(lay or layout()), q, n, begin, mask, words, nodes, ctypes.byref(bf or bf16_pool()), bpt,
                                       ctypes.byref(i4 or ob.Int4PoolC(FAKE, FAKE, FAKE, 4)), ipt, max_pages, T, he, batch, 0.1, ctypes.byref(part), out,
                                       lse, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=FAKE + 2), dict(begin=None), dict(n=-1), dict(n=65535 * 256 + 1), dict(nodes=0), dict(nodes=257), dict(words=0), dict(nodes=33),
    dict(words=-1), dict(bpt=None), dict(ipt=None), dict(T=None), dict(he=None), dict(out=None), dict(out=FAKE + 4), dict(max_pages=0),
    dict(max_pages=2 ** 30), dict(max_pages=2 ** 25 - 15), dict(batch=-1), dict(batch=65536), dict(splits=0), dict(splits=1025), dict(bf=ob.Bf16PoolC(None, FAKE, 4)),
    dict(bf=ob.Bf16PoolC(FAKE, FAKE, 0)), dict(i4=ob.Int4PoolC(FAKE, FAKE, FAKE + 8, 4)), dict(lay=layout(sink=40))])
def test_tree_attention_refuses(L, kw):
    assert tree(L, **kw) == INVALID
    assert L.oscar_last_error_string()


@pytest.mark.parametrize("kw", [dict(lay=layout(head_dim=64)), dict(lay=layout(gqa=3)), dict(lay=layout(group=16)), dict(lay=layout(page_size=128))])
def test_tree_attention_does_not_support(L, kw):
    assert tree(L, **kw) == UNSUPPORTED


def test_no_work_is_done_for_no_nodes(L):
    assert tree(L, n=0, q=None) == OK and tree(L, batch=0) == OK


def sample(L, x=FAKE, dtype=0, stride=100, rows=2, vocab=100, temp=FAKE, u=FAKE, tokens=FAKE):
    return L.oscar_sample(x, dtype, stride, rows, vocab, temp, None, None, None, u, tokens, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=FAKE + 2), dict(x=FAKE + 1, dtype=1), dict(stride=99), dict(rows=-1), dict(rows=65536), dict(vocab=0),
                                dict(vocab=262145, stride=2 ** 20), dict(temp=None), dict(u=None), dict(tokens=None)])
def test_sample_refuses(L, kw):
    assert sample(L, **kw) == INVALID


def test_sample_types_and_no_rows(L):
    assert sample(L, dtype=3) == UNSUPPORTED and sample(L, dtype=-1) == UNSUPPORTED
    assert sample(L, rows=0, x=None) == OK


def accept(L, lay=None, target=FAKE, draft=FAKE, parents=FAKE, n=3, begin=FAKE, nodes=3, T=FAKE, batch=1, accepted=FAKE, path=FAKE, tokens=FAKE, stride=3,
           new_len=FAKE + 4096, pools=None, n_pools=None, pt=FAKE, max_pages=4):
    pools = [bf16_pool()] if pools is None else pools
    array = (ob.Bf16PoolC * max(1, len(pools)))(*pools)
    return L.oscar_tree_accept(ctypes.byref(lay or layout()), target, draft, parents, n, begin, nodes, T, batch, accepted, path, tokens, stride, new_len, array,
                               len(pools) if n_pools is None else n_pools, pt, max_pages, None)


@pytest.mark.parametrize("kw", [
    dict(target=None), dict(draft=None), dict(parents=None), dict(n=-1), dict(begin=None), dict(nodes=0), dict(nodes=257, stride=300), dict(T=None), dict(batch=-1),
    dict(batch=65536), dict(accepted=None), dict(path=None), dict(tokens=None), dict(stride=2), dict(new_len=FAKE), dict(new_len=FAKE + 4, batch=3),
    dict(pools=[bf16_pool(), ob.Bf16PoolC(FAKE, None, 4)]), dict(pools=[bf16_pool(0)]), dict(n_pools=-1), dict(n_pools=4097), dict(pt=None), dict(max_pages=0),
    dict(lay=layout(sink=40))])
def test_accept_refuses(L, kw):
    assert accept(L, **kw) == INVALID


def test_accept_of_no_requests(L):
    assert accept(L, batch=0) == OK


def test_split_suggestions(L):
    lay = ob.Layout(8, 4, 64)
    for batch in (1, 3, 16, 64, 1000):
        for nodes in (1, 4, 8, 64, 256):
            for hist in (1, 500, 100000, 2 ** 31 - 1):
                assert 1 <= ob.oscar_suggest_splits_tree_int4(lay, batch, nodes, hist, 152) <= 1024
    assert ob.oscar_suggest_splits_tree_int4(lay, 0, 4, 100, 152) == 1 and ob.oscar_suggest_splits_tree_int4(lay, 4, 4, 0, 152) == 1


@no_gpu
def test_the_binding_refuses_without_a_device():
    x = torch.zeros((2, 10))
    with pytest.raises(ob.OscarError):
        ob.oscar_sample(x, torch.ones(2), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
