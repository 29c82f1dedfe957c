"""The bound on histories that chooses tree attention's kernel: refusals, without a GPU."""
import ctypes

import pytest

from bit_kv_cache_oscar_gb300 import binding as ob
from tests.test_tree_validation import FAKE, INVALID, L, OK, bf16_pool, layout  # noqa: F401


def bounded(L, max_hist, q=FAKE, n=3, lay=None, words=1, max_pages=4):  # noqa: F811
    part = ob.PartialsC(FAKE, FAKE, FAKE, 4)
    return L.oscar_tree_attention_int4_bounded(ctypes.byref(lay or layout()), q, n, FAKE, FAKE, words, 3, ctypes.byref(bf16_pool()), FAKE,
                                               ctypes.byref(ob.Int4PoolC(FAKE, FAKE, FAKE, 4)), FAKE, max_pages, max_hist, FAKE, FAKE, 1, 0.1,
                                               ctypes.byref(part), FAKE, FAKE, None)


@pytest.mark.parametrize("kw", [dict(max_hist=0), dict(max_hist=-1), dict(max_hist=100, q=None), dict(max_hist=100, words=0), dict(max_hist=100, max_pages=0),
                                dict(max_hist=100, lay=layout(sink=40))])
def test_the_bounded_call_refuses(L, kw):  # noqa: F811
    assert bounded(L, **kw) == INVALID
    assert L.oscar_last_error_string()


def test_the_bounded_call_without_nodes(L):  # noqa: F811
    assert bounded(L, 1, n=0) == OK and bounded(L, 2 ** 31 - 1, n=0) == OK
