"""A Layout handed to the INT4 calls stays what its fields say: copied, sent to another process, shared by threads."""
import copy
import gc
import pickle
import threading

import numpy as np
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from bit_kv_cache_oscar_gb300 import build
from tests import int4_case as ic


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


FIELDS = {"n_kv_heads", "gqa", "page_size", "group", "sink", "recent", "head_dim", "levels_k", "levels_v"}


def refused_call(lay):
    """A call that every machine refuses, its tensors being on the CPU."""
    i4, bf = ob.Int4Pool.empty(ob.Layout(2, 4, 16), 3, "cpu"), ob.Bf16Pool.empty(ob.Layout(2, 4, 16), 3, "cpu")
    pt, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ob.oscar_demote_int4(lay, bf, pt, i4, pt, one, one)


@pytest.mark.parametrize("other", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_a_used_layout_carries_nothing_but_its_fields(other):
    lay = ob.Layout(2, 4, 16)
    with pytest.raises(ob.OscarError, match="current CUDA device"):
        refused_call(lay)
    assert set(vars(lay)) == FIELDS
    twin = other(lay)
    assert twin == lay and set(vars(twin)) == FIELDS


@pytest.mark.parametrize("field,value,error,text", [("gqa", 1 << 31, ob.OscarError, "passes 32 bits"), ("sink", "64", TypeError, "integer"),
                                                     ("page_size", 16.0, TypeError, "integer"), ("levels_k", (0.0, 1.0, 2.0, 3.0), ob.OscarError, "levels"),
                                                     ("levels_v", (0.0, 1.0), ob.OscarError, "levels")])
def test_a_layout_of_other_types_is_refused(field, value, error, text):
    with pytest.raises(error, match=text):
        refused_call(ob.Layout(**{**dict(n_kv_heads=2, gqa=4, page_size=16), field: value}))
    with pytest.raises(AttributeError):
        refused_call(object())


def outputs(c, lay):
    part = ob.Partials.empty(lay, c.B, 3)
    out, lse = torch.empty(c.dq.shape, device="cuda"), torch.empty(c.dq.shape[:2], device="cuda")
    ob.oscar_decode_attention_int4(lay, *c.attention_args()[1:], part, None, out, lse)
    return out


@pytest.mark.gpu
def test_copies_outlive_the_original():
    c = ic.Cache([700, 400], n_kv=5, gqa=4, page=64, group=32, seed=1).upload()
    want = outputs(c, c.L)
    for make in (copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        first = ob.Layout(5, 4, 64, 32)
        assert torch.equal(outputs(c, first), want)
        twin = make(first)
        del first
        gc.collect()
        others = [ob.Layout(1, 1, 16) for _ in range(100)]
        for o in others[:10]:                                   # other layouts used in between
            ob.oscar_demote_int4(o, ob.Bf16Pool.empty(o, 1), torch.zeros((1, 1), dtype=torch.int32, device="cuda"), ob.Int4Pool.empty(o, 1),
                                 *(torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), 1, 1)))
        assert torch.equal(outputs(c, twin), want)
    assert ob.oscar_get_device_status() == 0


@pytest.mark.gpu
def test_threads_share_a_new_layout():
    c = ic.Cache([500], n_kv=2, gqa=4, page=16, seed=2).upload()
    want = outputs(c, c.L)
    for _ in range(20):
        lay, got, gate = ob.Layout(2, 4, 16), [None] * 4, threading.Barrier(4)

        def work(i):
            gate.wait()
            got[i] = outputs(c, lay)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        assert all(g is not None and torch.equal(g, want) for g in got)
    assert np.isfinite(want.cpu().numpy()).all() and ob.oscar_get_device_status() == 0
