"""Tables and arrays without rows whose other side passes 32 bits: refused like any other argument."""
import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob

pytestmark = pytest.mark.gpu
BIG = 1 << 31


def ints(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def test_sizes_above_32_bits_are_refused():
    L = ob.Layout(2, 4, 16)
    bf, i4 = ob.Bf16Pool.empty(L, 2), ob.Int4Pool.empty(L, 2)
    wide, none = ints(0, BIG), ints(0)
    floats = lambda *s: torch.empty(s, device="cuda")
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    part = ob.Partials.empty(L, 0, 2)
    mass = floats(0, 2, BIG * 16)
    kv = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ob.oscar_demote_int4(L, bf, wide, i4, wide, none, none),
                 lambda: ob.oscar_promote_int4(L, i4, wide, bf, wide, none, none),
                 lambda: ob.oscar_append_kv(L, None, kv, kv, bf, wide, none, none),
                 lambda: ob.oscar_decode_attention_int4(L, q, bf, wide, i4, wide, none, none, 1.0, part),
                 lambda: ob.oscar_attention_mass_int4(L, q, bf, wide, i4, wide, none, none, 1.0, floats(0, 8), mass),
                 lambda: ob.oscar_evict_int4(L, i4, wide, i4, ints(0, BIG), none, none, none, mass, floats(0, 2, BIG * 16), ints(0, 2, 1)),
                 lambda: ob.oscar_evict_int4(L, i4, ints(0, 4), i4, ints(0, 4), none, none, none, floats(0, 2, 64), floats(0, 2, 64), ints(0, 2, BIG))):
        with pytest.raises(ob.OscarError, match="more than 2.31 - 1"):
            call()
    ob.oscar_demote_int4(L, bf, ints(0, 4), i4, ints(0, 4), none, none)            # no requests, nothing to do
    with pytest.raises(ob.OscarError, match="max_pages_per_req"):                  # the library's own refusal
        ob.oscar_demote_int4(L, bf, ints(0, BIG - 1), i4, ints(0, BIG - 1), none, none)


def test_a_refused_call_leaves_the_thread_as_it_was():
    L = ob.Layout(1, 1, 16)
    bf, i4, none = ob.Bf16Pool.empty(L, 2), ob.Int4Pool.empty(L, 2), ints(0)
    for _ in range(100):
        with pytest.raises(ob.OscarError):
            ob.oscar_promote_int4(L, i4, ints(0, BIG), bf, ints(0, BIG), none, none)
    assert ob.oscar_get_device_status() == 0
