"""Calls from a thread that has made no CUDA call before."""
import threading

import pytest
import torch

from bit_kv_cache_oscar_gb300 import binding as ob
from tests import int4_case as ic
from tests import scenario as sc

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    error = []

    def work():
        try:
            f()
        except Exception as e:
            error.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if error:
        raise error[0]


@pytest.mark.parametrize("page", [16, 64])
def test_int4_calls_are_a_thread_s_first(page):
    c = ic.Cache([700, 330], n_kv=2, gqa=4, page=page, seed=1).upload()
    out = [torch.empty(c.dq.shape, device="cuda") for _ in range(2)]
    lse = [torch.empty(c.dq.shape[:2], device="cuda") for _ in range(2)]
    mass = [torch.zeros((2, 2, c.max_pages * page), device="cuda") for _ in range(2)]
    part = [ob.Partials.empty(c.L, 2, 3) for _ in range(2)]
    stream = torch.cuda.current_stream()
    decode = lambda i: ob.oscar_decode_attention_int4(*c.attention_args(), part[i], None, out[i], lse[i], stream=stream)
    weigh = lambda i: ob.oscar_attention_mass_int4(*c.attention_args(), lse[i], mass[i], stream)
    decode(0), weigh(0)                                 # what a process sets up once is set up
    in_a_new_thread(lambda: decode(1))
    in_a_new_thread(lambda: weigh(1))
    torch.cuda.synchronize()
    assert torch.equal(*out) and torch.equal(*lse) and torch.equal(*mass)
    assert ob.oscar_get_device_status() == 0


def test_the_two_bit_decode_too():
    case = sc.make_case(n_kv=8, gqa=4, page_size=64, seq=(1024,))
    dev, L = sc.upload(case), case.layout
    q = dev["q"]
    part = [ob.Partials.empty(L, 1, 4) for _ in range(2)]
    out = [torch.empty(q.shape, device="cuda") for _ in range(2)]
    stream = torch.cuda.current_stream()
    call = lambda i: ob.oscar_decode_attention_fused(L, q, dev["RK"], dev["bf16"], dev["bf16_table"], dev["int2"], dev["int2_table"], dev["seq_len"],
                                                     dev["hist_end"], case.sm_scale, part[i], R_V=dev["RV"], out_f32=out[i], stream=stream)
    call(0)
    in_a_new_thread(lambda: call(1))
    torch.cuda.synchronize()
    assert torch.equal(*out) and torch.isfinite(out[0]).all()
