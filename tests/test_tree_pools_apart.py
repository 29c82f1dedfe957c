"""The pools whose rows oscar_tree_accept moves in one launch lie apart: arrays given twice or overlapping are refused, without a GPU."""
import pytest

from bit_kv_cache_oscar_gb300 import binding as ob
from tests.test_tree_validation import FAKE, INVALID, L, OK, accept, layout  # noqa: F401

PAGE = 64 * 8 * 128 * 2                                          # bytes of a page of layout()


def pool(k, v, n_pages=4):
    return ob.Bf16PoolC(FAKE + k, FAKE + v, n_pages)


A, B, C = 0, 4 * PAGE, 8 * PAGE


@pytest.mark.parametrize("pools", [
    [pool(A, A)], [pool(A, B), pool(A, B)], [pool(A, B), pool(B, A)], [pool(A, B), pool(C, 12 * PAGE), pool(16 * PAGE, B)],
    [pool(A, 4 * PAGE - 16)], [pool(C, B, 5)], [pool(A, B), pool(C, C + PAGE, 2)], [pool(2 ** 40, A, 1), pool(2 ** 40 + PAGE - 16, B, 1)]])
def test_arrays_that_share_memory_are_refused(L, pools):  # noqa: F811
    assert accept(L, pools=pools) == INVALID
    assert b"share memory" in L.oscar_last_error_string()


def test_no_requests_and_missing_arguments_come_first(L):  # noqa: F811
    assert accept(L, pools=[pool(A, A)], batch=0) == OK
    assert accept(L, pools=[pool(A, A)], target=None) == INVALID and b"NULL" in L.oscar_last_error_string()
