"""Arrays that are not aligned to their elements are refused on the host: the kernels would fault on
them.  (No GPU is touched here.)"""
import ctypes

import pytest

from test_paged_abi import append, attn, cache


def at(address):
    return ctypes.c_void_p(address)


@pytest.mark.parametrize("call", [append, attn])
def test_a_misaligned_table_is_refused(call):
    st, msg = call(cache(table=4098))
    assert st == 1 and b"table" in msg


@pytest.mark.parametrize("kw", [dict(cu=at(4098)), dict(start=at(4100)), dict(inv_freq=at(4097))])
def test_append_refuses_misaligned_arrays(kw):
    st, msg = append(**kw)
    assert st == 1 and b"aligned to their elements" in msg


@pytest.mark.parametrize("kw", [dict(q_seq=at(4098)), dict(q_pos=at(4100)), dict(sink=at(4097)),
                                dict(lse=at(4102)), dict(inv_freq=at(4098))])
def test_attention_refuses_misaligned_arrays(kw):
    st, msg = attn(**kw)
    assert st == 1 and b"aligned to their elements" in msg


def test_arrays_at_any_element_are_taken():
    """Slices that begin at any element pass these checks: the refusals that are met here come
    after them."""
    st, msg = append(cache(table=4100), cu=at(4100), start=at(4104), inv_freq=at(4108), ratio=0)
    assert st == 1 and b"ratio" in msg
    st, msg = attn(cache(table=4100), q_seq=at(4100), q_pos=at(4104), sink=at(4108), lse=at(4100),
                   inv_freq=at(4100), ratio=0)
    assert st == 1 and b"ratio" in msg
