"""Refusals of the paged cache's entry points: argument errors are found on the host, before
anything is launched (no GPU is touched here)."""
import ctypes

import pytest
import torch

import csa2_compressed_sparse_gb300 as csa2

P = ctypes.c_void_p(4096)


def cache(**kw):
    a = dict(dtype=0, page_rows=64, data=4096, n_pages=10, page_stride=65536, table=4096, B=2,
             table_ld=8, table_cols=8)
    a.update(kw)
    return csa2._PagedC(*a.values())


def append(c=None, **kw):
    L = csa2.lib()
    a = dict(kv=P, kv_ld=512, T=4, cu=P, start=P, ratio=1, cache=ctypes.byref(c or cache()),
             inv_freq=P, stream=None)
    a.update(kw)
    return L.csa2_paged_append(*a.values()), L.csa2_last_error()


def attn(c=None, **kw):
    L = csa2.lib()
    a = dict(q=P, Q=2, H=64, q_seq=P, q_pos=P, cache=ctypes.byref(c or cache()), ratio=1, window=0,
             max_rows=512, sink=None, scale=0.04, out=P, lse=None, inv_freq=None, ws=P,
             ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return L.csa2_paged_attn(*a.values()), L.csa2_last_error()


BAD_CACHES = [
    (dict(dtype=3), b"dtype"), (dict(dtype=-1), b"dtype"),
    (dict(page_rows=0), b"page_rows"), (dict(page_rows=12), b"page_rows"),
    (dict(page_rows=65544, page_stride=1 << 30), b"page_rows"),
    (dict(data=None), b"data"), (dict(data=4104), b"data"),
    (dict(n_pages=0), b"n_pages"), (dict(n_pages=1 << 31), b"n_pages"),
    (dict(page_stride=65520), b"page_stride"), (dict(page_stride=65544), b"page_stride"),
    (dict(page_stride=1 << 40), b"page_stride"),
    (dict(dtype=1, page_stride=64 * 528 - 16), b"page_stride"),
    (dict(B=0), b"cache.B"), (dict(B=65536), b"cache.B"), (dict(table=None), b"table"),
    (dict(table_cols=0), b"table_cols"), (dict(table_ld=7), b"table_cols"),
]


@pytest.mark.parametrize("call", [append, attn])
@pytest.mark.parametrize("kw,word", BAD_CACHES)
def test_bad_caches_are_refused(call, kw, word):
    st, msg = call(cache(**kw))
    assert st == 1 and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T must"), (dict(kv=None), b"required"), (dict(cu=None), b"required"),
    (dict(start=None), b"required"), (dict(kv=ctypes.c_void_p(4104)), b"aligned"),
    (dict(kv_ld=504), b"kv_ld"), (dict(kv_ld=516), b"kv_ld"), (dict(ratio=0), b"ratio"),
    (dict(ratio=65537), b"ratio"), (dict(cache=None), b"cache"),
])
def test_append_refusals(kw, word):
    st, msg = append(**kw)
    assert st == 1 and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(Q=-1), b"Q must"), (dict(Q=65536), b"Q must"), (dict(H=0), b"H must"),
    (dict(H=129), b"H must"), (dict(q=None), b"required"), (dict(q_seq=None), b"required"),
    (dict(q_pos=None), b"required"), (dict(out=None), b"required"),
    (dict(q=ctypes.c_void_p(4104)), b"aligned"), (dict(out=ctypes.c_void_p(4104)), b"aligned"),
    (dict(ratio=0), b"ratio"), (dict(window=-1), b"window"), (dict(max_rows=-1), b"max_rows"),
    (dict(max_rows=1 << 31), b"max_rows"), (dict(scale=float("nan")), b"scale"),
    (dict(scale=float("inf")), b"scale"), (dict(ws=ctypes.c_void_p(4100)), b"256-byte"),
    (dict(cache=None), b"cache"),
])
def test_attn_refusals(kw, word):
    st, msg = attn(**kw)
    assert st == 1 and word in msg


def test_nothing_to_do_is_not_an_error():
    assert append(T=0, kv=None, cache=None)[0] == 0
    assert attn(Q=0, q=None, cache=None)[0] == 0


def test_workspace_size_and_its_check():
    size = csa2.csa2_paged_attn_workspace_size
    need = size(2, 64, 512)
    assert need > 0
    st, msg = attn(ws_bytes=need - 1)
    assert st == 5 and b"workspace" in msg
    st, msg = attn(ws=None, ws_bytes=0)
    assert st == 5 and b"workspace" in msg
    # at most two partial results per CTA, whatever the batch; items of one unit need none
    assert size(1, 64, 256) == 0 and size(4096, 128, 256) == 0
    assert size(64, 64, 1 << 20) <= 152 * 2 * 64 * (512 + 3) * 4 + 64 * 8 + 768
    assert size(1, 16, 1 << 20) < size(1, 64, 1 << 20)
    assert size(0, 64, 512) == 0
    for bad in ((-1, 64, 512), (65536, 64, 512), (1, 0, 512), (1, 129, 512), (1, 64, -1),
                (1, 64, 1 << 31)):
        assert size(*bad) == 0


def test_the_binding_checks_the_cache():
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        csa2.Paged(torch.zeros((4, 8, 512), dtype=torch.bfloat16), t)
    with pytest.raises(ValueError, match="paged cache"):
        csa2.Paged(torch.zeros((4, 8, 512)), t)
    with pytest.raises(ValueError, match="paged cache"):
        csa2.Paged(torch.zeros((4, 8, 520), dtype=torch.uint8), t)
    with pytest.raises(ValueError, match="table"):
        csa2.Paged(torch.zeros((4, 8, 512), dtype=torch.bfloat16), t.long())
