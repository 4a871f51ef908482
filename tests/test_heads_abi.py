"""Refusals of csa2_qk_norm_rope, csa2_paged_read and csa2_paged_chunk_attn: argument errors are found on
the host, before anything is launched (no GPU is touched here)."""
import ctypes

import pytest
import torch

import csa2_compressed_sparse_gb300 as csa2
from test_paged_abi import BAD_CACHES, cache

P = ctypes.c_void_p(4096)


def heads(**kw):
    a = dict(x=4096, out=4096, x_token=32768, x_head=512, out_token=32768, out_head=512, H=64, norm=1,
             norm_w=4096)
    a.update(kw)
    return csa2._HeadsC(*a.values())


def norm_rope(q=heads(), k=None, **kw):
    L = csa2.lib()
    a = dict(q=ctypes.byref(q) if q else None, k=ctypes.byref(k) if k else None, T=4, D=512, eps=1e-6, pos=P,
             inv_freq=P, r0=448, R=64, layout=0, factor=1.0, stream=None)
    a.update(kw)
    return L.csa2_qk_norm_rope(*a.values()), L.csa2_last_error()


def read(c=None, **kw):
    L = csa2.lib()
    a = dict(out=P, out_ld=512, T=4, cu=P, start=P, ratio=1, cache=ctypes.byref(c or cache()),
             inv_freq=P, stream=None)
    a.update(kw)
    return L.csa2_paged_read(*a.values()), L.csa2_last_error()


def chunk(c=None, **kw):
    L = csa2.lib()
    a = dict(q=P, T=4, H=64, cu=P, start=P, cache=ctypes.byref(c or cache()), ratio=1, window=0,
             max_rows=512, total_rows=1024, sink=None, scale=0.04, out=P, lse=None, inv_freq=None, ws=P,
             ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return L.csa2_paged_chunk_attn(*a.values()), L.csa2_last_error()


ODD = ctypes.c_void_p(4104)


@pytest.mark.parametrize("call", [read, chunk])
@pytest.mark.parametrize("kw,word", BAD_CACHES)
def test_bad_caches_are_refused(call, kw, word):
    st, msg = call(cache(**kw))
    assert st == 1 and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T must"), (dict(out=None), b"required"), (dict(cu=None), b"required"),
    (dict(start=None), b"required"), (dict(out=ODD), b"aligned"), (dict(out_ld=504), b"out_ld"),
    (dict(out_ld=516), b"out_ld"), (dict(ratio=0), b"ratio"), (dict(ratio=65537), b"ratio"),
    (dict(cache=None), b"cache"), (dict(cu=ctypes.c_void_p(4098)), b"aligned"),
    (dict(start=ctypes.c_void_p(4100)), b"aligned"), (dict(inv_freq=ctypes.c_void_p(4098)), b"aligned"),
])
def test_read_refusals(kw, word):
    st, msg = read(**kw)
    assert st == 1 and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T must"), (dict(T=1048577), b"T must"), (dict(H=0), b"H must"), (dict(H=129), b"H must"),
    (dict(q=None), b"required"), (dict(cu=None), b"required"), (dict(start=None), b"required"),
    (dict(out=None), b"required"), (dict(q=ODD), b"aligned"), (dict(out=ODD), b"aligned"),
    (dict(ratio=0), b"ratio"), (dict(ratio=65537), b"ratio"), (dict(window=-1), b"window"),
    (dict(max_rows=-1), b"max_rows"), (dict(max_rows=1 << 31), b"max_rows"),
    (dict(total_rows=-1), b"total_rows"), (dict(total_rows=1 << 31), b"total_rows"),
    (dict(scale=float("nan")), b"scale"), (dict(scale=float("inf")), b"scale"),
    (dict(ws=ODD), b"256-byte"), (dict(cache=None), b"cache"),
    (dict(cu=ctypes.c_void_p(4098)), b"aligned"), (dict(start=ctypes.c_void_p(4100)), b"aligned"),
    (dict(sink=ctypes.c_void_p(4098)), b"aligned"), (dict(lse=ctypes.c_void_p(4098)), b"aligned"),
    (dict(inv_freq=ctypes.c_void_p(4098)), b"aligned"),
])
def test_chunk_refusals(kw, word):
    st, msg = chunk(**kw)
    assert st == 1 and word in msg


def test_chunk_workspace_size_and_its_check():
    c = cache()
    size = lambda T, H, rows, total, c=c: csa2.lib().csa2_paged_chunk_attn_workspace_size(
        T, H, ctypes.byref(c) if c else None, rows, total)
    need = size(4, 64, 512, 1024)
    assert need > 0
    for kw in (dict(ws_bytes=need - 1), dict(ws=None, ws_bytes=0)):
        st, msg = chunk(**kw)
        assert st == 5 and b"workspace" in msg
    assert size(0, 64, 512, 1024) == 0
    for bad in ((-1, 64, 512, 9), (1048577, 64, 512, 9), (1, 0, 512, 9), (1, 129, 512, 9), (1, 64, -1, 9),
                (1, 64, 1 << 31, 9), (1, 64, 512, -1), (1, 64, 512, 9, None)):
        assert size(*bad) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"T must"), (dict(q=None), b"q or k"), (dict(D=0), b"D must"), (dict(D=516), b"D must"),
    (dict(D=520), b"D must"), (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"),
    (dict(pos=None), b"required"), (dict(inv_freq=None), b"required"), (dict(r0=-8), b"rope_dim0"),
    (dict(r0=444), b"rope_dim0"), (dict(r0=456), b"rope_dim0"), (dict(R=-8), b"rope_dim0"),
    (dict(R=60), b"rope_dim0"), (dict(R=1 << 30), b"rope_dim0"), (dict(r0=(1 << 31) - 8), b"rope_dim0"),
    (dict(layout=2), b"layout"), (dict(layout=1, R=56), b"multiple of 16"),
    (dict(factor=float("inf")), b"factor"), (dict(pos=ctypes.c_void_p(4100)), b"aligned"),
    (dict(inv_freq=ctypes.c_void_p(4098)), b"aligned"),
])
def test_norm_rope_refusals(kw, word):
    st, msg = norm_rope(**kw)
    assert st == 1 and word in msg


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("kw,word", [
    (dict(H=0), b".H must"), (dict(H=1025), b".H must"), (dict(x=None), b"required"),
    (dict(out=None), b"required"), (dict(x=4104), b"aligned"), (dict(out=4104), b"aligned"),
    (dict(x_token=4), b"strides"), (dict(x_head=516), b"strides"), (dict(out_token=-8), b"strides"),
    (dict(out_head=508), b"strides"), (dict(out_head=504), b"overlap"), (dict(out_token=0), b"overlap"),
    (dict(norm_w=4100), b"norm_w"),
])
def test_head_refusals(which, kw, word):
    st, msg = norm_rope(**{which: heads(**kw)})
    assert st == 1 and word in msg and which.encode() in msg


def test_nothing_to_do_is_not_an_error():
    assert read(T=0, out=None, cache=None)[0] == 0
    assert chunk(T=0, q=None, cache=None)[0] == 0
    assert norm_rope(T=0, pos=None)[0] == 0


def test_the_binding_checks_its_tensors():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        csa2.csa2_qk_norm_rope(x, x, torch.zeros(2, dtype=torch.int64), torch.zeros(8))
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        csa2.csa2_qk_norm_rope(x[0], x[0], torch.zeros(2, dtype=torch.int64), torch.zeros(8))
