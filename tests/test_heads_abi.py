"""Refusals of csa2_qk_norm_rope, csa2_paged_read and csa2_paged_chunk_attn: argument errors are found on
the host, before anything is launched (no GPU is touched here)."""
import ctypes
import os
import types

import pytest
import torch

import csa2_compressed_sparse_gb300 as csa2
from test_paged_abi import BAD_CACHES, cache
from test_paged_binding import On

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


# ---- tensors of another device than the cache's (nothing is called) --------------------------

@pytest.fixture
def recorded(monkeypatch):
    seen = []
    monkeypatch.setattr(csa2, "_call", lambda fn, dev, stream, *args: seen.append((fn, dev)))
    table = torch.empty((2, 8), dtype=torch.int32, device="meta")
    data = torch.empty((16, 64, 512), dtype=torch.bfloat16, device="meta")
    fake = types.SimpleNamespace(_dev=1, table=table, data=data, c=lambda: None, _c=types.SimpleNamespace(B=2))
    return fake, seen


def tensors(device, T=3, H=4):
    return dict(q=On.of(device, T, H, 512, dtype=torch.bfloat16), cu_seqlens=On.of(device, 3, dtype=torch.int32),
                start_pos=On.of(device, 2, dtype=torch.int64), out=On.of(device, T, H, 512, dtype=torch.bfloat16),
                ws=On.of(device, 1024), sink=On.of(device, H, dtype=torch.float32),
                lse=On.of(device, T, H, dtype=torch.float32), inv_freq=On.of(device, 32, dtype=torch.float32))


def test_the_caches_device_is_called(recorded):
    fake, seen = recorded
    csa2.csa2_paged_chunk_attn(cache=fake, **tensors(1))
    csa2.csa2_paged_read(On.of(1, 5, 512, dtype=torch.bfloat16), tensors(1)["cu_seqlens"], tensors(1)["start_pos"],
                         fake)
    assert [d for _, d in seen] == [1, 1]


@pytest.mark.parametrize("name", ["q", "cu_seqlens", "start_pos", "out", "ws", "sink", "lse", "inv_freq"])
@pytest.mark.parametrize("device", [-1, 0])
def test_chunk_tensors_elsewhere_are_refused(recorded, name, device):
    with pytest.raises(ValueError, match=name):
        csa2.csa2_paged_chunk_attn(cache=recorded[0], **{**tensors(1), name: tensors(device)[name]})
    assert not recorded[1]


@pytest.mark.parametrize("name,shape,dtype", [
    ("q", (3, 512), torch.bfloat16), ("q", (3, 4, 256), torch.bfloat16), ("q", (3, 4, 512), torch.float16),
    ("out", (2, 4, 512), torch.bfloat16), ("cu_seqlens", (2,), torch.int32), ("cu_seqlens", (3,), torch.int64),
    ("start_pos", (2,), torch.int32), ("lse", (3, 5), torch.float32), ("sink", (5,), torch.float32),
    ("inv_freq", (31,), torch.float32),
])
def test_chunk_shapes_are_refused(recorded, name, shape, dtype):
    with pytest.raises(ValueError, match=name):
        csa2.csa2_paged_chunk_attn(cache=recorded[0], **{**tensors(1), name: On.of(1, *shape, dtype=dtype)})
    assert not recorded[1]


@pytest.mark.parametrize("name,t", [
    ("out", On.of(0, 5, 512, dtype=torch.bfloat16)), ("out", On.of(1, 5, 256, dtype=torch.bfloat16)),
    ("out", On.of(1, 5, 512, dtype=torch.float32)), ("cu_seqlens", On.of(-1, 3, dtype=torch.int32)),
    ("cu_seqlens", On.of(1, 2, dtype=torch.int32)), ("start_row", On.of(0, 2, dtype=torch.int64)),
    ("start_row", On.of(1, 3, dtype=torch.int64)), ("inv_freq", On.of(0, 32, dtype=torch.float32)),
])
def test_read_tensors_are_refused(recorded, name, t):
    a = dict(out=On.of(1, 5, 512, dtype=torch.bfloat16), cu_seqlens=On.of(1, 3, dtype=torch.int32),
             start_row=On.of(1, 2, dtype=torch.int64), inv_freq=On.of(1, 32, dtype=torch.float32))
    with pytest.raises(ValueError, match=name):
        csa2.csa2_paged_read(cache=recorded[0], **{**a, name: t})
    assert not recorded[1]


@pytest.mark.parametrize("name", ["q_out", "pos", "inv_freq", "k", "k_out", "q_norm_w", "k_norm_w"])
@pytest.mark.parametrize("device", [-1, 0])
def test_head_tensors_elsewhere_are_refused(recorded, name, device):
    def all_on(d):
        a = {n: On.of(d, 3, h, 128, dtype=torch.bfloat16) for n, h in
             (("q", 4), ("q_out", 4), ("k", 2), ("k_out", 2))}
        return {**a, "pos": On.of(d, 3, dtype=torch.int64), "inv_freq": On.of(d, 16, dtype=torch.float32),
                "q_norm_w": On.of(d, 128, dtype=torch.float32), "k_norm_w": On.of(d, 128, dtype=torch.float32)}
    csa2.csa2_qk_norm_rope(**all_on(1))
    assert len(recorded[1]) == 1
    with pytest.raises(ValueError, match=name.replace("_out", "")):
        csa2.csa2_qk_norm_rope(**{**all_on(1), name: all_on(device)[name]})
    assert len(recorded[1]) == 1


def test_norm_rope_lets_no_kernel_start_before_it_ends():
    """The sparse step reads queries and window rows before its dependency wait; the header says that it may
    follow csa2_qk_norm_rope directly, so that kernel must not trigger its dependents."""
    src = os.path.join(os.path.dirname(csa2.__file__), "csrc", "k_heads.cu")
    with open(src) as f:
        assert "griddep_launch_dependents" not in f.read()


def test_the_search_for_a_sequence_does_not_read_around_the_dependency_wait():
    """Its array may be written by the kernel in front while the reader is resident: no read-only loads."""
    src = os.path.join(os.path.dirname(csa2.__file__), "csrc", "compress_dev.cuh")
    with open(src) as f:
        body = f.read().split("warp_find_seq(")[1].split("\n}")[0]
    assert "cu[probe]" in body and "__ldg" not in body


# ---- outputs whose rows overlap: D = 64 ------------------------------------------------------

def overlaps(T, H, token, head, D=64):
    """By the definition: two rows, of D elements each, that share one."""
    at = sorted(t * token + h * head for t in range(T) for h in range(H))
    return any(b - a < D for a, b in zip(at, at[1:]))


STRIDES = [0, 8, 56, 64, 72, 96, 128, 136, 192, 256, 320, 328, 384, 448, 512, 640, 1024, 1 << 40]


@pytest.mark.parametrize("T", [1, 2, 3, 7, 20])
@pytest.mark.parametrize("H", [1, 2, 3, 6])
def test_overlapping_outputs_are_refused(T, H):
    """The odd pointer comes after the overlap in the order of the checks: nothing is ever launched here."""
    for token in STRIDES:
        for head in STRIDES:
            h = heads(H=H, x_token=64 * H, x_head=64, out_token=token, out_head=head, norm_w=4100)
            st, msg = norm_rope(q=h, T=T, D=64, r0=0, R=64)
            assert st == 1 and (b"overlap" in msg) == overlaps(T, H, token, head), (token, head, msg)


@pytest.mark.parametrize("token,head,bad", [
    (512, 512, True), (512, 520, True), (32768, 512, False), (512, 1 << 62, False), (1 << 62, 512, False),
    ((1 << 62) + 8, (1 << 62), True), (1 << 62, 1 << 62, True)])
def test_overlaps_of_the_widest_strides(token, head, bad):
    st, msg = norm_rope(q=heads(out_token=token, out_head=head, norm_w=4100), T=1 << 20)
    assert st == 1 and (b"overlap" in msg) == bad


# ---- keys alone, through the binding ---------------------------------------------------------

def test_the_binding_takes_keys_alone(monkeypatch):
    seen = []
    monkeypatch.setattr(csa2, "_call", lambda fn, dev, stream, q, k, *args: seen.append((dev, q, k._obj.H, *args)))
    a = dict(pos=On.of(1, 3, dtype=torch.int64), inv_freq=On.of(1, 16, dtype=torch.float32),
             k=On.of(1, 3, 2, 128, dtype=torch.bfloat16), k_out=On.of(1, 3, 2, 128, dtype=torch.bfloat16))
    csa2.csa2_qk_norm_rope(None, None, **a)
    assert seen[0][:5] == (1, None, 2, 3, 128)
    for kw, word in ((dict(k=None, k_out=None), "q or k"), (dict(q_out=a["k"]), "q is missing"),
                     (dict(q_norm_w=On.of(1, 128, dtype=torch.float32)), "q is missing"), (dict(k_out=None), "k and k_out"),
                     (dict(k=On.of(1, 3, 128, dtype=torch.bfloat16)), "k must be"),
                     (dict(k_out=On.of(0, 3, 2, 128, dtype=torch.bfloat16)), "cuda:1")):
        with pytest.raises(ValueError, match=word):
            csa2.csa2_qk_norm_rope(None, **{"q_out": None, **a, **kw})
    assert len(seen) == 1
