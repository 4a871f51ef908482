"""The paged cache's binding refuses tensors of another device before anything is called.  No GPU
is needed: tensors of the meta device stand in, with a GPU's index as their own."""
import types

import pytest
import torch

import csa2_compressed_sparse_gb300 as csa2


class On(torch.Tensor):
    """A tensor without memory that says which GPU it is on (-1: the CPU)."""
    @staticmethod
    def of(device, *shape, dtype=torch.uint8):
        t = torch.empty(shape, dtype=dtype, device="meta").as_subclass(On)
        t.index = device
        return t

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 4096


@pytest.fixture
def call(monkeypatch):
    """csa2_paged_attn with a cache on GPU 1; the library's call is recorded, not made."""
    seen = []
    monkeypatch.setattr(csa2, "_call", lambda fn, dev, stream, *args: seen.append(args))
    table = torch.empty((2, 8), dtype=torch.int32, device="meta")
    data = torch.empty((16, 64, 512), dtype=torch.bfloat16, device="meta")
    cache = types.SimpleNamespace(_dev=1, table=table, data=data, c=lambda: None)

    def attn(**kw):
        a = dict(q=On.of(1, 2, 64, 512, dtype=torch.bfloat16),
                 q_seq=On.of(1, 2, dtype=torch.int32), q_pos=On.of(1, 2, dtype=torch.int64),
                 cache=cache, out=On.of(1, 2, 64, 512, dtype=torch.bfloat16))
        csa2.csa2_paged_attn(**{**a, **kw})
        return seen[-1]
    return attn


def test_a_workspace_of_the_caches_gpu_is_passed_on(call):
    assert call(ws=None)[-2:] == (None, 0)
    assert call(ws=On.of(1, 1024))[-2:] == (4096, 1024)
    assert call(ws=On.of(1, 256, dtype=torch.float32))[-2:] == (4096, 1024)


@pytest.mark.parametrize("device", [-1, 0, 2])
def test_a_workspace_elsewhere_is_refused(call, device):
    with pytest.raises(ValueError, match="ws must be"):
        call(ws=On.of(device, 1024))


def test_a_workspace_with_holes_is_refused(call):
    t = On.of(1, 64, 64)[:, ::2]
    t.index = 1
    with pytest.raises(ValueError, match="ws must be"):
        call(ws=t)


@pytest.mark.parametrize("name", ["q", "q_seq", "q_pos", "out"])
def test_every_other_tensor_elsewhere_is_refused(call, name):
    made = dict(q=((2, 64, 512), torch.bfloat16), q_seq=((2,), torch.int32),
                q_pos=((2,), torch.int64), out=((2, 64, 512), torch.bfloat16))
    shape, dtype = made[name]
    with pytest.raises(ValueError, match=name):
        call(**{name: On.of(0, *shape, dtype=dtype)})
