"""Chunk attention behind other kernels of the stream: calls in a row that share what they may share.

Tolerances as in test_gpu_chunk.py; runs with the stream drained between the calls are equal to the bit."""
import pytest
import torch

from test_gpu_chunk import Case, status
from test_gpu_paged import BF16, DTYPES, E8M0, S128, put, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("dtype,page", [(S128, 64), (E8M0, 16), (BF16, 8)])
def test_copied_rows_of_calls_in_a_row(dtype, page):
    """Sequences of other numbers and lengths from call to call: the places of the copied rows, which one
    workspace holds for all of the calls, are others each time."""
    shapes = [([30, 2, 41], [900, 0, 77]), ([7] * 40, [20 * i for i in range(40)]), ([200], [1]),
              ([1, 0, 130], [2000, 5, 300]), ([3] * 5, [40, 1000, 0, 333, 64])]
    cases = [Case(60 + i, dtype, 64, page, new, hist) for i, (new, hist) in enumerate(shapes)]
    ws = max((c.ws for c in cases), key=lambda w: w.numel())
    first = []
    for c in cases:
        c.call().check()
        first.append((c.out.clone(), c.lse.clone()))
    for _ in range(4):
        for c in cases:
            c.out.fill_(5)
            c.lse.fill_(6)
        torch.cuda.synchronize()
        for c in cases:
            c.call(ws=ws)
        assert status() == 0
        for c, (out, lse) in zip(cases, first):
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,hist", [([40, 9, 128], [700, 1500, 0]), ([6] * 90, [300] * 90), ([3], [30000])])
def test_maxima_that_move_in_every_key_tile(dtype, new, hist):
    """Each key tile rescales what the tensor memory holds, and segments end while others begin: the warps
    that hand a block of weights on are not those that rescaled or read all of it."""
    c = Case(70, dtype, 64, 64, new, hist)
    g = torch.Generator(device="cuda").manual_seed(70)
    x = torch.randn((1, 512), generator=g, device="cuda")
    c.q.copy_((x * (1 + 0.1 * torch.rand((c.T, 64, 1), generator=g, device="cuda"))).bfloat16())
    for b, n in enumerate(c.rows):
        top = 6.0 * -(-n // 256)  # scores of some 130 more from tile to tile: beyond 2^64 of a weight
        r = x * torch.linspace(0, top, n, device="cuda")[:, None] + torch.randn((n, 512), generator=g, device="cuda")
        put(c.data, c.table, b, quantised(r, dtype))
    c.call().check(only=[0, 1, 2, 5, 31, 39, 64, 127])
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(6):
        c.out.fill_(5)
        c.lse.fill_(6)
        c.call()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert status() == 0
