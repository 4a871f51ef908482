"""Chunk attention behind other kernels of the stream: calls in a row that share what they may share.

Tolerances as in test_gpu_chunk.py; runs with the stream drained between the calls are equal to the bit."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Case, check_tokens, status, workspace
from test_gpu_paged import BF16, DTYPES, E8M0, S128, decode, get, inv_freq, paged, pool, put, quantised

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


@pytest.mark.parametrize("dtype", DTYPES)
def test_layers_without_a_wait_between_their_calls(dtype):
    """Norm and rotation, append, attention, and the attention's outputs as the next layer's queries; then the
    rows read back.  Queries, latents and workspace are one buffer for all layers."""
    import csa2_compressed_sparse_gb300 as csa2
    L, H, new, hist, f = 5, 64, [60, 1, 130], [300, 1000, 0], inv_freq().cuda()
    T, rows = sum(new), [h + n for h, n in zip(hist, new)]
    g = torch.Generator(device="cuda").manual_seed(7)
    pools = [pool(np.random.default_rng(i), dtype, 64, rows, poison=False)[:2] for i in range(L)]
    for data, table in pools:
        for b, n in enumerate(rows):
            put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    start = [d.clone() for d, _ in pools]
    caches = [paged(d, t, dtype) for d, t in pools]
    x = torch.randn((L, T, 1, 512), generator=g, device="cuda").bfloat16()
    x0 = torch.randn((T, H, 512), generator=g, device="cuda").bfloat16()
    cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    at = torch.tensor(hist, device="cuda")
    pos = torch.cat([torch.arange(h, h + n, device="cuda") for h, n in zip(hist, new)])
    q, kv = torch.zeros_like(x0), torch.zeros((T, 1, 512), dtype=torch.bfloat16, device="cuda")
    w = 4 * torch.ones(512, device="cuda")
    ws = workspace(T, H, caches[0], max(rows), sum(rows))
    cu_all = torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device="cuda")
    zero = torch.zeros(3, dtype=torch.int64, device="cuda")

    def layers(outs, back, drain):
        for i in range(L):
            for call in (lambda: csa2.csa2_qk_norm_rope(outs[i - 1] if i else x0, q, pos, f, q_norm_w=w),
                         lambda: csa2.csa2_qk_norm_rope(None, None, pos, None, k=x[i], k_out=kv),
                         lambda: csa2.csa2_paged_append(kv[:, 0], cu, at, caches[i], inv_freq=f),
                         lambda: csa2.csa2_paged_chunk_attn(q, cu, at, caches[i], outs[i], ws, max_rows=max(rows),
                                                            total_rows=sum(rows), inv_freq=f),
                         lambda: csa2.csa2_paged_read(back[i], cu_all, zero, caches[i])):
                call()
                if drain:
                    assert status() == 0
            if drain:
                for b, n in enumerate(rows):
                    t = slice(int(cu[b]), int(cu[b + 1]))
                    p = pos[t]
                    check_tokens(outs[i][t], None, q[t], decode(get(*pools[i], b, 0, n), dtype), torch.zeros_like(p),
                                 p + 1, None, 512 ** -0.5, p, True, dtype)

    def run(how):
        outs = torch.zeros((L, T, H, 512), dtype=torch.bfloat16, device="cuda")
        back = torch.zeros((L, sum(rows), 512), dtype=torch.bfloat16, device="cuda")
        for (d, _), s in zip(pools, start):
            d.copy_(s)
        torch.cuda.synchronize()
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layers(outs, back, False)
            outs.zero_()
            graph.replay()
        else:
            layers(outs, back, how == "drained")
        assert status() == 0
        return outs, back

    ref = run("drained")
    for how in ("in a row", "in a row", "in a row", "graph", "graph"):
        got = run(how)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
