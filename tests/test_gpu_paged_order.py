"""The paged cache's calls behind other kernels of the stream.

Every kernel of the library lets the next one start while it drains, so what a call is given may
still be under way when its kernel begins.  Each chain here is run twice: call after call, and
with the stream drained between the calls; a call's results depend on its inputs alone, to the
bit (no atomics, a fixed order of sums), so both have to be equal to the bit.  What the buffers
hold before (other rows, other pages, all of them valid) is no answer of the chain.
"""
import numpy as np
import pytest
import torch

from test_gpu_paged import BF16, DTYPES, check_query, decode, get, inv_freq, paged, pool, put
from test_gpu_paged import quantised, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# one CTA an item, clusters, items split over the GPU and joined
PATHS = {"whole": [200, 17, 256], "clusters": [1800, 5, 700], "split": [9000, 40, 3000]}


def cache_of(dtype, lens, page, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    data, table, _ = pool(np.random.default_rng(seed), dtype, page, lens)
    for b, n in enumerate(lens):
        put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    return data, table, g


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_the_output_of_a_call_is_the_query_of_the_next(dtype, path):
    import csa2_compressed_sparse_gb300 as csa2
    lens = PATHS[path]
    data, table, g = cache_of(dtype, lens, 64, 5)
    B, H, n = len(lens), 64, 8
    seq = torch.arange(B, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lens, device="cuda") - 1
    ws = workspace(B, H, max(lens))
    c = paged(data, table, dtype)
    f = inv_freq().cuda()
    q0 = torch.randn((B, H, 512), generator=g, device="cuda").bfloat16()
    stale = torch.randn((n, B, H, 512), generator=g, device="cuda").bfloat16()

    def chain(drain):
        outs, lses = stale.clone(), torch.zeros((n, B, H), device="cuda")
        torch.cuda.synchronize()
        q = q0
        for i in range(n):
            # the scale keeps the scores of an output, a mean of rows, as spread as the first ones
            csa2.csa2_paged_attn(q, seq, pos, c, outs[i], ws, max_rows=max(lens), lse=lses[i],
                                 scale=0.5, inv_freq=f)
            q = outs[i]
            if drain:
                csa2.csa2_device_status()
        csa2.csa2_device_status()
        return outs, lses

    ref = chain(True)
    for i, q in enumerate([q0] + list(ref[0][:1])):  # the drained chain, against the formula
        for b, m in enumerate(lens):
            check_query(ref[0][i, b], ref[1][i, b], q[b], decode(get(data, table, b, 0, m), dtype),
                        None, 0.5, m - 1, True)
    for _ in range(3):
        got = chain(False)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_a_page_table_written_by_the_kernel_before(dtype, path):
    """A top-k whose row ids are the pages of the call behind it."""
    import csa2_compressed_sparse_gb300 as csa2
    lens = PATHS[path]
    page, H, B = 64, 64, len(lens)
    k = -(-max(lens) // page)  # pages of a table row: all sequences have as many
    data, _, g = cache_of(dtype, [B * k * page], page, 6)
    pages = data.shape[0]
    spare = torch.randn((pages * page, 512), generator=g, device="cuda")
    data.copy_(quantised(spare, dtype).reshape(data.shape))  # every page, no NaN left
    rng = np.random.default_rng(7)
    scores = torch.zeros((B, pages), device="cuda")
    want = np.sort(np.stack([rng.permutation(pages)[:k] for _ in range(B)]), axis=1)
    for b in range(B):
        scores[b, torch.tensor(want[b], device="cuda")] = 1.0 + torch.rand(k, generator=g, device="cuda")
    n = torch.full((B,), pages, dtype=torch.int32, device="cuda")
    seq = torch.arange(B, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lens, device="cuda") - 1
    q = torch.randn((B, H, 512), generator=g, device="cuda").bfloat16()
    ws = workspace(B, H, max(lens))
    res = []
    for drain in (True, False, False, False):
        table = torch.zeros((B, k), dtype=torch.int32, device="cuda")  # page 0 is a page, too
        out, lse = torch.zeros_like(q), torch.zeros((B, H), device="cuda")
        torch.cuda.synchronize()
        csa2.csa2_topk_scores(scores, n, k, table)
        if drain:
            csa2.csa2_device_status()
        csa2.csa2_paged_attn(q, seq, pos, paged(data, table, dtype), out, ws, max_rows=max(lens),
                             lse=lse)
        csa2.csa2_device_status()
        assert torch.equal(table.cpu(), torch.tensor(want, dtype=torch.int32))
        res.append((out, lse))
    for b, m in enumerate(lens):
        check_query(res[0][0][b], res[0][1][b], q[b], decode(get(data, table, b, 0, m), dtype), None,
                    512 ** -0.5, m - 1, False)
    for out, lse in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(lse, res[0][1])
