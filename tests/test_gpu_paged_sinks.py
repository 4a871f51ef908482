"""Sinks far from the scores: the running maximum starts at the sink's logit and has to find the
scores from there.  Formulas and tolerances as in test_gpu_paged.py: a sink of -1e9 or less has
no mass beside scores of hundreds, and none of these tolerances depends on the sink."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DTYPES, check_query, decode, get, inv_freq, paged, pool, put
from test_gpu_paged import quantised, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# one CTA an item, clusters, items split over the GPU and joined
PATHS = {"whole": [200, 0, 256], "clusters": [1800, 0, 5, 700], "split": [9000, 0, 40, 3000]}


def run(dtype, lens, H, sinks, scale, seed):
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(seed)
    data, table, _ = pool(np.random.default_rng(seed), dtype, 64, lens)
    for b, n in enumerate(lens):
        if n:
            put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    B = len(lens)
    q = torch.randn((B, H, 512), generator=g, device="cuda").bfloat16()
    sink = torch.tensor(sinks, dtype=torch.float32, device="cuda").repeat(H)[:H].contiguous()
    out = torch.full((B, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    csa2.csa2_paged_attn(q, torch.arange(B, dtype=torch.int32, device="cuda"),
                         torch.tensor(lens, device="cuda") - 1, paged(data, table, dtype), out,
                         workspace(B, H, max(lens)), max_rows=max(lens), sink=sink, lse=lse,
                         scale=scale, inv_freq=inv_freq().cuda())
    csa2.csa2_device_status()
    for b, n in enumerate(lens):
        x = decode(get(data, table, b, 0, n), dtype)
        check_query(out[b], lse[b], q[b], x, sink, scale, n - 1, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale", [512 ** -0.5, 1.5])
def test_sinks_far_below_the_scores(dtype, path, scale):
    sinks = [-1e30, -1e9, 0.5, -1e20, -float("inf"), -3e4, -1e12]
    run(dtype, PATHS[path], 64, sinks, scale, 3)
    run(dtype, PATHS[path], 7, sinks, -scale, 4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,copies", [(1, 1), (64, 1), (700, 1), (5000, 1), (70, 160)])
def test_a_sink_far_below_zero_and_above_the_scores(dtype, n, copies):
    """Every row is the query itself and the scale negative: scores of some -1.5e7 under a sink
    of -1e7, which takes all the mass."""
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(n)
    data, table, _ = pool(np.random.default_rng(n), dtype, 64, [n])
    x = quantised(torch.randn((1, 512), generator=g, device="cuda"), dtype)
    put(data, table, 0, x.expand(n, -1))
    rows = decode(get(data, table, 0, 0, n), dtype)
    q = rows[:1, None].expand(copies, 64, 512).bfloat16().contiguous()
    sink = torch.full((64,), -1e7, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((copies, 64), 7.0, device="cuda")
    csa2.csa2_paged_attn(q, torch.zeros(copies, dtype=torch.int32, device="cuda"),
                         torch.full((copies,), n - 1, device="cuda"), paged(data, table, dtype), out,
                         workspace(copies, 64, n), max_rows=n, sink=sink, lse=lse, scale=-3e4)
    csa2.csa2_device_status()
    for i in range(0, copies, 53):
        check_query(out[i], lse[i], q[i], rows, sink, -3e4, n - 1, False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("path", PATHS)
def test_sinks_at_the_ends_of_fp32(dtype, path):
    """Finite sinks whose base-2 logit is not: no mass below, all of it above, and lse of a query
    without rows is the sink."""
    big = float(np.finfo(np.float32).max)
    run(dtype, PATHS[path], 64, [big, -big, 3e38, -3e38, 0.25, 2e38, -2e38], 512 ** -0.5, 5)
