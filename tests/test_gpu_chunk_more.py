"""Chunk attention and rows read back: calls that the header allows and test_gpu_chunk.py does not make, and
comparisons with the definition where it looks at less.  Tolerances are those of test_gpu_chunk.py."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Case, check_tokens, status, workspace
from test_gpu_paged import BF16, DTYPES, E8M0, S128, decode, get, inv_freq, paged, pool, put, quantised, rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# ---- rows and queries that are not finite -----------------------------------------------------

def spoiled(c, bad, what):
    row = get(c.data, c.table, 0, bad, bad + 1).clone()
    if c.dtype == BF16:
        row[0, 3::7] = float("nan")
    elif what == "codes":
        row[0, 3:512:7] = 0x7F
    elif c.dtype == S128:
        row[0, 516:520] = torch.tensor([float(what)], device="cuda").view(torch.uint8)
    else:
        row[0, 514] = 255
    put(c.data, c.table, 0, row, first=bad)


@pytest.mark.parametrize("dtype,what", [(BF16, "codes"), (S128, "codes"), (S128, "nan"), (S128, "inf"), (S128, "3e38"),
                                        (E8M0, "codes"), (E8M0, "nan")])
@pytest.mark.parametrize("H,page", [(64, 64), (5, 16)])
@pytest.mark.parametrize("bad", [300, 302, 319])
def test_a_row_that_is_not_finite_shows_in_those_that_see_it_alone(dtype, what, H, page, bad):
    c = Case(90, dtype, H, page, [20], [300])
    spoiled(c, bad, what)
    x = decode(get(c.data, c.table, 0, 0, 320), dtype)
    c.call()
    assert status() == 0
    n = bad - 300
    p, lo, hi = c.seen(0)
    if n:
        check_tokens(c.out[:n], c.lse[:n], c.q[:n], x[:bad], lo[:n], hi[:n], c.sink, c.scale, p[:n], True, dtype)
    assert bool((~c.out[n:].isfinite()).flatten(1).any(1).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [0, 50])
def test_queries_of_nan_leave_the_other_heads_right(dtype, window):
    """A NaN query flags every row that its token does not see, whose values then are looked at: finite ones stay."""
    c = Case(91, dtype, 64, 64, [9, 70], [300, 20], window=window)
    gone = [(4, 7), (0, 63), (40, 0), (78, 5)]
    for t, h in gone:
        c.q[t, h, ::3] = float("nan")
    c.call()
    assert status() == 0
    for t, h in gone:
        assert bool(c.out[t, h].isnan().all()) and bool(c.lse[t, h].isnan())
        c.q[t, h] = 0  # what the definition gets: a query of zeros, whose result replaces the NaN
    fixed = c.out.clone(), c.lse.clone()
    c.call()
    for t, h in gone:
        fixed[0][t, h], fixed[1][t, h] = c.out[t, h], c.lse[t, h]
    c.out, c.lse = fixed
    c.check()


def test_the_clipped_sequence_sees_the_rows_there_is_room_for():
    """Room for 200 rows, 16 a sequence and 256 more: 488, of which the first sequence has 160."""
    for dtype, page in ((BF16, 8), (S128, 64), (E8M0, 16)):
        c = Case(92, dtype, 64, page, [60, 70], [100, 900])
        ws = workspace(c.T, c.H, c.cache, c.max_rows, 200)
        c.call(total_rows=200, ws=ws)
        assert status() == 4
        for b, (t0, rows) in enumerate(((0, 160), (60, 328))):
            x = decode(get(c.data, c.table, b, 0, rows), dtype)
            p, lo, hi = c.seen(b)
            t = slice(t0, t0 + c.new[b])
            check_tokens(c.out[t], c.lse[t], c.q[t], x, lo, hi.clamp(max=rows), c.sink, c.scale, p, True, dtype)


# ---- the ends of the ranges -------------------------------------------------------------------

@pytest.mark.parametrize("dtype,page", [(BF16, 64), (BF16, 8), (S128, 64), (E8M0, 16)])
def test_sequences_that_share_pages(dtype, page):
    """A common prefix: the same pages in several rows of the table, and the same page twice in one."""
    c = Case(93, dtype, 64, page, [40, 9, 300], [256, 512, 256])
    for b in (1, 2):
        c.table[b, :256 // page] = c.table[0, :256 // page]
    c.table[1, 256 // page] = c.table[1, 0]
    c.call().check()


@pytest.mark.parametrize("dtype", [BF16, S128])
def test_as_many_sequences_as_a_call_takes(dtype):
    B = 65535
    new = [0] * B
    for b, n in ((0, 3), (1, 1), (1023, 2), (1024, 5), (32767, 130), (65533, 1), (65534, 4)):
        new[b] = n
    c = Case(94, dtype, 16, 64, new, [b % 300 for b in range(B)], pad=3)
    c.call().check()
    c.new[65534] = 0  # the last ones without tokens
    c.cu[-1] = c.cu[-2]
    c.out.fill_(5)
    c.lse.fill_(6)
    c.call().check()


@pytest.mark.parametrize("dtype", [BF16, E8M0])
def test_as_many_tokens_as_a_call_takes(dtype):
    n = 1 << 20
    c = Case(95, dtype, 1, 64, [n - 5, 5], [0, 70], window=20, want_lse=False)
    c.call().check(only=[0, 1, 19, 20, 255, 256, 500000, n - 7, n - 6], at_most=1 << 25)


@pytest.mark.parametrize("page", [64, 32])
def test_the_widest_bounds(page):
    """Bounds on rows that no table here holds: the table's capacity counts."""
    c = Case(96, BF16, 64, page, [5, 70], [3000, 0])
    ws = workspace(c.T, c.H, c.cache, 0x7FFFFF00, 1 << 30)
    c.call(max_rows=0x7FFFFF00, total_rows=1 << 30, ws=ws).check()


def test_a_table_with_strided_rows():
    for dtype in DTYPES:
        c = Case(97, dtype, 64, 64, [50, 3], [400, 900])
        wide = torch.full((2, c.table.shape[1] + 7), 1 << 30, dtype=torch.int32, device="cuda")
        wide[:, :c.table.shape[1]] = c.table
        c.cache = paged(c.data, wide[:, :c.table.shape[1]], dtype)
        c.call().check()


# ---- rows read back ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_read_back_by_a_graph(dtype):
    """Replayed with other rows, lengths, places and pages, on another stream than the capture's."""
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(1), dtype, 64, [400, 300])
    g = torch.Generator(device="cuda").manual_seed(1)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    first = torch.zeros(2, dtype=torch.int64, device="cuda")
    out = torch.empty((500, 512), dtype=torch.bfloat16, device="cuda")
    f, cache = inv_freq().cuda(), paged(data, table, dtype)
    csa2.csa2_paged_read(out, cu, first, cache, inv_freq=f, ratio=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.csa2_paged_read(out, cu, first, cache, inv_freq=f, ratio=2)
    s = torch.cuda.Stream()
    for lens, at in (([300, 200], [0, 100]), ([1, 0], [399, 0]), ([0, 33], [5, 267]), ([0, 0], [0, 0])):
        for b, n in enumerate((400, 300)):
            put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
        table.copy_(table.flip(0).contiguous() if lens[0] == 1 else table)
        if lens[0] == 1:  # the sequences change places: 300 and 400 rows
            at = [299, 0]
        cu.copy_(torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))
        first.copy_(torch.tensor(at))
        out.fill_(9)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        assert status() == 0
        t = 0
        for b, n in enumerate(lens):
            x = decode(get(data, table, b, at[b], at[b] + n), dtype)
            pair = 2.0 ** -20 * x[:, 448:].abs().reshape(n, 32, 2).sum(-1).repeat_interleave(2, 1)
            x = rotated(x, (at[b] + torch.arange(n, device="cuda")) * 2, -1)
            tol = 2.0 ** -8 * x.abs() * (1 + 2.0 ** -23) + 1e-38
            tol[:, 448:] += pair
            assert bool(((out[t:t + n].double() - x).abs() <= tol).all())
            t += n
        assert bool((out[t:] == 9).all())
        if lens[0] == 1:
            table.copy_(table.flip(0).contiguous())
