"""Cache rows with infinities whose scores are -inf: the weight is 0, and 0 times infinity is NaN in the dims
that hold one, for each token that sees the row and for no other, whichever tokens share its tile.

Tolerances as check_tokens of test_gpu_chunk.py (the row has no weight, so the other dims are those of the rows
without it); which outputs are not finite has to be as the definition says."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import Case, check_tokens, status
from test_gpu_paged import BF16, DTYPES, E8M0, S128, decode, get, put

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def spoil(c, b, row, dims, value):
    """Sets dims of a cache row to +-infinity (FP8: to +-1 with an infinite or huge scale, which makes the whole
    group of the scale infinite); returns the dims that are not finite then."""
    r = get(c.data, c.table, b, row, row + 1).clone()
    if c.dtype == BF16:
        r[0, dims] = value
    elif c.dtype == S128:
        for g in {d // 128 for d in dims}:
            r[0, 128 * g:128 * g + 128] = 0x38 | (0x80 if value < 0 else 0)
            r[0, 512 + 4 * g:516 + 4 * g] = torch.tensor([float("inf")], device="cuda").view(torch.uint8)
    else:
        for g in {d // 32 for d in dims}:
            r[0, 32 * g:32 * g + 32] = 0x7E | (0x80 if value < 0 else 0)  # 448 * 2^127
            r[0, 512 + g] = 254
    put(c.data, c.table, b, r, first=row)
    x = r[0].double() if c.dtype == BF16 else decode(r, c.dtype)[0]
    return (~x.float().isfinite()).nonzero()[:, 0]


def negative(c, b, bad, dims, sign, heads):
    """Queries of sequence b: the heads `heads` get scores of -inf with the row, the others of +inf."""
    t = slice(int(c.cu[b]), int(c.cu[b + 1]))
    q = c.q[t]
    v = q[..., dims].float().abs().clamp(min=2.0 ** -10).bfloat16()
    side = torch.full((c.H,), sign, device="cuda", dtype=torch.bfloat16)
    side[heads] = -sign
    q[..., dims] = v * side[:, None]


def check_sequence(c, b, bads, dims, heads):
    """Tokens of sequence b: those that see a row of `bads` are NaN in `dims` (turned pairs with both of their
    dims) for `heads`, whole for the other heads; the others, and the other dims, as without these rows."""
    p, lo, hi = c.seen(b)
    x = decode(get(c.data, c.table, b, 0, c.rows[b]), c.dtype)
    keep = torch.tensor([j for j in range(c.rows[b]) if j not in bads], device="cuda")
    less = lambda n: sum((n > j).long() for j in bads)  # rows of `bads` below n
    t0, n = int(c.cu[b]), c.new[b]
    out, lse = c.out[t0:t0 + n], c.lse[t0:t0 + n]
    sees = sum(((lo <= j) & (j < hi)).long() for j in bads) > 0
    gone = torch.zeros((n, c.H, 512), dtype=torch.bool, device="cuda")
    d = torch.zeros(512, dtype=torch.bool, device="cuda")
    d[dims] = True
    if c.rope:
        d[448:] = d[448:].view(32, 2).any(1).repeat_interleave(2)
    h = torch.zeros(c.H, dtype=torch.bool, device="cuda")
    h[heads] = True
    gone |= sees[:, None, None] & (d | ~h[:, None])
    assert torch.equal(~out.isfinite(), gone)
    assert torch.equal(~lse.isfinite(), sees[:, None] & ~h)
    # the finite outputs: as without the rows (those of `gone` get what the formula has there)
    q = c.q[t0:t0 + n][:, heads].contiguous()
    sink = None if c.sink is None else c.sink[heads]
    l2, h2 = lo - less(lo), hi - less(hi)
    xs = x[keep]
    s = (c.scale * q.double().flatten(0, 1) @ xs.T).masked_fill(
        ~((torch.arange(len(keep), device="cuda") >= l2[:, None]) & (torch.arange(len(keep), device="cuda") < h2[:, None]))
        .repeat_interleave(len(heads), 0), -np.inf)
    full = s if sink is None else torch.cat([s, sink.double().repeat(n)[:, None]], 1)
    ref = torch.softmax(full, 1)[:, :len(keep)] @ xs
    if c.rope:
        from test_gpu_paged import rotated
        ref = rotated(ref, p.repeat_interleave(len(heads)), -1)
    o = torch.where(gone[:, heads], ref.view(n, len(heads), 512).to(torch.bfloat16), out[:, heads])
    check_tokens(o, lse[:, heads].contiguous(), q, xs, l2, h2, sink, c.scale, p, c.rope, c.dtype)


HEADS = [0, 1, 5, 17, 30, 31, 32, 33, 62, 63]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("bad", [3, 255, 256, 300, 301, 305, 319])
@pytest.mark.parametrize("dims", [[5], [450], [130, 200, 511]])
def test_rows_that_only_later_tokens_see(dtype, value, bad, dims):
    """Twenty tokens behind 300 rows: key tile 0 is seen by all of them, tile 1 is not."""
    c = Case(80, dtype, 64, 64, [20], [300])
    d = spoil(c, 0, bad, dims, value)
    negative(c, 0, bad, d, 1.0 if value > 0 else -1.0, HEADS)
    c.call()
    assert status() == 0
    check_sequence(c, 0, [bad], d, HEADS)


@pytest.mark.parametrize("dtype,page", [(BF16, 64), (BF16, 8), (BF16, 48), (S128, 64), (E8M0, 16)])
@pytest.mark.parametrize("window", [0, 100])
def test_rows_of_every_way_to_the_rows(dtype, page, window):
    """Whole pages and pieces, copied rows; several such rows in a tile, also behind a window's beginning."""
    c = Case(81, dtype, 64, page, [30, 90, 8], [500, 0, 250], window=window, rope=False)
    for b, bads in ((0, [440, 505, 529]), (1, [40]), (2, [249, 256])):
        for j in bads:
            d = spoil(c, b, j, [77], float("inf"))
        negative(c, b, bads, d, 1.0, HEADS)
    c.call()
    assert status() == 0
    for b, bads in ((0, [440, 505, 529]), (1, [40]), (2, [249, 256])):
        check_sequence(c, b, bads, d, HEADS)


@pytest.mark.parametrize("dtype", [BF16, S128])
@pytest.mark.parametrize("hist,new", [(20000, [3]), (3000, [200] * 8)])
def test_tiles_of_several_pairs(dtype, hist, new):
    """Parts that are joined: the row lies in the last part, whose key tile is masked."""
    c = Case(82, dtype, 64, 64, new, [hist] * len(new))
    for b, n in enumerate(new):
        d = spoil(c, b, hist + n // 2, [300], -float("inf"))
        negative(c, b, 0, d, -1.0, HEADS)
    c.call()
    assert status() == 0
    for b, n in enumerate(new):
        check_sequence(c, b, [hist + n // 2], d, HEADS)


def test_the_same_in_chunks_of_any_size():
    """A token's outputs do not depend on which others share its tile."""
    c = Case(83, BF16, 16, 64, [24], [290])
    heads = list(range(0, 16, 2))
    d = spoil(c, 0, 300, [9, 449], float("inf"))
    negative(c, 0, 300, d, 1.0, heads)
    c.call()
    torch.cuda.synchronize()
    whole = c.out.clone()
    check_sequence(c, 0, [300], d, heads)
    cu, start = c.cu.clone(), c.start.clone()
    for size in (1, 5, 8):
        for t in range(0, 24, size):
            n = min(size, 24 - t)
            out = torch.full((n, 16, 512), 5.0, dtype=torch.bfloat16, device="cuda")
            cu[1] = n
            start[0] = 290 + t
            c.call(q=c.q[t:t + n], cu_seqlens=cu, start_pos=start, out=out, lse=None)
            assert torch.equal(out.isfinite(), whole[t:t + n].isfinite())
    assert status() == 0


def test_scores_below_fp32_of_finite_rows_weigh_nothing():
    """A score that overflows to -inf although row and query are finite: weight 0, and 0 times finite is 0."""
    c = Case(84, BF16, 64, 64, [20], [300], rope=False)
    row = get(c.data, c.table, 0, 305, 306).clone()
    row[0, 3:6] = 3.0e38
    put(c.data, c.table, 0, row, first=305)
    c.q[:, :, 3:6] = -c.q[:, :, 3:6].abs().clamp(min=0.5)
    c.call()
    assert status() == 0
    p, lo, hi = c.seen(0)
    x = decode(get(c.data, c.table, 0, 0, 320), BF16)
    keep = torch.cat([x[:305], x[306:]])
    check_tokens(c.out, c.lse, c.q, keep, lo, hi - (hi > 305).long(), c.sink, c.scale, p, False, BF16)
