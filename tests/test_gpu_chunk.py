"""Chunks of new tokens over the paged cache, and its rows read back, against their formulas in 64 bits.

Tolerances, with those of test_gpu_paged.py for products, weights and lse.  FP8_S128 rows are rounded to
bf16 in two parts on the way, 2^-8 of 2^-8 off (the others are exact in one): a score is off by a further
2^-16 scale sum |q x|, the output by a further 2^-16 of the mean of |x|.
Read back: code times scale in fp32 (2^-24), the rotation 2^-20 (|x0| + |x1|), then bf16's 2^-8."""
import numpy as np
import pytest
import torch

from test_gpu_paged import (BF16, DTYPES, E8M0, S128, decode, get, inv_freq, paged, pool, put, quantised,
                            rotated)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def workspace(T, H, cache, max_rows, total_rows):
    from csa2_compressed_sparse_gb300 import csa2_paged_chunk_attn_workspace_size
    n = csa2_paged_chunk_attn_workspace_size(T, H, cache, max_rows, total_rows)
    # what the workspace holds at first must not matter
    return torch.full((max(1, n),), 0xFF, dtype=torch.uint8, device="cuda")


def check_tokens(out, lse, q, x, lo, hi, sink, scale, pos, rope, dtype):
    """Tokens out [n, H, 512], lse [n, H], q [n, H, 512] that see rows lo[i] .. hi[i] - 1 of x [m, 512]
    (64 bits; lo, hi relative to x), at positions pos."""
    n, H = q.shape[:2]
    qd = q.double().reshape(n * H, 512)
    x = x.nan_to_num(0.0, 0.0, 0.0)  # (rows that no token of these sees)
    xa = x.abs()
    j = torch.arange(x.shape[0], device="cuda")
    seen = ((j >= lo[:, None]) & (j < hi[:, None]))[:, None].expand(n, H, -1).reshape(n * H, -1)
    s = (scale * qd @ x.T).masked_fill(~seen, -np.inf)
    size = abs(scale) * (qd.abs() @ xa.T).masked_fill(~seen, 0.0)
    extra = 2.0 ** -16 if dtype == S128 else 0.0
    tau = (512 * 2.0 ** -23 + extra) * (size.amax(1) if x.shape[0] else torch.zeros(n * H, device="cuda"))
    tau = tau.double()
    full = s if sink is None else torch.cat([s, sink.double().repeat(n)[:, None]], 1)
    z = torch.logsumexp(full, 1) if full.shape[1] else torch.full((n * H,), -np.inf, device="cuda",
                                                                dtype=torch.float64)
    w = torch.exp(s - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[:, None])
    ref, A = w @ x, w @ xa
    tol = (2 * 2.0 ** -8 * 1.01 + extra + 2 * tau * torch.exp(tau) + 2.0 ** -19)[:, None] * A
    if rope:
        ref = rotated(ref, pos.repeat_interleave(H), -1)
        pair = (tol + 2.0 ** -20 * A).reshape(n * H, 256, 2).sum(-1).repeat_interleave(2, 1)
        tol = torch.cat([tol[:, :448], pair[:, 448:]], 1)
    tol = tol + 2.0 ** -8 * ref.abs() + 1e-37
    err = (out.double().reshape(n * H, 512) - ref).abs()
    assert bool((err <= tol).all()), f"output off by {float((err / tol).nan_to_num(1e30).max()):.3g} x its tolerance"
    if lse is not None:
        got = lse.double().reshape(-1)
        fin = torch.isfinite(z)
        assert torch.equal(got[~fin], z[~fin])
        e = (got - z).abs()[fin]
        t = (tau + 2.0 ** -19 + 2.0 ** -22 * z.abs())[fin]
        assert bool((e <= t).all()), f"lse off by {float((e / t).max()):.3g} x its tolerance"


class Case:
    """A cache of sequences with hist[b] positions behind them and new[b] new tokens, and a call."""

    def __init__(self, seed, dtype, H, page, new, hist, ratio=1, window=0, pad=0, sink="normal", rope=True,
                 want_lse=True, scale=512 ** -0.5, layers=0, spread=1.0, tail=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, page=page, new=new, hist=hist, ratio=ratio, window=window,
                             rope=rope, scale=scale)
        self.rows = [max(0, (h + n) // ratio) if n else 0 for h, n in zip(hist, new)]
        self.data, self.table, self.whole = pool(rng, dtype, page, [r + tail for r in self.rows], layers=layers)
        for b, n in enumerate(self.rows):
            if n:
                x = spread * torch.randn((n, 512), generator=g, device="cuda")
                put(self.data, self.table, b, quantised(x, dtype))
        T = sum(new) + pad
        self.T, self.B = T, len(new)
        self.q = torch.randn((T, H, 512), generator=g, device="cuda").bfloat16()
        self.cu = torch.tensor(np.cumsum([0] + list(new)), dtype=torch.int32, device="cuda")
        self.start = torch.tensor(hist, dtype=torch.int64, device="cuda")
        self.sink = {"normal": torch.randn((H,), generator=g, device="cuda"), None: None,
                     "-inf": torch.full((H,), -np.inf, device="cuda")}.get(sink, sink) if isinstance(
                         sink, (str, type(None))) else sink
        self.freq = inv_freq().cuda() if rope else None
        self.out = torch.full((T, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, H), 6.0, device="cuda") if want_lse else None
        self.cache = paged(self.data, self.table, dtype)
        self.max_rows, self.total = max(self.rows + [0]), sum(self.rows)
        self.ws = workspace(T, H, self.cache, self.max_rows, self.total)

    def call(self, **kw):
        import csa2_compressed_sparse_gb300 as csa2
        a = dict(q=self.q, cu_seqlens=self.cu, start_pos=self.start, cache=self.cache, out=self.out,
                 ws=self.ws, max_rows=self.max_rows, total_rows=self.total, ratio=self.ratio,
                 window=self.window, sink=self.sink, lse=self.lse, scale=self.scale,
                 inv_freq=self.freq)
        a.update(kw)
        csa2.csa2_paged_chunk_attn(**a)
        return self

    def seen(self, b):
        p = self.hist[b] + torch.arange(self.new[b], device="cuda")
        hi = torch.where(p < 0, 0, (p + 1) // self.ratio)
        lo = (hi - self.window).clamp(min=0) if self.window else torch.zeros_like(hi)
        return p, lo, hi

    def check(self, only=None, at_most=1 << 26):
        """Every token of every sequence, or those of the indices `only`, in blocks."""
        import csa2_compressed_sparse_gb300 as csa2
        torch.cuda.synchronize()
        csa2.csa2_device_status()
        for b in range(self.B):
            if self.new[b] == 0:
                continue
            p, lo, hi = self.seen(b)
            x = decode(get(self.data, self.table, b, 0, self.rows[b]), self.dtype)
            t0 = int(self.cu[b])
            idx = torch.arange(self.new[b], device="cuda") if only is None else torch.tensor(
                [i for i in only if i < self.new[b]], device="cuda")
            n = max(1, at_most // (self.H * max(1, self.rows[b])))
            for k in range(0, idx.numel(), n):
                i = idx[k:k + n]
                a, e = int(lo[i].min()), int(hi[i].max())
                check_tokens(self.out[t0 + i], None if self.lse is None else self.lse[t0 + i], self.q[t0 + i],
                             x[a:e], lo[i] - a, hi[i] - a, self.sink, self.scale, p[i], self.rope, self.dtype)
        end = int(self.cu[-1])
        assert bool((self.out[end:] == 5).all()), "padded tokens keep what they hold"
        if self.lse is not None:
            assert bool((self.lse[end:] == 6).all())
        return self


# ================================ attention ====================================================

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 5, 16, 63, 64, 65, 100, 128])
def test_head_counts(dtype, H):
    Case(H, dtype, H, 64, [9, 0, 1, 40], [100, 3, 0, 513]).call().check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 72, 128, 256, 1000])
def test_page_sizes(dtype, page):
    Case(page, dtype, 64, page, [7, 30], [650, 300]).call().check()


def test_codes_times_scales_are_not_rounded_once():
    """FP8_S128 rows with scales of a full mantissa.  One row is seen and no sink, so lse is its score:
    rounded once it would be some 2^-10 of sum |q x| off."""
    c = Case(40, S128, 64, 64, [1], [0], sink=None, spread=1.2345678).call().check()
    c2 = Case(41, S128, 64, 64, [1] * 30, [0] * 30, sink=None, spread=3.1).call().check()
    for d in (c, c2):
        for b in range(d.B):
            x = decode(get(d.data, d.table, b, 0, 1), S128)[0]
            s = d.q[b].double() @ x * d.scale
            size = d.q[b].double().abs() @ x.abs() * d.scale
            assert bool(((d.lse[b].double() - s).abs() <= (2.0 ** -16 + 512 * 2.0 ** -23) * size + 2.0 ** -19).all())
            # its weight is one: the output is the row (rotated back from position 0), rounded once
            assert bool(((d.out[b].double() - x).abs() <= (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -19) * x.abs()).all())


def test_scales_at_the_ends_of_the_range():
    """FP8_S128 rows whose values overflow bf16 when rounded give infinite scores, not others' NaN."""
    c = Case(42, S128, 64, 64, [9], [300])
    row = get(c.data, c.table, 0, 305, 306).clone()
    row[0, 512:516] = torch.tensor([3.0e38], device="cuda").view(torch.uint8)
    put(c.data, c.table, 0, row, first=305)
    x = decode(get(c.data, c.table, 0, 0, 309), S128)
    c.call()
    torch.cuda.synchronize()
    p, lo, hi = c.seen(0)
    check_tokens(c.out[:5], c.lse[:5], c.q[:5], x[:305], lo[:5], hi[:5], c.sink, c.scale, p[:5], True, S128)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("H", [64, 16])
def test_one_sequence_of_any_length(n, H):
    Case(n, BF16, H, 64, [n], [0]).call().check()


@pytest.mark.parametrize("rows", [1, 7, 8, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1025])
def test_rows_around_tile_borders(rows):
    Case(rows, BF16, 64, 64, [1, 3], [rows - 1, max(0, rows - 3)]).call().check()
    Case(rows, E8M0, 32, 16, [2], [rows - 1]).call().check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_whole_prompts_packed(dtype):
    Case(11, dtype, 64, 64, [300, 1, 0, 777, 64], [0] * 5, pad=3).call().check()


@pytest.mark.parametrize("ratio", [2, 3, 128])
def test_ratios(ratio):
    """Tokens of the first group see no row."""
    Case(ratio, BF16, 64, 64, [2 * ratio + 3, 5, 17], [0, ratio - 1, 700], ratio=ratio).call().check()
    Case(ratio, S128, 8, 16, [2 * ratio + 3, 5, 1], [0, 3 * ratio, 0], ratio=ratio).call().check()


@pytest.mark.parametrize("window", [1, 7, 64, 100, 128, 256, 257, 1000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_windows(window, dtype):
    Case(window, dtype, 64, 16 if dtype == E8M0 else 64, [50, 3], [900, 10], window=window).call().check()


@pytest.mark.parametrize("window", [5, 300])
def test_windows_of_few_heads(window):
    """128 tokens to a tile: the window of the first begins well before that of the last."""
    Case(window, BF16, 1, 64, [700], [50], window=window).call().check()


@pytest.mark.parametrize("sink", [None, "-inf", "normal"])
@pytest.mark.parametrize("rope", [True, False])
def test_sinks_and_rotation(sink, rope):
    Case(1, BF16, 64, 64, [20, 1], [300, 0], sink=sink, rope=rope, ratio=2, want_lse=rope).call().check()


def test_extreme_sinks():
    """Sinks far above and far below all scores, up to the ends of fp32."""
    sink = torch.zeros(64, device="cuda")
    top = torch.finfo(torch.float32).max
    for i, v in enumerate([top, -top, 1e30, -1e30, 200.0, -200.0, 1e5, -1e5]):
        sink[i] = v
    c = Case(2, BF16, 64, 64, [6], [700], sink=sink).call()
    torch.cuda.synchronize()
    assert bool(c.out[:, 0].eq(0).all()) and bool(c.out[:, 2].eq(0).all()) and bool(c.out[:, 6].eq(0).all())
    assert bool(c.lse.isfinite().all()) and bool(c.out.isfinite().all())
    c.out = c.out[:, 8:].contiguous()
    c.lse, c.q, c.sink, c.H = c.lse[:, 8:].contiguous(), c.q[:, 8:].contiguous(), sink[8:], 56
    c.check()


@pytest.mark.parametrize("spread,scale", [(8.0, 0.3), (1e-3, 1.0), (1.0, 0.0), (1.0, -512 ** -0.5)])
def test_score_sizes(spread, scale):
    """Scores of some hundred, whose maximum moves often; of nearly zero; of exactly zero; negative scale."""
    Case(3, BF16, 64, 64, [9], [3000], spread=spread, scale=scale).call().check()


def test_rising_scores():
    """Each tile's scores are far above the last one's: every tile moves the maximum."""
    c = Case(4, BF16, 16, 64, [8], [2040])
    x = torch.randn((1, 512), device="cuda").bfloat16()
    c.q.copy_(x.expand_as(c.q))
    n = c.rows[0]
    put(c.data, c.table, 0, (x.float() * torch.linspace(0, 40, n, device="cuda")[:, None]).bfloat16())
    c.call().check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_layers_interleaved_in_one_pool(dtype):
    Case(5, dtype, 64, 64, [30, 5], [200, 40], layers=3).call().check()


@pytest.mark.parametrize("H,n,hist", [(64, 2, 70000), (64, 16, 40000), (16, 1, 140000), (128, 3, 20000)])
def test_few_tokens_of_a_long_sequence(H, n, hist):
    """The rows of one tile of queries are shared out over the whole GPU and joined."""
    Case(6, BF16, H, 64, [n], [hist]).call().check()


def test_long_chunk():
    Case(7, BF16, 64, 64, [1500, 700], [9000, 0], ratio=2).call().check(only=list(range(0, 1500, 37)) + [1499, 699])


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_wide_ragged_batch(dtype):
    rng = np.random.default_rng(8)
    new = [int(x) for x in rng.integers(0, 12, 150)]
    hist = [int(x) for x in rng.integers(0, 900, 150)]
    Case(8, dtype, 32, 16, new, hist, pad=5).call().check()


def test_the_same_as_token_by_token():
    """csa2_paged_attn sees the same: both are within their tolerance, so they differ by at most two."""
    import csa2_compressed_sparse_gb300 as csa2
    c = Case(9, BF16, 64, 64, [33, 4], [500, 0]).call()
    q_seq = torch.tensor([0] * 33 + [1] * 4, dtype=torch.int32, device="cuda")
    q_pos = torch.cat([c.seen(0)[0], c.seen(1)[0]])
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    ws = torch.empty(csa2.csa2_paged_attn_workspace_size(37, 64, c.max_rows), dtype=torch.uint8, device="cuda")
    csa2.csa2_paged_attn(c.q, q_seq, q_pos, c.cache, out, ws, max_rows=c.max_rows, sink=c.sink, lse=lse,
                         inv_freq=inv_freq().cuda())
    c.check()
    c.out, c.lse = out, lse
    c.check()


def test_results_do_not_depend_on_the_run():
    for new, hist in (([200, 3], [900, 5]), ([2], [50000]), ([40] * 20, [300] * 20)):
        c = Case(10, BF16, 64, 64, new, hist).call()
        first, lse = c.out.clone(), c.lse.clone()
        for _ in range(3):
            c.out.fill_(1)
            c.ws.random_(0, 255)
            c.call()
            assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [64, 4])
def test_a_later_tokens_row_does_not_reach_earlier_ones(value, H):
    """A row that only later tokens of the same tile see holds NaN or infinities."""
    for bad in (300, 301, 305, 319):
        c = Case(12, BF16, H, 64, [20], [300])
        row = get(c.data, c.table, 0, bad, bad + 1)
        row[0, 3::7] = value
        put(c.data, c.table, 0, row, first=bad)
        c.call()
        torch.cuda.synchronize()
        n = bad - 300  # tokens before it
        if n:
            x = decode(get(c.data, c.table, 0, 0, c.rows[0]), BF16)
            p, lo, hi = c.seen(0)
            check_tokens(c.out[:n], c.lse[:n], c.q[:n], x[:bad], lo[:n], hi[:n], c.sink, c.scale, p[:n], True, BF16)
        assert bool((~c.out[n:].isfinite()).flatten(1).any(1).all()), "tokens that see it show it"


def test_rows_before_the_window_do_not_reach_later_tokens():
    c = Case(13, BF16, 64, 64, [12], [500], window=100)
    row = torch.full((1, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    for bad in (0, 300, 401, 403):  # token i sees rows 401 + i .. 500 + i
        put(c.data, c.table, 0, row, first=bad)
    c.call()
    torch.cuda.synchronize()
    assert bool(c.out[:3].isnan().flatten(1).any(1).all())
    x = decode(get(c.data, c.table, 0, 0, c.rows[0]), BF16)
    p, lo, hi = c.seen(0)
    check_tokens(c.out[3:], c.lse[3:], c.q[3:], x[404:], lo[3:] - 404, hi[3:] - 404, c.sink, c.scale, p[3:], True, BF16)


def test_queries_of_nan_stay_in_their_head():
    c = Case(14, BF16, 64, 64, [9], [300])
    c.q[4, 7] = float("nan")
    c.call()
    torch.cuda.synchronize()
    assert bool(c.out[4, 7].isnan().all()) and bool(c.lse[4, 7].isnan())
    c.q[4, 7] = 0  # the reference's
    keep = torch.ones((9, 64), dtype=torch.bool, device="cuda")
    keep[4, 7] = False
    assert bool(c.out[keep].isfinite().all())


# ---- data-dependent faults, found by the kernels' own checks --------------------------------

def status():
    import csa2_compressed_sparse_gb300 as csa2
    torch.cuda.synchronize()
    try:
        csa2.csa2_device_status()
    except csa2.Csa2Error as e:
        return e.status
    return 0


def test_pages_outside_the_pool_are_skipped():
    for dtype, page in ((BF16, 64), (BF16, 16), (S128, 64)):
        c = Case(15, dtype, 64, page, [5, 40], [200, 300])
        x = [decode(get(c.data, c.table, b, 0, c.rows[b]), dtype) for b in (0, 1)]
        c.table[0, 1] = c.data.shape[0]  # one past the last
        c.table[0, 2] = -1
        c.call()
        assert status() == 4
        p, lo, hi = c.seen(0)
        gone = slice(page, 3 * page)
        keep = torch.cat([x[0][:page], x[0][3 * page:]])
        check_tokens(c.out[:5], c.lse[:5], c.q[:5], keep, lo, hi - 2 * page, c.sink, c.scale, p, True, dtype)
        p, lo, hi = c.seen(1)
        check_tokens(c.out[5:45], c.lse[5:45], c.q[5:45], x[1], lo, hi, c.sink, c.scale, p, True, dtype)


def test_more_rows_than_announced_are_clipped():
    c = Case(16, BF16, 64, 64, [4], [300])
    c.call(max_rows=256)
    assert status() == 4
    x = decode(get(c.data, c.table, 0, 0, 256), BF16)
    p, lo, hi = c.seen(0)
    check_tokens(c.out, c.lse, c.q, x, lo, hi.clamp(max=256), c.sink, c.scale, p, True, BF16)
    c.call()
    assert status() == 0


def test_positions_below_zero_see_nothing():
    c = Case(17, BF16, 64, 64, [6], [0])
    c.start.fill_(-3)
    c.hist = [-3]
    c.call().check()


@pytest.mark.parametrize("dtype,H", [(BF16, 64), (S128, 64), (E8M0, 3), (BF16, 128)])
def test_no_rows_at_all(dtype, H):
    """Bounds of zero: the first tokens of groups that are not complete, of one sequence or of hundreds."""
    for B in (1, 300):
        c = Case(50, dtype, H, 64, [2] * B, [0] * B, ratio=128)
        assert c.max_rows == 0 and c.total == 0
        c.call().check()
        assert bool((c.out == 0).all()) and torch.equal(c.lse, c.sink.expand_as(c.lse))


def test_positions_at_the_end_of_int64():
    c = Case(18, BF16, 64, 64, [2], [500])
    c.start.fill_(2 ** 63 - 2)
    c.call(ratio=65536)
    assert status() == 4
    c.start.fill_(500)
    c.call().check()


# ---- calls as programs make them ------------------------------------------------------------

def test_another_stream():
    s = torch.cuda.Stream()
    c = Case(19, BF16, 64, 64, [30, 2], [700, 10])
    torch.cuda.synchronize()
    c.call(stream=s).check()
    with torch.cuda.stream(s):
        c.out.fill_(5)
        c.call()
    c.check()


@pytest.mark.parametrize("dtype", [BF16, S128])
def test_a_graph_replayed_with_other_lengths(dtype):
    """Lengths, positions and pages change between replays; the bounds hold for all of them."""
    c = Case(20, dtype, 64, 64, [20, 40, 3], [1000, 0, 90], pad=10)
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    g.replay()
    c.check()
    c.new, c.hist = [1, 0, 25], [1019, 5, 68]
    c.cu.copy_(torch.tensor(np.cumsum([0] + c.new), dtype=torch.int32))
    c.start.copy_(torch.tensor(c.hist))
    c.out.fill_(5)
    c.lse.fill_(6)
    c.q.copy_(torch.randn(c.q.shape, device="cuda"))
    c.rows = [1020, 0, 93]
    g.replay()
    c.check()


def test_two_calls_at_once():
    a = Case(21, BF16, 64, 64, [300], [4000])
    b = Case(22, S128, 32, 16, [100, 7], [2000, 3])
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a.call(stream=s)
        b.call(stream=t)
    torch.cuda.synchronize()
    a.check(only=range(0, 300, 11))
    b.check()


def test_bounds_may_be_left_out():
    c = Case(23, S128, 16, 64, [5, 6], [100, 0])
    ws = workspace(c.T, c.H, c.cache, None, None)
    c.call(max_rows=None, total_rows=None, ws=ws).check()


def test_one_workspace_for_many_calls_in_a_row():
    cases = [Case(24 + i, BF16, 64, 64, [n], [h]) for i, (n, h) in enumerate([(3, 9000), (200, 0), (2, 30000)])]
    ws = max((c.ws for c in cases), key=lambda w: w.numel())
    for _ in range(2):
        for c in cases:
            c.call(ws=ws)
    for c in cases:
        c.check(only=range(0, 200, 7))


# ---- long segments: tensor memory sums up 65536 rows at most, the rest joins in fp32 ----------

@pytest.mark.parametrize("case", ["plain", "rising", "no_pages", "window", "s128"])
def test_segments_longer_than_a_run(case):
    """Eighty tiles of 300 key tiles and more each: those that one pair works on alone, and the longer parts
    of those that two share, are done in runs."""
    n = 90000 if case == "no_pages" else 80000
    c = Case(30, S128 if case == "s128" else BF16, 64, 64, [160], [n - 160], window=77000 if case == "window" else 0)
    if case == "rising":  # the maximum moves in every run
        x = decode(get(c.data, c.table, 0, 0, n), BF16).float()
        put(c.data, c.table, 0, (x * torch.linspace(0.1, 20, n, device="cuda")[:, None]).bfloat16())
    if case != "no_pages":
        c.call().check(only=range(0, 160, 13))
        return
    gone = 1100 * 64  # the first run sees nothing at all
    x = decode(get(c.data, c.table, 0, gone, n), BF16)
    c.table[0, :1100] = -1
    c.call()
    assert status() == 4
    p, lo, hi = c.seen(0)
    for i in range(0, 160, 13):
        check_tokens(c.out[i:i + 1], c.lse[i:i + 1], c.q[i:i + 1], x, lo[i:i + 1], hi[i:i + 1] - gone, c.sink,
                     c.scale, p[i:i + 1], True, BF16)


def test_runs_do_not_depend_on_the_run():
    c = Case(31, BF16, 64, 64, [160], [70000]).call()
    first, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(1)
    c.ws.random_(0, 255)
    c.call()
    assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


# ---- every way to the rows: whole pages, pieces of 32, 16 and 8 rows, copied first -------------

@pytest.mark.parametrize("page", [8, 24, 16, 48, 32, 96])
@pytest.mark.parametrize("new", [[1, 3], [40, 2], [130, 50]])
@pytest.mark.parametrize("window", [0, 90])
def test_small_pages(page, new, window):
    Case(page, BF16, 64, page, new, [700, 333], window=window, ratio=1 + (page == 48)).call().check()


@pytest.mark.parametrize("dtype,page", [(BF16, 8), (BF16, 16), (S128, 64), (E8M0, 24)])
def test_bad_pages_of_copied_rows(dtype, page):
    c = Case(32, dtype, 64, page, [100], [300])
    x = decode(get(c.data, c.table, 0, 0, 400), dtype)
    c.table[0, 3] = c.data.shape[0]
    c.table[0, 4] = -7
    c.call()
    assert status() == 4
    p, lo, hi = c.seen(0)
    there = hi.clamp(max=3 * page) + (hi - 5 * page).clamp(min=0)  # of the rows 0 .. hi - 1
    check_tokens(c.out, c.lse, c.q, torch.cat([x[:3 * page], x[5 * page:]]), lo, there, c.sink, c.scale, p, True,
                 dtype)


@pytest.mark.parametrize("dtype,page", [(BF16, 8), (S128, 64)])
def test_more_rows_than_announced_are_left_out(dtype, page):
    """Room for the first sequence's rows and a few of the second's."""
    c = Case(33, dtype, 64, page, [60, 70], [100, 900])
    c.call(total_rows=200)
    assert status() == 4
    x = decode(get(c.data, c.table, 0, 0, 160), dtype)
    p, lo, hi = c.seen(0)
    check_tokens(c.out[:60], c.lse[:60], c.q[:60], x, lo, hi, c.sink, c.scale, p, True, dtype)
    assert bool(c.out[60:].isfinite().all()) and bool((c.out[60:] != 5).any())
    c.out.fill_(5)
    c.call().check()


@pytest.mark.parametrize("B", [3, 32, 33, 60, 256, 257, 300])
def test_few_tokens_of_many_sequences(B):
    """Up to 256 sequences the pairs find their own tiles, with empty sequences among the others."""
    new = [0] * B
    for i, b in enumerate(range(B - 1, 0, -max(1, B // 9))):
        new[b] = 1 + i % 5
    Case(B, BF16, 64, 64, new, [17 * b % 900 for b in range(B)], pad=2).call().check()


@pytest.mark.parametrize("n,hist", [(40, 300), (2, 40000)])
def test_outputs_at_odd_chunks(n, hist):
    """16-byte aligned, not 32."""
    c = Case(34, BF16, 64, 64, [n], [hist])
    for name in ("q", "out"):
        t = getattr(c, name)
        whole = torch.full((t.numel() + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
        view = whole[8:-8].view(t.shape)
        view.copy_(t)
        setattr(c, name, view)
        setattr(c, name + "_whole", whole)
    assert c.out.data_ptr() % 32 == 16
    c.call().check()
    assert bool((c.out_whole[:8] == 5).all()) and bool((c.out_whole[-8:] == 5).all())


def test_queries_beyond_4_gib():
    c = Case(51, BF16, 128, 64, [9, 35000], [0, 3], window=16, want_lse=False, rope=False)
    assert c.q.numel() > 1 << 31
    c.call().check(only=[0, 1, 8, 20000, 32760, 32768, 34990, 34998, 34999], at_most=1 << 24)
    del c
    torch.cuda.empty_cache()


# ================================ read =========================================================

def read_case(seed, dtype, page, lens, first, back=False, ratio=1, pad=0, gap=0, stream=None, layers=0):
    import csa2_compressed_sparse_gb300 as csa2
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    data, table, _ = pool(rng, dtype, page, [f + n for f, n in zip(first, lens)], layers=layers)
    for b, n in enumerate(lens):
        if n:
            x = torch.randn((n, 512), generator=g, device="cuda")
            put(data, table, b, quantised(x, dtype), first=first[b])
    T = sum(lens) + pad
    whole = torch.full((max(1, T), 512 + gap), 9.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:T, :512]
    cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    csa2.csa2_paged_read(out, cu, torch.tensor(first, dtype=torch.int64, device="cuda"), paged(data, table, dtype),
                         inv_freq=inv_freq().cuda() if back else None, ratio=ratio, stream=stream)
    torch.cuda.synchronize()
    csa2.csa2_device_status()
    at = 0
    for b, n in enumerate(lens):
        x = decode(get(data, table, b, first[b], first[b] + n), dtype)
        got = out[at:at + n].double()
        if dtype == BF16:
            assert torch.equal(got[:, :448], x[:, :448])
        tol = 2.0 ** -8 * x.abs() * (1 + 2.0 ** -23) + 1e-38
        if back:
            pair = 2.0 ** -20 * x[:, 448:].abs().reshape(n, 32, 2).sum(-1).repeat_interleave(2, 1)
            x = rotated(x, (first[b] + torch.arange(n, device="cuda")) * ratio, -1)
            tol = 2.0 ** -8 * x.abs() * (1 + 2.0 ** -23) + 1e-38
            tol[:, 448:] += pair
        elif dtype == BF16:
            assert torch.equal(got, x)
        assert bool(((got - x).abs() <= tol).all())
        at += n
    assert bool((whole[sum(lens):] == 9).all()) and bool((whole[:, 512:] == 9).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 24, 64, 1000])
@pytest.mark.parametrize("back", [False, True])
def test_rows_read_back(dtype, page, back):
    read_case(page, dtype, page, [5, 0, 1, 130, 77], [0, 9, 3, 63, 1000], back=back, pad=4, gap=8 if back else 0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows_read_back(dtype):
    read_case(2, dtype, 64, [30000, 1, 17, 0, 9000], [5, 0, 100, 0, 700], back=True, ratio=2, pad=3)
    read_case(3, dtype, 16, [40] * 300, [11] * 300, layers=2)
    read_case(4, dtype, 64, [1], [0])


def test_rows_beyond_4_gib():
    import csa2_compressed_sparse_gb300 as csa2
    n, ld = 300000, 8192
    data, table, _ = pool(np.random.default_rng(5), BF16, 64, [n])
    x = torch.randn((n, 512), device="cuda").bfloat16()
    put(data, table, 0, x)
    whole = torch.full((n, ld), 9.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    csa2.csa2_paged_read(whole[:, :512], cu, torch.zeros(1, dtype=torch.int64, device="cuda"), paged(data, table, BF16))
    assert torch.equal(whole[:, :512], x) and bool((whole[:, 512:520] == 9).all())


def test_read_is_the_inverse_of_append():
    """What is appended rotated is read rotated back; each of the two roundings to bf16 is 2^-8."""
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(1), BF16, 64, [100, 300])
    kv = torch.randn((400, 512), device="cuda").bfloat16()
    cu = torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int64, device="cuda")
    cache, f = paged(data, table, BF16), inv_freq().cuda()
    csa2.csa2_paged_append(kv, cu, start, cache, inv_freq=f)
    out = torch.empty_like(kv)
    csa2.csa2_paged_read(out, cu, start, cache, inv_freq=f)
    x = kv.double()
    pair = x[:, 448:].abs().reshape(400, 32, 2).sum(-1).repeat_interleave(2, 1)
    assert torch.equal(out[:, :448], kv[:, :448])
    assert bool(((out.double() - x)[:, 448:].abs() <= (2.0 ** -7 + 2.0 ** -18) * pair).all())


def test_bad_pages_leave_their_rows():
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(1), BF16, 8, [40], poison=False)
    put(data, table, 0, torch.ones((40, 512), device="cuda").bfloat16())
    table[0, 2] = data.shape[0]
    out = torch.full((60, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    csa2.csa2_paged_read(out, cu, torch.tensor([-4], device="cuda"), paged(data, table, BF16))
    assert status() == 4
    want = torch.full((60,), 9.0, device="cuda")
    want[4:20] = 1
    want[28:44] = 1
    assert torch.equal(out.float(), want[:, None].expand(60, 512))


def test_read_in_a_graph_and_on_another_stream():
    read_case(5, S128, 64, [50, 3], [0, 7], back=True, stream=torch.cuda.Stream())


# ================================ together =====================================================

@pytest.mark.parametrize("dtype", DTYPES)
def test_a_prompt_in_chunks(dtype):
    """Projections' outputs normed and rotated, appended and attended chunk by chunk, then read back: the
    whole in 64 bits on the rows that the cache holds."""
    import csa2_compressed_sparse_gb300 as csa2
    H, B, f = 64, 2, inv_freq().cuda()
    chunks = [[70, 130], [1, 40], [33, 0]]
    total = [sum(c[b] for c in chunks) for b in range(B)]
    data, table, _ = pool(np.random.default_rng(3), dtype, 64, total)
    cache = paged(data, table, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    done = [0, 0]
    for new in chunks:
        T = sum(new)
        x = torch.randn((T, H + 1, 512), generator=g, device="cuda").bfloat16()
        cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
        start = torch.tensor(done, device="cuda")
        pos = torch.cat([torch.arange(d, d + n, device="cuda") for d, n in zip(done, new)])
        q, kv = torch.empty((T, H, 512), dtype=torch.bfloat16, device="cuda"), x[:, H:]
        csa2.csa2_qk_norm_rope(x[:, :H], q, pos, f)
        csa2.csa2_qk_norm_rope(kv, kv, pos, None)  # the latent's norm; csa2_paged_append rotates it
        csa2.csa2_paged_append(kv[:, 0], cu, start, cache, inv_freq=f)
        out, lse = torch.empty_like(q), torch.empty((T, H), device="cuda")
        rows = [d + n for d, n in zip(done, new)]
        ws = workspace(T, H, cache, max(rows), sum(rows))
        csa2.csa2_paged_chunk_attn(q, cu, start, cache, out, ws, max_rows=max(rows), total_rows=sum(rows),
                                   lse=lse, inv_freq=f)
        torch.cuda.synchronize()
        csa2.csa2_device_status()
        for b in range(B):
            t0, n = int(cu[b]), new[b]
            if n == 0:
                continue
            y = decode(get(data, table, b, 0, rows[b]), dtype)
            p = done[b] + torch.arange(n, device="cuda")
            check_tokens(out[t0:t0 + n], lse[t0:t0 + n], q[t0:t0 + n], y, torch.zeros_like(p), p + 1, None,
                         512 ** -0.5, p, True, dtype)
        done = rows
    back = torch.empty((sum(total), 512), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, total[0], sum(total)], dtype=torch.int32, device="cuda")
    csa2.csa2_paged_read(back, cu, torch.zeros(2, dtype=torch.int64, device="cuda"), cache)
    y = torch.cat([decode(get(data, table, b, 0, total[b]), dtype) for b in range(B)])
    assert bool(((back.double() - y).abs() <= 2.0 ** -8 * y.abs() * (1 + 2.0 ** -23)).all())
