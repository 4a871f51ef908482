"""The paged latent cache against its formulas in 64 bits.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to E4M3 by 2^-4 (2^-10 of
the scale among the subnormal codes), to fp32 by 2^-24.
  * stored rows: bf16 dims below 448 are copied and equal; a rotated value x0 c - x1 s carries
    the angle's rounding (|angle| <= pi: pi 2^-24), sine and cosine (2 units: 2^-22), three
    fp32 roundings: together below 2^-20 (|x0| + |x1|), then the store's own rounding
  * scores: 512 products summed in fp32 are off by at most tau = 512 * 2^-23 * scale sum |q x|
    (2^-23: the tensor core may cut instead of rounding)
  * weights: e^{s - m} is rounded to bf16 (2^-8), its argument is off by tau, ex2 by 2^-21; the
    output is the weighted mean of x, so with A = sum w |x| it is off by at most
    (2 * 2^-8 * 1.01 + 2 tau + 2^-19) A, the factor 2 for numerator and normaliser, and by its
    own rounding 2^-8 |out|; the rotation back adds 2^-20 (|o0| + |o1|) and mixes the errors of
    a pair, so a pair's A are added
  * lse: off by tau + 2^-19 (sum and logarithm) + 2^-22 |lse|
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, S128, E8M0 = "bf16", "fp8_s128", "fp8_e8m0"
DTYPES = [BF16, S128, E8M0]
THETA = 160000.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def inv_freq():
    return torch.tensor(THETA ** (-np.arange(0, 64, 2) / 64.0), dtype=torch.float32)


def e4m3_values():
    v = np.empty(256)
    for k in range(256):
        e, m = (k >> 3) & 15, k & 7
        x = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[k] = -x if k & 128 else x
    return torch.tensor(v, device="cuda")


def decode(rows, dtype):
    """Cache rows [n, 512] bf16 or [n, 528] uint8 -> [n, 512] in 64 bits."""
    if dtype == BF16:
        return rows.double()
    v = e4m3_values()[rows[:, :512].long()]
    tail = rows[:, 512:].contiguous()
    if dtype == S128:
        return v * tail.view(torch.float32).double().repeat_interleave(128, 1)
    return v * torch.exp2(tail.double() - 127).repeat_interleave(32, 1)


def rotated(x, pos, sign):
    """x [..., 512] in 64 bits, rotated by sign * pos theta."""
    f = inv_freq().double().to(x.device)
    z = torch.view_as_complex(x[..., 448:].reshape(*x.shape[:-1], 32, 2).contiguous())
    z = z * torch.polar(torch.ones_like(z.real), sign * pos.double()[..., None] * f)
    return torch.cat([x[..., :448], torch.view_as_real(z).flatten(-2)], -1)


def pool(rng, dtype, page, seqs, poison=True, extra=3, layers=0):
    """A pool for sequences of `seqs` rows in shuffled pages; unused pages and rows hold NaN.
    Returns (data, table, where): where[b] = (pages, offsets) of the rows of b."""
    need = [-(-n // page) for n in seqs]
    n_pages = sum(need) + extra
    cols = max(need + [1]) + 1
    ids = rng.permutation(n_pages)[:sum(need)]
    table = np.full((len(seqs), cols), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    width = 512 if dtype == BF16 else 528
    kind = torch.bfloat16 if dtype == BF16 else torch.uint8
    if layers:  # pages of several layers interleaved: this is the middle one
        whole = torch.empty((n_pages, layers, page, width), dtype=kind, device="cuda")
        data = whole[:, layers // 2]
    else:
        whole = data = torch.empty((n_pages, page, width), dtype=kind, device="cuda")
    if dtype == BF16:
        whole.fill_(float("nan") if poison else 0.0)
    else:
        whole.fill_(0xFF if poison else 0)  # NaN codes, NaN scales
    return data, torch.tensor(table, device="cuda"), whole


def quantised(x, dtype):
    """Valid cache rows of x [n, 512] for tests of the attention (any codes will do)."""
    if dtype == BF16:
        return x.bfloat16()
    g = 128 if dtype == S128 else 32
    v = x.double().reshape(x.shape[0], -1, g)
    top = v.abs().amax(-1, keepdim=True).clamp(min=1e-30)
    if dtype == S128:
        sc = (top / 448).float()
        tail = sc[..., 0].contiguous().view(torch.uint8)
    else:
        e = torch.ceil(torch.log2(top / 448))
        sc = torch.exp2(e).float()
        tail = (e[..., 0] + 127).to(torch.uint8)
    codes = (v.float() / sc).reshape(x.shape).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes, tail], 1)


def put(data, table, b, rows, first=0):
    page = data.shape[1]
    j = torch.arange(first, first + rows.shape[0], device="cuda")
    data[table[b, j // page].long(), j % page] = rows


def get(data, table, b, lo, hi):
    page = data.shape[1]
    j = torch.arange(lo, hi, device="cuda")
    return data[table[b, j // page].long(), j % page]


def paged(data, table, dtype):
    from csa2_compressed_sparse_gb300 import Paged
    return Paged(data, table, fp8_dtype=2 if dtype == E8M0 else 1)


def workspace(Q, H, max_rows):
    from csa2_compressed_sparse_gb300 import csa2_paged_attn_workspace_size
    # what the workspace holds at first must not matter
    return torch.full((max(1, csa2_paged_attn_workspace_size(Q, H, max_rows)),), 0xFF,
                      dtype=torch.uint8, device="cuda")


def check_query(out, lse, q, x, sink, scale, pos, rope):
    """One query: out [H, 512], lse [H], q [H, 512], x [n, 512] in 64 bits."""
    H = q.shape[0]
    qd = q.double()
    s = scale * qd @ x.T
    tau = 512 * 2.0 ** -23 * abs(scale) * (qd.abs() @ x.abs().T)
    tau = tau.amax(1) if x.shape[0] else torch.zeros(H, device="cuda", dtype=torch.float64)
    full = s if sink is None else torch.cat([s, sink.double()[:, None]], 1)
    z = torch.logsumexp(full, 1) if full.shape[1] else torch.full((H,), -np.inf, device="cuda",
                                                                dtype=torch.float64)
    w = torch.exp(s - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[:, None])
    ref = w @ x
    A = w @ x.abs()
    tol = (2 * 2.0 ** -8 * 1.01 + 2 * tau + 2.0 ** -19)[:, None] * A
    if rope:
        ref = rotated(ref, torch.full((H,), int(pos), device="cuda"), -1)
        pair = (tol + 2.0 ** -20 * A).reshape(H, 256, 2).sum(-1).repeat_interleave(2, 1)
        tol = torch.cat([tol[:, :448], pair[:, 448:]], 1)
    tol = tol + 2.0 ** -8 * ref.abs() + 1e-37
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), f"output off by {float((err / tol).max()):.3g} x its tolerance"
    if lse is not None:
        fin = torch.isfinite(z)
        assert torch.equal(lse.double()[~fin], z[~fin])
        e = (lse.double() - z).abs()[fin]
        t = (tau + 2.0 ** -19 + 2.0 ** -22 * z.abs())[fin]
        assert bool((e <= t).all()), f"lse off by {float((e / t).max()):.3g} x its tolerance"


def run_case(seed, dtype, H, page, lens, tokens=1, ratio=1, window=0, pad=0, sink="normal",
             rope=True, want_lse=True, scale=512 ** -0.5, layers=0, tail=0, stream=None, spread=1.0):
    """Random cache and queries; `tail` rows beyond the visible ones hold NaN.  Every query is
    checked; padded ones keep what out and lse hold."""
    import csa2_compressed_sparse_gb300 as csa2
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    data, table, _ = pool(rng, dtype, page, [n + tail for n in lens], layers=layers)
    for b, n in enumerate(lens):
        if n:
            put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda") * spread,
                                          dtype))
    seqs, pos = [], []
    for b, n in enumerate(lens):
        for i in range(tokens):
            seqs.append(b)
            # a position whose last complete group is row n - tokens + i
            pos.append((n - tokens + 1 + i) * ratio - 1 + int(rng.integers(0, ratio)))
    order = rng.permutation(len(seqs))
    seqs = [seqs[i] for i in order] + [-1] * pad
    pos = [pos[i] for i in order] + [12345] * pad
    if pad:  # padded queries in the middle too
        m = len(seqs) // 2
        seqs.insert(m, -1)
        pos.insert(m, 99)
    Q = len(seqs)
    q = torch.randn((Q, H, 512), generator=g, device="cuda").bfloat16()
    sk = None
    if sink != "none":
        sk = torch.randn((H,), generator=g, device="cuda")
        if sink == "inf":
            sk[::2] = -float("inf")
        elif sink == "large":
            sk += 30.0
    out = torch.full((Q, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Q, H), 7.0, device="cuda") if want_lse else None
    hi = [0 if p < 0 else (p + 1) // ratio for p in pos]
    max_rows = max([h for h, b in zip(hi, seqs) if b >= 0] + [0])
    csa2.csa2_paged_attn(q, torch.tensor(seqs, dtype=torch.int32, device="cuda"),
                         torch.tensor(pos, device="cuda"), paged(data, table, dtype), out,
                         workspace(Q, H, max_rows), max_rows=max_rows, ratio=ratio, window=window,
                         sink=sk, lse=lse, scale=scale,
                         inv_freq=inv_freq().cuda() if rope else None, stream=stream)
    csa2.csa2_device_status(stream)
    for i in range(Q):
        if seqs[i] < 0:
            assert bool((out[i] == 7.0).all()) and (lse is None or bool((lse[i] == 7.0).all()))
            continue
        lo = max(0, hi[i] - window) if window else 0
        x = decode(get(data, table, seqs[i], lo, hi[i]), dtype)
        check_query(out[i], None if lse is None else lse[i], q[i], x, sk, scale, pos[i], rope)


# ---- attention ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 256, 257, 1000])
def test_one_sequence(dtype, n):
    run_case(n, dtype, 64, 64, [n], tail=70)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 5, 8, 16, 17, 32, 33, 48, 64, 65, 100, 128])
def test_heads(dtype, H):
    run_case(H, dtype, H, 32, [300, 1, 77])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 16, 24, 40, 48, 64, 96, 128, 1024])
def test_pages(dtype, page):
    run_case(page, dtype, 64, page, [700, 8, 431], tail=9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_ragged_batch_with_padding_and_empty_rows(dtype):
    lens = [0, 1, 3000, 64, 0, 511, 128, 2049, 7]
    run_case(3, dtype, 64, 64, lens, pad=5, sink="normal")
    run_case(4, dtype, 64, 16, lens, pad=1, sink="none", rope=False)
    run_case(5, dtype, 16, 64, lens, tokens=3, sink="inf")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", [1, 63, 64, 65, 128, 300, 5000])
def test_window(dtype, window):
    run_case(window, dtype, 64, 64, [1, 64, 130, 1000, 2222], window=window)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ratio", [2, 3, 128])
def test_ratio(dtype, ratio):
    run_case(ratio, dtype, 64, 16, [5, 400, 1111], ratio=ratio, tail=3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_several_tokens_of_a_sequence(dtype):
    run_case(11, dtype, 64, 64, [3, 900, 64], tokens=5)  # the first ones see nothing


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sink", ["none", "normal", "inf", "large"])
def test_sinks_and_scales(dtype, sink):
    run_case(1, dtype, 64, 64, [200, 600], sink=sink)
    run_case(2, dtype, 64, 64, [200, 600], sink=sink, scale=-0.1)
    run_case(3, dtype, 64, 64, [200, 600], sink=sink, scale=0.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores_move_the_maximum(dtype):
    """Scores of hundreds in standard deviation: the running maximum moves often."""
    run_case(6, dtype, 64, 64, [2000, 300], scale=1.5, sink="none")
    run_case(7, dtype, 20, 64, [2000], scale=1.5, sink="normal")


@pytest.mark.parametrize("dtype", DTYPES)
def test_interleaved_layers(dtype):
    run_case(8, dtype, 64, 64, [500, 90], layers=3)
    run_case(9, dtype, 64, 8, [500, 90], layers=2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_split_over_the_gpu(dtype):
    """Long sequences: every CTA works on a part, alone and beside short ones."""
    run_case(21, dtype, 64, 64, [40000], want_lse=False)
    run_case(22, dtype, 64, 64, [20011, 1, 9000, 64, 33333])
    run_case(23, dtype, 128, 128, [20011, 5])
    run_case(24, dtype, 8, 16, [50001])


@pytest.mark.parametrize("dtype", DTYPES)
def test_more_queries_than_sms(dtype):
    rng = np.random.default_rng(2)
    run_case(31, dtype, 16, 64, [int(n) for n in rng.integers(0, 300, 400)], pad=3)
    run_case(32, dtype, 64, 64, [1] * 700)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,most", [(1, 2048), (7, 1000), (10, 2000), (15, 700), (20, 2048), (33, 900),
                                    (50, 300), (66, 2000), (120, 256), (152, 200)])
def test_small_batches_one_cluster_per_item(dtype, B, most):
    """One CTA per item up to four tiles, else clusters of 8, 4 and 2 by the batch; lengths from
    zero to the bound, so some CTAs of a cluster have no tile; padded queries among them."""
    rng = np.random.default_rng(B)
    lens = [most] + [int(n) for n in rng.integers(0, most + 1, B - 1)]
    run_case(100 + B, dtype, 64, 64, lens, pad=1 if B < 100 else 0)
    run_case(200 + B, dtype, 7, 24, lens[:B // 2 + 1], sink="none", rope=False, tail=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,B,sink", [(64, 1, "inf"), (33, 2, "large"), (20, 16, "none"), (3, 25, "normal"),
                                      (100, 3, "inf"), (128, 12, "normal"), (64, 60, "none")])
def test_clusters_weigh_their_parts(dtype, H, B, sink):
    rng = np.random.default_rng(B)
    lens = [0, 2048] + [int(x) for x in rng.integers(0, 2049, B)]  # some parts have no rows
    run_case(50 + B, dtype, H, 64, lens[:B] if B > 2 else lens[1:1 + B], sink=sink, spread=4.0)
    run_case(51 + B, dtype, H, 16, [min(n, 600) for n in lens[1:1 + B]], sink=sink, rope=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 24, 48, 192])
def test_long_sequences_in_small_pages(dtype, page):
    run_case(300 + page, dtype, 64, page, [9001, 200, 4097])


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_head_groups_in_clusters_and_windows(dtype):
    run_case(41, dtype, 128, 64, [700, 3, 1200])
    run_case(42, dtype, 100, 16, [2000, 1500], window=333)
    run_case(43, dtype, 64, 64, [90000], window=20000)


@pytest.mark.parametrize("dtype", DTYPES)
def test_pages_beyond_four_gigabytes(dtype):
    """Offsets of pages and rows that pass 32 bits, written by the append, read by the attention."""
    import csa2_compressed_sparse_gb300 as csa2
    width = 512 if dtype == BF16 else 528
    size = 64 * width * (2 if dtype == BF16 else 1)
    n_pages = (5 << 30) // size
    data = torch.empty((n_pages, 64, width), dtype=torch.bfloat16 if dtype == BF16 else torch.uint8,
                       device="cuda")
    n = 700
    pages = [n_pages - 1 - i for i in range(0, 11)]
    table = torch.tensor([pages], dtype=torch.int32, device="cuda")
    kv = torch.randn((n, 512), device="cuda").bfloat16()
    csa2.csa2_paged_append(kv, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                           torch.zeros(1, dtype=torch.int64, device="cuda"),
                           paged(data, table, dtype))
    got = get(data, table, 0, 0, n)
    check_rows(got, kv, None, dtype, False)
    q = torch.randn((1, 64, 512), device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty((1, 64), device="cuda")
    csa2.csa2_paged_attn(q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         torch.tensor([n - 1], device="cuda"), paged(data, table, dtype), out,
                         workspace(1, 64, n), max_rows=n, lse=lse)
    csa2.csa2_device_status()
    check_query(out[0], lse[0], q[0], decode(got, dtype), None, 512 ** -0.5, n - 1, False)


def test_positions_far_beyond_the_cache_and_below_zero():
    """Positions at the ends of int64: clipped and reported, or empty; nothing else is touched."""
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(3), BF16, 64, [100])
    x = torch.randn((100, 512), device="cuda").bfloat16()
    put(data, table, 0, x)
    q = torch.randn((2, 64, 512), device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty((2, 64), device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    pos = torch.tensor([2 ** 63 - 1, -2 ** 63], device="cuda")
    for ratio in (1, 3):
        with pytest.raises(csa2.Csa2Error) as e:
            csa2.csa2_paged_attn(q, seq, pos, paged(data, table, BF16), out, workspace(2, 64, 100),
                                 max_rows=100, lse=lse, ratio=ratio)
            csa2.csa2_device_status()
        assert e.value.status == 4
        check_query(out[0], lse[0], q[0], x.double(), None, 512 ** -0.5, 0, False)
        assert bool((out[1] == 0).all()) and bool((lse[1] == -float("inf")).all())


def test_a_step_on_another_stream_and_a_shared_workspace_in_order():
    """Calls that follow one another on one stream may share a workspace."""
    import csa2_compressed_sparse_gb300 as csa2
    lens = [6000, 31]
    g = torch.Generator(device="cuda").manual_seed(2)
    data, table, _ = pool(np.random.default_rng(2), BF16, 64, lens)
    for b, n in enumerate(lens):
        put(data, table, b, torch.randn((n, 512), generator=g, device="cuda").bfloat16())
    ws = workspace(2, 64, 6000)
    seq = torch.arange(2, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lens, device="cuda") - 1
    qs = [torch.randn((2, 64, 512), generator=g, device="cuda").bfloat16() for _ in range(6)]
    outs = [torch.empty_like(q) for q in qs]
    lses = [torch.empty((2, 64), device="cuda") for _ in qs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for q, out, lse in zip(qs, outs, lses):
        csa2.csa2_paged_attn(q, seq, pos, paged(data, table, BF16), out, ws, max_rows=6000, lse=lse,
                             stream=st)
    csa2.csa2_device_status(st)
    for q, out, lse in zip(qs, outs, lses):
        for b, n in enumerate(lens):
            x = decode(get(data, table, b, 0, n), BF16)
            check_query(out[b], lse[b], q[b], x, None, 512 ** -0.5, n - 1, False)


def test_matches_the_sparse_attention():
    """Window-free csa2_sparse_attn with every row selected is the same computation: both are
    within their tolerances of it (this one's is checked by run_case), so they differ by at most
    both."""
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(5)
    n, page = 500, 64
    data, table, _ = pool(np.random.default_rng(5), BF16, page, [n])
    x = torch.randn((n, 512), generator=g, device="cuda").bfloat16()
    put(data, table, 0, x)
    q = torch.randn((1, 64, 512), generator=g, device="cuda").bfloat16()
    sink = torch.randn((64,), generator=g, device="cuda")
    out = torch.empty((1, 64, 512), dtype=torch.bfloat16, device="cuda")
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    csa2.csa2_paged_attn(q, seq, torch.tensor([n - 1], device="cuda"), paged(data, table, BF16),
                         out, workspace(1, 64, n), max_rows=n, sink=sink)
    # the sparse call's window: the last 128 rows; the selection: the others
    ring = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda")
    p = torch.arange(n - 128, n, device="cuda")
    ring[0, p % 128] = x[p]
    sel = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
    sel[0, :n - 128] = torch.arange(n - 128, device="cuda")
    ref = torch.empty_like(out)
    csa2.csa2_sparse_attn(q, seq, torch.tensor([n - 1], device="cuda"), csa2.Swa(ring), x,
                          torch.zeros(1, dtype=torch.int64, device="cuda"), sel, sink, ref)
    csa2.csa2_device_status()
    s = 512 ** -0.5 * q[0].double() @ x.double().T
    w = torch.exp(s) / (torch.exp(s).sum(1) + torch.exp(sink.double()))[:, None]
    A = w @ x.double().abs()
    tol = 2 * (2 * 2.0 ** -8 * 1.02 * A + 2.0 ** -8 * ref[0].double().abs())
    assert bool(((out - ref)[0].double().abs() <= tol).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_pages_rows_and_sequences_are_reported(dtype):
    """Page ids outside the pool, a sequence outside the table and rows beyond the bound raise
    the bounds fault; the rows are left out, everything else is computed."""
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(9)
    n, page, H = 400, 32, 64
    data, table, _ = pool(np.random.default_rng(9), dtype, page, [n, n])
    for b in range(2):
        put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    good = table.clone()
    table[0, 3] = data.shape[0]
    table[0, 7] = -5
    q = torch.randn((3, H, 512), generator=g, device="cuda").bfloat16()
    seq = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([n - 1, n - 1, 10], device="cuda")
    out = torch.full((3, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, H), 7.0, device="cuda")
    with pytest.raises(csa2.Csa2Error) as e:
        csa2.csa2_paged_attn(q, seq, pos, paged(data, table, dtype), out, workspace(3, H, n),
                             max_rows=n, lse=lse)
        csa2.csa2_device_status()
    assert e.value.status == 4
    keep = [j for j in range(n) if j // page not in (3, 7)]
    x = decode(get(data, good, 0, 0, n), dtype)[keep]
    check_query(out[0], lse[0], q[0], x, None, 512 ** -0.5, n - 1, False)
    check_query(out[1], lse[1], q[1], decode(get(data, good, 1, 0, n), dtype), None, 512 ** -0.5,
                n - 1, False)
    assert bool((out[2] == 7.0).all()) and bool((lse[2] == 7.0).all())
    with pytest.raises(csa2.Csa2Error) as e:
        csa2.csa2_paged_attn(q[:2], seq[:2], pos[:2], paged(data, good, dtype), out[:2],
                             workspace(2, H, 100), max_rows=100, lse=lse[:2])
        csa2.csa2_device_status()
    assert e.value.status == 4
    for b in range(2):
        check_query(out[b], lse[b], q[b], decode(get(data, good, b, 0, 100), dtype), None,
                    512 ** -0.5, n - 1, False)
    csa2.csa2_device_status()  # the flag is cleared


def test_the_same_call_twice_gives_the_same_bits():
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(10)
    lens = [9000, 17, 4000]
    data, table, _ = pool(np.random.default_rng(1), BF16, 64, lens)
    for b, n in enumerate(lens):
        put(data, table, b, torch.randn((n, 512), generator=g, device="cuda").bfloat16())
    q = torch.randn((3, 64, 512), generator=g, device="cuda").bfloat16()
    seq = torch.arange(3, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lens, device="cuda") - 1
    ws = workspace(3, 64, 9000)
    outs = []
    for _ in range(3):
        out = torch.empty((3, 64, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((3, 64), device="cuda")
        csa2.csa2_paged_attn(q, seq, pos, paged(data, table, BF16), out, ws, max_rows=9000, lse=lse)
        outs.append((out, lse))
    csa2.csa2_device_status()
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_a_window_of_any_size_beyond_the_rows_is_no_window():
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(12)
    n = 5000
    data, table, _ = pool(np.random.default_rng(2), BF16, 64, [n])
    put(data, table, 0, torch.randn((n, 512), generator=g, device="cuda").bfloat16())
    q = torch.randn((1, 64, 512), generator=g, device="cuda").bfloat16()
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([n - 1], device="cuda")
    outs = []
    for window in (0, n, n + 1, 1 << 31, (1 << 63) - 62, (1 << 63) - 1):
        out = torch.empty_like(q)
        csa2.csa2_paged_attn(q, seq, pos, paged(data, table, BF16), out, workspace(1, 64, n),
                             max_rows=n, window=window)
        outs.append(out)
    csa2.csa2_device_status()
    for out in outs[1:]:  # the rows are shared out in the same way, too
        assert torch.equal(out, outs[0])


def test_a_page_table_beyond_two_to_the_31_rows():
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(13)
    data, small, _ = pool(np.random.default_rng(2), BF16, 1024, [3000])
    x = torch.randn((3000, 512), generator=g, device="cuda").bfloat16()
    put(data, small, 0, x)
    table = torch.full((1, (1 << 21) + 1), -1, dtype=torch.int32, device="cuda")
    table[:, :small.shape[1]] = small
    q = torch.randn((1, 64, 512), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    csa2.csa2_paged_attn(q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         torch.tensor([2999], device="cuda"), paged(data, table, BF16), out,
                         workspace(1, 64, 0x7FFFFF00))
    csa2.csa2_device_status()
    check_query(out[0], None, q[0], x.double(), None, 512 ** -0.5, 2999, False)


# ---- append ---------------------------------------------------------------------------------

def check_rows(got, x, pos, dtype, rope):
    """got: stored rows; x: the tokens [n, 512] bf16; pos their positions."""
    ref = x.double()
    slack = torch.zeros_like(ref)
    if rope:
        ref = rotated(ref, pos, 1)
        s = x.double()[:, 448:].abs().reshape(-1, 32, 2).sum(-1).repeat_interleave(2, 1)
        slack[:, 448:] = 2.0 ** -20 * s
    if dtype == BF16:
        if not rope:
            assert torch.equal(got.view(torch.int16), x.view(torch.int16))
            return
        assert torch.equal(got[:, :448].contiguous().view(torch.int16),
                           x[:, :448].contiguous().view(torch.int16))
        assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + slack).all())
        return
    g = 128 if dtype == S128 else 32
    top = ref.abs().reshape(ref.shape[0], -1, g).amax(-1)
    loose = slack.reshape(ref.shape[0], -1, g).amax(-1)
    tail = got[:, 512:].contiguous()
    if dtype == S128:
        sc = tail.view(torch.float32).double()
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        # one fp32 rounding (2^-24 relative; 2^-150 among the subnormals)
        assert bool(((sc - want).abs() <= 2.0 ** -23 * want + loose / 448 + 2.0 ** -150).all())
    else:
        e = tail.double() - 127
        sc = torch.exp2(e)
        # the smallest scale that holds the largest value, up to the rotation's rounding
        assert bool((top <= 448 * sc * (1 + 1e-12) + loose).all())
        low = (e > -127) & (top > 0)
        assert bool((top + loose > 224 * sc)[low].all())
        assert bool((tail[top == 0] == 127).all())
    v = decode(got, dtype)
    s = sc.repeat_interleave(g, 1)
    # half a step of E4M3 (2^-4 relative, 2^-10 of the scale below its normal range); the
    # quotient's fp32 rounding moves a tie by 2^-22 at most
    tol = (2.0 ** -4 * ref.abs() + 2.0 ** -10 * s) * (1 + 2.0 ** -20) + slack + 2.0 ** -22 * ref.abs()
    assert bool(((v - ref).abs() <= tol).all())


def run_append(seed, dtype, page, hist, new, ratio=1, rope=True, kv_ld=512, pad=0, layers=0,
               values=None):
    import csa2_compressed_sparse_gb300 as csa2
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    data, table, whole = pool(rng, dtype, page, [h + n for h, n in zip(hist, new)], poison=False,
                              layers=layers)
    whole.copy_(torch.randint(0, 120, whole.shape, generator=g, device="cuda").to(whole.dtype))
    T = sum(new) + pad
    wide = torch.randn((T, kv_ld), generator=g, device="cuda").bfloat16()
    if values is not None:
        wide[:, :512] = values(T, g)
    kv = wide[:, :512]
    before = whole.clone()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    csa2.csa2_paged_append(kv, cu, torch.tensor(hist, dtype=torch.int64, device="cuda"),
                           paged(data, table, dtype),
                           inv_freq=inv_freq().cuda() if rope else None, ratio=ratio)
    csa2.csa2_device_status()
    at = 0
    touched = torch.zeros(data.shape[:2], dtype=torch.bool, device="cuda")
    for b, (h, n) in enumerate(zip(hist, new)):
        if n == 0:
            continue
        j = torch.arange(h, h + n, device="cuda")
        got = get(data, table, b, h, h + n)
        check_rows(got, kv[at:at + n], j * ratio, dtype, rope)
        touched[table[b, j // page].long(), j % page] = True
        at += n
    # every other row of the pool, other layers' pages among them, is as it was
    old = before[:, layers // 2] if layers else before
    assert torch.equal(data[~touched].view(torch.uint8), old[~touched].view(torch.uint8))
    for i in range(layers):
        if i != layers // 2:
            assert torch.equal(whole[:, i].contiguous().view(torch.uint8),
                               before[:, i].contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rope", [True, False])
def test_append_decode_batch(dtype, rope):
    run_append(1, dtype, 64, [0, 63, 64, 1000, 5], [1] * 5, rope=rope)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 24, 64, 256])
def test_append_ragged(dtype, page):
    run_append(page, dtype, page, [0, 7, 300, 0, 20, 1], [130, 0, 1, 700, 0, 33], pad=9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_ratio_strides_layers(dtype):
    run_append(2, dtype, 16, [3, 100], [50, 21], ratio=2, kv_ld=1536)
    run_append(3, dtype, 16, [3, 100], [50, 21], ratio=128, layers=3)
    run_append(4, dtype, 64, [8000], [5], ratio=128, kv_ld=520)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_many_tokens(dtype):
    run_append(5, dtype, 64, [0, 11], [9001, 3000])


@pytest.mark.parametrize("dtype", [S128, E8M0])
def test_append_quantiser_edges(dtype):
    """All-zero groups, values at the scales' borders, tiny and large magnitudes."""
    def values(T, g):
        x = torch.randn((T, 512), generator=g, device="cuda")
        x = x * torch.exp2(torch.randint(-30, 30, (T, 1), generator=g, device="cuda").float())
        x[0] = 0.0
        x[1, 128:256] = 0.0
        x[2] = 448.0 * 2.0 ** -3
        x[3] = 450.0
        x[4] = 2.0 ** -120
        x[5, ::2] = 1e-6
        x[6] = 2.0 ** 100
        x[7, :] = 0.0
        x[7, 511] = 1.0
        return x.bfloat16()
    run_append(6, dtype, 64, [0], [40], rope=False, values=values)
    run_append(7, dtype, 64, [0, 5], [40, 60], values=values)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_skips_and_reports_rows_without_a_page(dtype):
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(4), dtype, 16, [32, 32], poison=False)
    table[1, 0] = data.shape[0]
    kv = torch.randn((40, 512), device="cuda").bfloat16()
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    with pytest.raises(csa2.Csa2Error) as e:
        # sequence 0 begins before its first row, sequence 1's first page is outside the pool
        csa2.csa2_paged_append(kv, cu, torch.tensor([-3, 0], device="cuda"),
                               paged(data, table, dtype))
        csa2.csa2_device_status()
    assert e.value.status == 4
    check_rows(get(data, table, 0, 0, 17), kv[3:20], None, dtype, False)
    check_rows(get(data, table, 1, 16, 20), kv[36:40], None, dtype, False)
    before = data.clone()
    with pytest.raises(csa2.Csa2Error) as e:
        # rows in the table's unmapped last column and past it; nothing for sequence 1
        csa2.csa2_paged_append(kv[:20], torch.tensor([0, 20, 20], dtype=torch.int32, device="cuda"),
                               torch.tensor([16 * table.shape[1] - 4, 0], device="cuda"),
                               paged(data, table, dtype))
        csa2.csa2_device_status()
    assert e.value.status == 4 and torch.equal(data.view(torch.uint8), before.view(torch.uint8))


# ---- together -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_steps_in_a_graph(dtype):
    """A decode step (append the new token's row, then attend over everything) captured once and
    replayed: positions advance on the device, each step sees the rows of the steps before."""
    import csa2_compressed_sparse_gb300 as csa2
    B, H, page, steps = 3, 64, 16, 6
    hist = [5, 300, 31]
    g = torch.Generator(device="cuda").manual_seed(3)
    data, table, _ = pool(np.random.default_rng(3), dtype, page, [h + steps for h in hist])
    rows = [torch.randn((h + steps, 512), generator=g, device="cuda").bfloat16() for h in hist]
    f = inv_freq().cuda()
    c = paged(data, table, dtype)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(hist)]), dtype=torch.int32, device="cuda")
    csa2.csa2_paged_append(torch.cat([r[:h] for r, h in zip(rows, hist)]), cu,
                           torch.zeros(B, dtype=torch.int64, device="cuda"), c, inv_freq=f)
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    seq = torch.arange(B, dtype=torch.int32, device="cuda")
    pos = torch.tensor(hist, device="cuda")
    kv = torch.empty((B, 512), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((B, H, 512), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    lse = torch.empty((B, H), device="cuda")
    mx = 2000  # a bound, as a server captures it
    ws = workspace(B, H, mx)

    def step():
        csa2.csa2_paged_append(kv, one, pos, c, inv_freq=f)
        csa2.csa2_paged_attn(q, seq, pos, c, out, ws, max_rows=mx, lse=lse, inv_freq=f)

    graph = torch.cuda.CUDAGraph()
    kv.zero_()
    q.zero_()
    with torch.cuda.graph(graph):
        step()
        pos += 1
    pos.copy_(torch.tensor(hist, device="cuda"))
    for t in range(steps):
        kv.copy_(torch.stack([r[h + t] for r, h in zip(rows, hist)]))
        q.copy_(torch.randn((B, H, 512), generator=g, device="cuda").bfloat16())
        graph.replay()
        csa2.csa2_device_status()
        for b in range(B):
            n = hist[b] + t + 1
            got = get(data, table, b, 0, n)
            check_rows(got, rows[b][:n], torch.arange(n, device="cuda"), dtype, True)
            check_query(out[b], lse[b], q[b], decode(got, dtype), None, 512 ** -0.5, n - 1, True)


def test_two_streams_with_a_workspace_each():
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i, st in enumerate(s):
        with torch.cuda.stream(st):
            run_case(60 + i, BF16, 64, 64, [5000, 40], stream=st if i else None)


def test_the_binding_refuses_what_the_call_cannot_read():
    import csa2_compressed_sparse_gb300 as csa2
    data, table, _ = pool(np.random.default_rng(4), BF16, 16, [32])
    c = paged(data, table, BF16)
    q = torch.zeros((1, 64, 512), dtype=torch.bfloat16, device="cuda")
    seq = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.empty_like(q)
    ok = dict(q=q, q_seq=seq, q_pos=pos, cache=c, out=out)
    for kw in (dict(q=q.half()), dict(q=q.cpu()), dict(q_seq=seq.long()), dict(q_pos=pos.int()),
               dict(out=out[:, :32]), dict(out=out.transpose(1, 2)), dict(sink=q[0, :, 0]),
               dict(lse=torch.empty((1, 63), device="cuda")),
               dict(inv_freq=torch.empty(31, device="cuda")), dict(q=q.transpose(1, 2))):
        with pytest.raises(ValueError):
            csa2.csa2_paged_attn(**{**ok, **kw})
    kv = torch.zeros((2, 512), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(kv=kv.float()), dict(kv=kv.cpu()), dict(kv=kv[:, :256]), dict(kv=kv.T),
               dict(cu_seqlens=cu[:1]), dict(cu_seqlens=cu.long()), dict(start_row=pos.int())):
        with pytest.raises(ValueError):
            csa2.csa2_paged_append(**{**dict(kv=kv, cu_seqlens=cu, start_row=pos, cache=c), **kw})
    for bad in (data[:, :, :256], data.transpose(0, 1), data[:, ::2], data[:0]):
        with pytest.raises(ValueError):
            csa2.Paged(bad, table)
    with pytest.raises(ValueError):
        csa2.Paged(data, table[:, ::2])
