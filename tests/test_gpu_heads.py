"""csa2_qk_norm_rope against its formula in 64 bits.

Tolerance.  The sum of D <= 512 squares carries at most D roundings of 2^-24 of it, its root and the
products a few more: a normed value is off by at most 2^-15 of itself.  A rotated one, y0 c - y1 s,
adds the angle's rounding (|angle| <= pi: pi 2^-24), sine and cosine (2 units: 2^-22), three
roundings and the factor's: together below 2^-15 (|y0| + |y1|) |factor| with the norm's.  Then the
result is rounded to bf16, 2^-8 of it (1 + 2^-15 for the value that is rounded)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PAIRS, HALVES = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def freq(n, theta=160000.0):
    return torch.tensor(theta ** (-np.arange(n) / max(1, n)), dtype=torch.float32, device="cuda")


def ref(x, w, norm, eps, pos, f, r0, layout, factor):
    """(value, error bound) in 64 bits."""
    y = x.double()
    if norm:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            y = y * w.double()
    n = f.numel() if f is not None else 0
    tol = y.abs() * 2.0 ** -15
    if n:
        a = pos.double()[:, None, None] * f.double()
        a0, a1 = (slice(r0, r0 + 2 * n, 2), slice(r0 + 1, r0 + 2 * n, 2)) if layout == PAIRS else \
            (slice(r0, r0 + n), slice(r0 + n, r0 + 2 * n))
        e, o = y[..., a0].clone(), y[..., a1].clone()
        y[..., a0] = (e * a.cos() - o * a.sin()) * factor
        y[..., a1] = (e * a.sin() + o * a.cos()) * factor
        tol[..., a0] = tol[..., a1] = (e.abs() + o.abs()) * abs(factor) * 2.0 ** -15
    return y, tol + y.abs() * 2.0 ** -8 * (1 + 2.0 ** -15) + 1e-38


def check(out, x, *args):
    y, tol = ref(x, *args)
    err = (out.double() - y).abs()
    assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.3g} x its tolerance"


def run(seed, T, H, K, D, R, layout, r0=None, factor=1.0, norm=(True, True), weights=(True, True), eps=1e-6,
        far=1 << 20, spread=1.0, stream=None):
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(seed)
    r0 = D - R if r0 is None else r0
    x = (spread * torch.randn((T, H + K, D), generator=g, device="cuda")).bfloat16()
    w = [1 + 0.3 * torch.randn((D,), generator=g, device="cuda") if on else None for on in weights]
    pos = torch.randint(0, far, (T,), generator=g, device="cuda")
    f = freq(R // 2) if R else None
    q, k = x[:, :H], x[:, H:] if K else None
    qo = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T, K, D), 7.0, dtype=torch.bfloat16, device="cuda") if K else None
    torch.cuda.synchronize()
    csa2.csa2_qk_norm_rope(q, qo, pos, f, k=k, k_out=ko, q_norm=norm[0], k_norm=norm[1], q_norm_w=w[0],
                           k_norm_w=w[1] if K else None, eps=eps, rope_dim0=r0, layout=layout,
                           factor=factor, stream=stream)
    torch.cuda.synchronize()
    csa2.csa2_device_status()
    check(qo, q, w[0], norm[0], eps, pos, f, r0, layout, factor)
    if K:
        check(ko, k, w[1], norm[1], eps, pos, f, r0, layout, factor)


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("D,R", [(512, 64), (512, 512), (128, 64), (64, 64), (192, 64), (256, 16), (136, 48),
                                 (8, 0), (24, 16), (504, 496), (264, 144)])
def test_widths_and_layouts(layout, D, R):
    run(D + R + layout, 37, 5, 2, D, R, layout)


@pytest.mark.parametrize("T,H,K", [(1, 1, 0), (1, 64, 1), (3, 128, 3), (65, 7, 1), (1001, 64, 1), (5000, 2, 2),
                                   (700, 33, 16), (2, 1024, 1)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
def test_tokens_and_heads(T, H, K, layout):
    run(T + H, T, H, K, 128, 64, layout)


@pytest.mark.parametrize("T,H,K,D", [(40, 1023, 5, 512), (600, 64, 1, 512), (700, 129, 17, 512), (1500, 128, 1, 512),
                                     (5000, 32, 8, 128), (3001, 30, 3, 64), (9000, 5, 0, 256)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
def test_rows_dealt_to_warps(T, H, K, D, layout):
    """However many rows a warp takes of a token, each is done once (in place a second time would show)."""
    run(T, T, H, K, D, 64, layout)
    import csa2_compressed_sparse_gb300 as csa2
    x = torch.randn((T, H + K, D), device="cuda").bfloat16()
    y, pos, f = torch.empty_like(x), torch.arange(T, device="cuda"), freq(32)
    k = (x[:, H:], y[:, H:]) if K else (None, None)
    csa2.csa2_qk_norm_rope(x[:, :H], y[:, :H], pos, f, k=k[0], k_out=k[1], layout=layout, factor=1.25)
    csa2.csa2_qk_norm_rope(x[:, :H], x[:, :H], pos, f, k=k[0], k_out=k[0], layout=layout, factor=1.25)
    assert torch.equal(x, y)


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("r0", [0, 8, 64, 320])
def test_the_rotated_part_may_lie_anywhere(layout, r0):
    run(r0, 40, 3, 1, 384, 64, layout, r0=r0)


@pytest.mark.parametrize("norm,weights", [((True, True), (False, True)), ((False, True), (False, False)),
                                          ((True, False), (True, False)), ((False, False), (False, False))])
def test_norms_and_weights(norm, weights):
    run(3, 50, 9, 2, 512, 64, PAIRS, norm=norm, weights=weights)
    run(4, 50, 9, 2, 128, 64, HALVES, norm=norm, weights=weights, factor=-1.5)


@pytest.mark.parametrize("spread", [1e-6, 1e-30, 1e15])
def test_small_and_large_values(spread):
    """eps decides where the values are far below it; the square of 1e15 stays within fp32."""
    run(5, 20, 4, 1, 512, 64, PAIRS, spread=spread)
    run(6, 20, 4, 1, 64, 32, HALVES, spread=spread, factor=1.25)


def test_a_zero_row_stays_zero_and_nan_stays_in_its_row():
    import csa2_compressed_sparse_gb300 as csa2
    x = torch.randn((4, 3, 128), device="cuda").bfloat16()
    x[1, 1] = 0
    x[2, 0, 5] = float("nan")
    x[3, 2, 100] = float("inf")
    out = torch.empty_like(x)
    csa2.csa2_qk_norm_rope(x, out, torch.arange(4, device="cuda"), freq(32))
    assert bool((out[1, 1] == 0).all())
    assert bool(out[2, 0].isnan().all()) and bool(out[3, 2, 100:102].isnan().all())
    rest = torch.ones((4, 3), dtype=torch.bool, device="cuda")
    rest[2, 0] = rest[3, 2] = False
    assert bool(out[rest].isfinite().all())


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
def test_positions_of_any_size_and_sign(layout):
    """The phase is exact modulo a turn: positions near the ends of int64 against integer arithmetic."""
    import csa2_compressed_sparse_gb300 as csa2
    from fractions import Fraction
    pos = [0, 1, -1, 2 ** 40 + 3, 2 ** 62 + 12345, -2 ** 63, 2 ** 63 - 1]
    f = freq(4)
    # theta / 2 pi to 64 binary places, as the library keeps it, from the 64-bit product
    turn = [int((float(t) * 0.15915494309189535) % 1.0 * 2.0 ** 64) for t in f.tolist()]
    x = torch.zeros((len(pos), 1, 8), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((len(pos), 1, 16), dtype=torch.bfloat16, device="cuda")
    first = slice(8, 16, 2) if layout == PAIRS else slice(8, 12)
    second = slice(9, 16, 2) if layout == PAIRS else slice(12, 16)
    x[..., first] = 1
    out = torch.empty_like(x)
    if layout == HALVES:  # halves want 16 dims: eight pairs, of which four are checked
        f = torch.cat([f, f])
        turn = turn + turn
        x = torch.zeros((len(pos), 1, 16), dtype=torch.bfloat16, device="cuda")
        x[..., :8] = 1
        first, second = slice(0, 8), slice(8, 16)
    csa2.csa2_qk_norm_rope(x, out, torch.tensor(pos, device="cuda"), f, q_norm=False, layout=layout)
    for i, p in enumerate(pos):
        for k in range(len(turn)):
            a = 2 * np.pi * float(Fraction((p * turn[k]) % 2 ** 64, 2 ** 64))
            assert abs(float(out[i, 0, first][k]) - np.cos(a)) <= 2.0 ** -8 + 2.0 ** -20
            assert abs(float(out[i, 0, second][k]) - np.sin(a)) <= 2.0 ** -8 + 2.0 ** -20


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("D,T", [(512, 300), (64, 50), (128, 9)])
def test_in_place(layout, D, T):
    import csa2_compressed_sparse_gb300 as csa2
    x = torch.randn((T, 12, D), device="cuda").bfloat16()
    y = x.clone()
    pos = torch.arange(T, device="cuda") * 77
    f = freq(16)
    csa2.csa2_qk_norm_rope(y[:, :9], y[:, :9], pos, f, k=y[:, 9:], k_out=y[:, 9:], layout=layout)
    check(y, x, None, True, 1e-6, pos, f, D - 32, layout, 1.0)


def test_strides():
    """Heads before tokens, gaps between both, outputs likewise; what lies between is left alone."""
    import csa2_compressed_sparse_gb300 as csa2
    T, H, D = 33, 6, 128
    x = torch.randn((H, T, D + 8), device="cuda").bfloat16()
    o = torch.full((T, H, D + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, device="cuda")
    f = freq(32)
    xv = x[:, :, 8:].transpose(0, 1)
    csa2.csa2_qk_norm_rope(xv, o[..., 8:8 + D], pos, f)
    check(o[..., 8:8 + D], xv, None, True, 1e-6, pos, f, D - 64, PAIRS, 1.0)
    assert bool((o[..., :8] == 3).all()) and bool((o[..., 8 + D:] == 3).all())
    one = torch.randn((T, 1, D), device="cuda").bfloat16()
    csa2.csa2_qk_norm_rope(one.expand(T, H, D), o[..., 8:8 + D], pos, f)  # one head for all
    check(o[..., 8:8 + D], one.expand(T, H, D), None, True, 1e-6, pos, f, D - 64, PAIRS, 1.0)


def test_tensors_beyond_4_gib():
    import csa2_compressed_sparse_gb300 as csa2
    T, H, D = 4200, 1024, 512  # 4.4 GB
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, H, D), device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda")
    f = freq(32)
    csa2.csa2_qk_norm_rope(x, x, pos, f)
    y = x[-3:].clone()
    del x
    assert bool((y.double().square().mean(-1) - 1).abs().max() < 0.02)


def test_another_stream_and_a_graph():
    import csa2_compressed_sparse_gb300 as csa2
    s = torch.cuda.Stream()
    run(9, 100, 8, 1, 512, 64, PAIRS, stream=s)
    x = torch.randn((64, 8, 512), device="cuda").bfloat16()
    out = torch.empty_like(x)
    pos, f = torch.arange(64, device="cuda"), freq(32)
    g = torch.cuda.CUDAGraph()
    csa2.csa2_qk_norm_rope(x, out, pos, f)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        csa2.csa2_qk_norm_rope(x, out, pos, f)
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, device="cuda"))
        pos.add_(1000)
        g.replay()
        torch.cuda.synchronize()
        check(out, x, None, True, 1e-6, pos, f, 448, PAIRS, 1.0)


def test_refusals_of_the_binding():
    import csa2_compressed_sparse_gb300 as csa2
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos, f = torch.zeros(4, dtype=torch.int64, device="cuda"), freq(8)
    for kw in (dict(q=x.float()), dict(q_out=x[:3]), dict(pos=pos.int()), dict(pos=pos[:3]),
               dict(inv_freq=f.double()), dict(q=x.transpose(1, 2)), dict(k_out=x), dict(k=x),
               dict(q_norm_w=f), dict(k_norm_w=f)):
        a = dict(q=x, q_out=torch.empty_like(x), pos=pos, inv_freq=f)
        a.update(kw)
        with pytest.raises(ValueError):
            csa2.csa2_qk_norm_rope(**a)
    with pytest.raises(csa2.Csa2Error):  # rotated dims beyond the head
        csa2.csa2_qk_norm_rope(x, torch.empty_like(x), pos, freq(40))
