"""The sparse attention's running maximum at its edges: sinks of -inf on some heads, sinks far
below the scores or at the ends of fp32, and heads whose scores are NaN.  Heads of one warp then
differ in whether they have a maximum, which must not part the warp.

Tolerances: outputs as in test_gpu_paged.py (the same products, weights rounded to bf16, numerator
and normaliser).  lse is the logarithm of a sum of weights that are rounded to bf16 (each off by
2^-8 at most, and so is the sum): 1.01 * 2^-8 besides the scores' tau, 2^-19 and 2^-22 |lse|."""
import numpy as np
import pytest
import torch

from test_gpu_paged import check_query

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# queries: a pair of CTAs each, one CTA each, CTAs that go on from query to query
LAYOUTS = {"pair": 3, "one": 100, "persistent": 200}


def attend(Q, nsel, sink, scale, seed, spoil=None):
    """Random window and selection; returns what check_query needs."""
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = 900
    x = torch.randn((n, 512), generator=g, device="cuda").bfloat16()
    q = torch.randn((Q, 64, 512), generator=g, device="cuda").bfloat16()
    if spoil is not None:
        q[:, spoil] = float("nan")
    ring = torch.empty((1, 128, 512), dtype=torch.bfloat16, device="cuda")
    p = torch.arange(n - 128, n, device="cuda")
    ring[0, p % 128] = x[p]
    sel = torch.argsort(torch.rand((Q, n - 128), generator=g, device="cuda"), 1)[:, :nsel].int()
    sel = sel.sort(1).values.contiguous()
    out = torch.full((Q, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Q, 64), 7.0, device="cuda")
    seq = torch.zeros(Q, dtype=torch.int32, device="cuda")
    pos = torch.full((Q,), n - 1, dtype=torch.int64, device="cuda")
    ws = torch.empty(max(1, csa2.csa2_attn_workspace_size(Q, nsel)), dtype=torch.uint8, device="cuda")
    csa2.csa2_sparse_attn(q, seq, pos, csa2.Swa(ring), x, torch.zeros(1, dtype=torch.int64, device="cuda"),
                          sel, sink, out, lse=lse, scale=scale, ws=ws)
    csa2.csa2_device_status()
    return q, x, p, sel, out, lse


def check(i, heads, q, x, p, sel, out, lse, sink, scale):
    rows = x[torch.cat([p, sel[i].long()])].double()
    sk = None if sink is None else sink[heads]
    check_query(out[i, heads], None, q[i, heads], rows, sk, scale, 899, False)
    qd = q[i, heads].double()
    s = scale * qd @ rows.T
    z = torch.logsumexp(s if sk is None else torch.cat([s, sk.double()[:, None]], 1), 1)
    tau = (512 * 2.0 ** -23 * abs(scale) * (qd.abs() @ rows.abs().T)).amax(1)
    assert bool(((lse[i, heads].double() - z).abs() <=
                 tau + 1.01 * 2.0 ** -8 + 2.0 ** -19 + 2.0 ** -22 * z.abs()).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("nsel", [0, 192, 512])
@pytest.mark.parametrize("scale", [512 ** -0.5, 1.5])
def test_sinks_at_their_edges(layout, nsel, scale):
    big = float(np.finfo(np.float32).max)
    kinds = [-float("inf"), -1e30, 0.5, -1e9, -big, -1e20, big, 3.0, -3e38, 2e38, -3e4]
    sink = torch.tensor(kinds * 6, device="cuda")[:64].contiguous()
    Q = LAYOUTS[layout]
    res = attend(Q, nsel, sink, scale, 3 + nsel)
    # (a sink beyond 2.36e38 takes all the mass, but its lse is 2.36e38: csa2.h)
    heads = torch.arange(64, device="cuda")[sink < 2.3e38]
    assert bool((res[4][:, sink > 2.3e38] == 0).all())
    assert bool((res[5][:, sink > 2.3e38] > 2.35e38).all())
    for i in range(0, Q, 1 if Q < 10 else 33):
        check(i, heads, *res, sink, scale)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("with_sink", [False, True])
def test_a_head_of_nan_queries_leaves_the_others_as_they_are(layout, with_sink):
    Q = LAYOUTS[layout]
    sink = torch.linspace(-2, 2, 64, device="cuda") if with_sink else None
    res = attend(Q, 512, sink, 512 ** -0.5, 9, spoil=21)
    heads = torch.tensor([h for h in range(64) if h != 21], device="cuda")
    out, lse = res[4], res[5]
    assert bool(out[:, 21].isnan().all()) and bool(lse[:, 21].isnan().all())
    for i in range(0, Q, 1 if Q < 10 else 33):
        check(i, heads, *res, sink, 512 ** -0.5)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_no_sink(layout):
    Q = LAYOUTS[layout]
    res = attend(Q, 512, None, 1.5, 10)
    for i in range(0, Q, 1 if Q < 10 else 33):
        check(i, torch.arange(64, device="cuda"), *res, None, 1.5)
