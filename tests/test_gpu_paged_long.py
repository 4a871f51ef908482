"""More rows than the tensor core's sums are good for: its fp32 accumulators cut low bits instead
of rounding them, so a sum of one sign comes out short by 2^-23 of itself at most (and half of
that in the mean) per product of 16 rows.

Every row is one and the same here, so every weight is equal (1, as the running maximum is their
score) and the output is that row whatever their number.  A run of at most 65536 rows is 4096 products: short by 2^-11 at most, and adding up
the runs in fp32 adds 2^-24 per run.  The rows' values are bf16, whose half step is 2^-9 of the
value at least, so the output has to be the row to the bit; lse is the score plus ln n."""
import math

import pytest
import torch

from test_gpu_paged import BF16, DTYPES, E8M0, S128, decode, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def the_row(dtype, g):
    """A cache row whose values, and whose scales, are bf16 values."""
    if dtype == BF16:
        x = torch.rand((1, 512), generator=g, device="cuda") + 0.5
        x[:, 1::2] *= -1
        return x.bfloat16()
    codes = torch.randint(0x30, 0x50, (1, 512), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, 1::2] |= 0x80
    if dtype == S128:
        tail = torch.tensor([[0.5, 1.5, 0.0625, 2.0]], device="cuda").view(torch.uint8)
    else:
        tail = torch.randint(120, 130, (1, 16), generator=g, device="cuda", dtype=torch.uint8)
    return torch.cat([codes, tail], 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [3, 64])
@pytest.mark.parametrize("Q,n", [(152, 65536), (152, 65537), (152, 1048576 + 77), (305, 400000),
                                 (1, 33000000)])
def test_equal_rows_of_any_number_give_the_row(dtype, H, Q, n):
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(n)
    row = the_row(dtype, g)
    page = 4096
    data = row.expand(page, -1).reshape(1, page, -1).contiguous()
    table = torch.zeros((1, -(-n // page)), dtype=torch.int32, device="cuda")  # one page, many times
    x = decode(row, dtype)
    q = (torch.randn((Q, H, 512), generator=g, device="cuda") * 0.02).bfloat16()
    out, lse = torch.empty_like(q), torch.empty((Q, H), device="cuda")
    ws = torch.full((csa2.csa2_paged_attn_workspace_size(Q, H, n),), 0xFF, dtype=torch.uint8, device="cuda")
    csa2.csa2_paged_attn(q, torch.zeros(Q, dtype=torch.int32, device="cuda"),
                         torch.full((Q,), n - 1, device="cuda"), paged(data, table, dtype), out, ws,
                         max_rows=n, lse=lse)
    csa2.csa2_device_status()
    s = 512 ** -0.5 * (q.double() @ x[0])
    assert torch.equal(out, x[0].bfloat16().expand_as(out))
    tau = 512 * 2.0 ** -23 * 512 ** -0.5 * (q.double().abs() @ x[0].abs())
    z = s + math.log(n)
    # a run's sums are at most 1024 additions a thread, each a rounding of 2^-24
    assert bool(((lse.double() - z).abs() <= tau + 2.0 ** -19 + 2.0 ** -22 * z.abs() + 2.0 ** -14).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,order,window", [(64, "rising", 0), (64, "falling", 0), (20, "rising", 200001),
                                            (100, "mixed", 0)])
def test_runs_of_unlike_rows_add_up(dtype, H, order, window):
    """Three pages, many times each, whose scores differ in spread: the runs' maxima differ, in
    either direction.  The rows' multiplicities enter the formula as logarithms.  Tolerances as in
    test_gpu_paged.py, and the cut sums' 2^-11 of the weighted magnitudes."""
    import csa2_compressed_sparse_gb300 as csa2
    from test_gpu_paged import quantised
    g = torch.Generator(device="cuda").manual_seed(H + window)
    page, Q = 4096, 160
    spread = torch.tensor([0.5, 2.0, 8.0], device="cuda")
    x = torch.randn((3, page, 512), generator=g, device="cuda") * spread[:, None, None]
    data = torch.stack([quantised(x[i], dtype) for i in range(3)])
    ids = {"rising": [0] * 25 + [1] * 25 + [2] * 25, "falling": [2] * 25 + [1] * 25 + [0] * 25,
           "mixed": [0, 2, 1] * 25}[order]
    n = 75 * page - 1234
    lo = n - window if window else 0
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    count = torch.zeros((3, page), dtype=torch.float64, device="cuda")
    for i, p in enumerate(ids):
        a, b = max(0, lo - i * page), min(page, n - i * page)
        if b > a:
            count[p, a:b] += 1
    q = torch.randn((Q, H, 512), generator=g, device="cuda").bfloat16()
    sink = torch.randn((H,), generator=g, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((Q, H), device="cuda")
    ws = torch.full((csa2.csa2_paged_attn_workspace_size(Q, H, n),), 0xFF, dtype=torch.uint8, device="cuda")
    csa2.csa2_paged_attn(q, torch.zeros(Q, dtype=torch.int32, device="cuda"),
                         torch.full((Q,), n - 1, device="cuda"), paged(data, table, dtype), out, ws,
                         max_rows=n, window=window, sink=sink, lse=lse)
    csa2.csa2_device_status()
    rows = torch.cat([decode(data[i], dtype) for i in range(3)])
    logs = count.reshape(-1).log()
    for i in (0, 1, 79, 158, 159):
        qd = q[i].double()
        s = 512 ** -0.5 * qd @ rows.T
        tau = (512 * 2.0 ** -23 * 512 ** -0.5 * (qd.abs() @ rows.abs().T)).amax(1)
        z = torch.logsumexp(torch.cat([s + logs, sink.double()[:, None]], 1), 1)
        w = torch.exp(s + logs - z[:, None])
        ref, A = w @ rows, w @ rows.abs()
        tol = (2 * 2.0 ** -8 * 1.01 + 2 * tau + 2.0 ** -19 + 2.0 ** -11)[:, None] * A
        assert bool(((out[i].double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())
        assert bool(((lse[i].double() - z).abs() <=
                     tau + 2.0 ** -14 + 2.0 ** -19 + 2.0 ** -22 * z.abs()).all())
