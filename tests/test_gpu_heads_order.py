"""csa2_qk_norm_rope directly in front of the sparse step, whose calls read queries and window rows before
the kernel in front of them has finished.

Each chain runs call after call and with the stream drained between the calls; the same buffers take other
values in each pass, so what they hold before is the answer of another pass.  A call's results depend on its
inputs alone, to the bit, so both runs have to be equal to the bit."""
import numpy as np
import pytest
import torch

from test_gpu_paged import check_query, inv_freq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def inputs(T, H, D, passes, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((passes, T, H, D), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("name", ["csa2_reuse_attn", "csa2_sparse_attn"])
@pytest.mark.parametrize("T", [3, 100, 700])
def test_queries_and_window_of_the_attention(name, T):
    """A reused selection: nothing is launched between the norm and the attention."""
    import csa2_compressed_sparse_gb300 as csa2
    n = 6
    x = inputs(T, 65, 512, n, T)
    pos, f = torch.arange(T, device="cuda"), inv_freq().cuda()
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    q = torch.zeros((T, 64, 512), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((T, 1, 512), dtype=torch.bfloat16, device="cuda")
    swa = csa2.Swa(k.view(T, 512), csa2.SWA_LINEAR, lin_base=zero, lin_pos0=zero)

    def step(i, out, drain=False):
        csa2.csa2_qk_norm_rope(x[i, :, :64], q, pos, f, k=x[i, :, 64:], k_out=k)
        if drain:
            csa2.csa2_device_status()
        getattr(csa2, name)(q, seq, pos, swa, None, None, None, None, out)
        if drain:
            csa2.csa2_device_status()

    ref = torch.zeros((n, T, 64, 512), dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        step(i, ref[i], drain=True)
        for t in {0, T // 2, T - 1}:
            check_query(ref[i, t], None, q[t], k[max(0, t - 127):t + 1, 0].double(), None, 512 ** -0.5, t, False)
    for _ in range(5):
        out = torch.zeros_like(ref)
        torch.cuda.synchronize()
        for i in range(n):
            step(i, out[i])
        csa2.csa2_device_status()
        assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(ref)
    with torch.cuda.graph(g):
        for i in range(n):
            step(i, out[i])
    for _ in range(3):
        out.zero_()
        g.replay()
        csa2.csa2_device_status()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("Q", [2, 64])
def test_queries_of_the_indexer(Q):
    import csa2_compressed_sparse_gb300 as csa2
    n, rows, k = 6, 5000, 64
    x = inputs(Q, 64, 128, n, Q)
    g = torch.Generator(device="cuda").manual_seed(1)
    index_k = torch.randn((rows, 128), generator=g, device="cuda").bfloat16()
    w = torch.randn((Q, 64), generator=g, device="cuda")
    pos = torch.full((Q,), rows - 1, device="cuda")
    f = torch.tensor(160000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device="cuda")
    seq, zero = torch.zeros(Q, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    iq = torch.zeros((Q, 64, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(csa2.csa2_index_topk_workspace_size(Q, 64, rows, k), dtype=torch.uint8, device="cuda")

    def chain(drain):
        sel = torch.zeros((n, Q, k), dtype=torch.int32, device="cuda")
        scores = torch.zeros((n, Q, k), device="cuda")
        torch.cuda.synchronize()
        for i in range(n):
            csa2.csa2_qk_norm_rope(x[i], iq, pos, f, layout=csa2.ROPE_HALVES)
            if drain:
                csa2.csa2_device_status()
            csa2.csa2_index_topk(iq, w, index_k, zero, seq, pos, 1, k, rows, sel[i], ws, sel_scores=scores[i])
            if drain:
                csa2.csa2_device_status()
        csa2.csa2_device_status()
        return sel, scores

    ref = chain(True)
    assert not torch.equal(ref[0][0], ref[0][1])
    for _ in range(5):
        got = chain(False)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("layout", [0, 1])
def test_keys_alone_are_as_with_queries(layout):
    import csa2_compressed_sparse_gb300 as csa2
    x = inputs(50, 7, 192, 1, 3)[0]
    pos = torch.arange(50, device="cuda") * 1001
    f = torch.tensor(160000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device="cuda")
    w = torch.linspace(0.5, 2, 192, device="cuda")
    q, k, alone = torch.empty_like(x[:, :4]), torch.empty_like(x[:, 4:]), torch.empty_like(x[:, 4:])
    csa2.csa2_qk_norm_rope(x[:, :4], q, pos, f, k=x[:, 4:], k_out=k, k_norm_w=w, layout=layout)
    csa2.csa2_qk_norm_rope(None, None, pos, f, k=x[:, 4:], k_out=alone, k_norm_w=w, layout=layout)
    assert torch.equal(k, alone)


def test_rows_beyond_4_gib_are_normed_and_turned():
    import csa2_compressed_sparse_gb300 as csa2
    from test_gpu_heads import check, freq
    T, H, D = 4200, 1024, 512  # 4.4 GB
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, H, D), device="cuda").bfloat16()
    last = x[-3:].clone()
    pos, f = torch.arange(T, device="cuda"), freq(32)
    csa2.csa2_qk_norm_rope(x, x, pos, f)
    check(x[-3:], last, None, True, 1e-6, pos[-3:], f, D - 64, 0, 1.0)
    assert bool((x[:-3] == 0).all())
