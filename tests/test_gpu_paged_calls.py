"""Calls of the paged cache as a server makes them: on two streams at once, with a table that has
a row for every slot, with thousands of queries, captured before any other call."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_paged import BF16, DTYPES, E8M0, S128, check_query, check_rows, decode, get, inv_freq
from test_gpu_paged import paged, pool, put, quantised, workspace

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


class Side:
    """Six calls over caches of its own; their outputs, by call."""
    def __init__(self, dtype, lens, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.lens, B = dtype, lens, len(lens)
        self.data, self.table, _ = pool(np.random.default_rng(seed), dtype, 64, lens)
        for b, n in enumerate(lens):
            if n:
                put(self.data, self.table, b,
                    quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
        self.c = paged(self.data, self.table, dtype)
        self.seq = torch.arange(B, dtype=torch.int32, device="cuda")
        self.pos = torch.tensor(lens, device="cuda") - 1
        self.q = torch.randn((6, B, 64, 512), generator=g, device="cuda").bfloat16()
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros((6, B, 64), device="cuda")
        self.ws = workspace(B, 64, max(lens))

    def call(self, i, stream=None):
        import csa2_compressed_sparse_gb300 as csa2
        csa2.csa2_paged_attn(self.q[i], self.seq, self.pos, self.c, self.out[i], self.ws,
                             max_rows=max(self.lens), lse=self.lse[i], stream=stream)


@pytest.mark.parametrize("kinds", [(BF16, BF16), (S128, BF16), (E8M0, S128)])
@pytest.mark.parametrize("lens", [[5000, 40], [1500, 0, 700], [200, 256]])
def test_calls_in_flight_on_two_streams(kinds, lens):
    """Twelve calls, six on each stream, all enqueued before the first is waited for; each stream
    has its workspace.  A call's bits depend on its inputs alone."""
    import csa2_compressed_sparse_gb300 as csa2
    sides = [Side(k, lens, 70 + i) for i, k in enumerate(kinds)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sides:
        for i in range(6):
            s.call(i)
            csa2.csa2_device_status()
    want = [(s.out.clone(), s.lse.clone()) for s in sides]
    for s in sides:
        for i in (0, 5):
            for b, n in enumerate(lens):
                check_query(s.out[i, b], s.lse[i, b], s.q[i, b],
                            decode(get(s.data, s.table, b, 0, n), s.dtype), None, 512 ** -0.5, n - 1,
                            False)
    for _ in range(4):
        for s in sides:
            s.out.zero_()
            s.lse.zero_()
        torch.cuda.synchronize()
        for i in range(6):
            for s, st in zip(sides, streams):
                s.call(i, st)
        for st in streams:
            csa2.csa2_device_status(st)
        for s, (out, lse) in zip(sides, want):
            assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,H", [(1, 64), (4, 64), (2, 100)])
def test_a_table_of_slots_most_of_them_empty(dtype, tokens, H):
    """A table with a row for each of 300 slots; five sequences live, in slots of any order."""
    import csa2_compressed_sparse_gb300 as csa2
    g = torch.Generator(device="cuda").manual_seed(8)
    slots, lens = [299, 3, 150, 0, 77], [3000, 17, 900, 64, 2222]
    data, small, _ = pool(np.random.default_rng(8), dtype, 64, lens)
    table = torch.full((300, small.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[torch.tensor(slots, device="cuda")] = small
    for s, n in zip(slots, lens):
        put(data, table, s, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    seq = [s for s in slots for _ in range(tokens)]
    pos = [n - tokens + i for n in lens for i in range(tokens)]
    Q = len(seq)
    q = torch.randn((Q, H, 512), generator=g, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty((Q, H), device="cuda")
    csa2.csa2_paged_attn(q, torch.tensor(seq, dtype=torch.int32, device="cuda"),
                         torch.tensor(pos, device="cuda"), paged(data, table, dtype), out,
                         workspace(Q, H, 3000), max_rows=3000, lse=lse, inv_freq=inv_freq().cuda())
    # and a token for each live slot: all others have none
    kv = torch.randn((5, 512), generator=g, device="cuda").bfloat16()
    cu = torch.zeros(301, dtype=torch.int32)
    for s in slots:
        cu[s + 1:] += 1
    start = torch.zeros(300, dtype=torch.int64, device="cuda")
    start[torch.tensor(slots, device="cuda")] = torch.tensor(lens, device="cuda") - 1  # the last row anew
    csa2.csa2_paged_append(kv, cu.cuda(), start, paged(data, table, dtype), inv_freq=inv_freq().cuda())
    csa2.csa2_device_status()
    for i, t in enumerate(sorted(zip(slots, lens))):
        check_rows(get(data, table, t[0], t[1] - 1, t[1]), kv[i:i + 1],
                   torch.tensor([t[1] - 1], device="cuda"), dtype, True)
    for i in range(Q):
        if pos[i] + 1 == lens[i // tokens]:
            continue  # (its last row has been replaced since)
        x = decode(get(data, table, seq[i], 0, pos[i] + 1), dtype)
        check_query(out[i], lse[i], q[i], x, None, 512 ** -0.5, pos[i], True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Q,H,most", [(5000, 16, 700), (65535, 1, 20), (3000, 128, 300)])
def test_thousands_of_queries(dtype, Q, H, most):
    import csa2_compressed_sparse_gb300 as csa2
    rng = np.random.default_rng(Q)
    g = torch.Generator(device="cuda").manual_seed(Q)
    lens = [int(n) for n in rng.integers(0, most + 1, 40)]
    data, table, _ = pool(rng, dtype, 16, lens)
    for b, n in enumerate(lens):
        if n:
            put(data, table, b, quantised(torch.randn((n, 512), generator=g, device="cuda"), dtype))
    seq = rng.integers(-1, 40, Q)
    seq[-1] = int(np.argmax(lens))
    pos = np.array([rng.integers(-1, max(lens[s], 1)) if s >= 0 else 0 for s in seq])
    pos = np.minimum(pos, [lens[s] - 1 if s >= 0 else 0 for s in seq])
    q = torch.randn((Q, H, 512), generator=g, device="cuda").bfloat16()
    out = torch.full((Q, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Q, H), 7.0, device="cuda")
    csa2.csa2_paged_attn(q, torch.tensor(seq, dtype=torch.int32, device="cuda"),
                         torch.tensor(pos, dtype=torch.int64, device="cuda"),
                         paged(data, table, dtype), out, workspace(Q, H, most), max_rows=most, lse=lse)
    csa2.csa2_device_status()
    pad = torch.tensor(seq < 0, device="cuda")
    assert bool((out[pad] == 7.0).all()) and bool((lse[pad] == 7.0).all())
    assert not bool((lse[~pad] == 7.0).any())
    for i in list(range(0, Q, Q // 60)) + [Q - 1]:
        if seq[i] >= 0:
            x = decode(get(data, table, int(seq[i]), 0, int(pos[i]) + 1), dtype)
            check_query(out[i], lse[i], q[i], x, None, 512 ** -0.5, int(pos[i]), False)


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import csa2_compressed_sparse_gb300 as csa2
torch.manual_seed(1)
B, H, n = 2, 64, {n}
data = torch.randn((2 * n // 64, 64, 512), device="cuda").bfloat16()
table = torch.arange(2 * n // 64, dtype=torch.int32, device="cuda").reshape(2, -1)
c = csa2.Paged(data, table)
kv = torch.randn((B, 512), device="cuda").bfloat16()
q = torch.randn((B, H, 512), device="cuda").bfloat16()
out, again = torch.zeros_like(q), torch.zeros_like(q)
one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
seq = torch.arange(B, dtype=torch.int32, device="cuda")
pos = torch.full((B,), n - 1, device="cuda")
ws = torch.empty(max(1, csa2.csa2_paged_attn_workspace_size(B, H, n)), dtype=torch.uint8, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # the first calls of the process
    csa2.csa2_paged_append(kv, one, pos, c)
    csa2.csa2_paged_attn(q, seq, pos, c, out, ws, max_rows=n)
graph.replay()
csa2.csa2_device_status()
csa2.csa2_paged_attn(q, seq, pos, c, again, ws, max_rows=n)
csa2.csa2_device_status()
assert torch.equal(data.reshape(2, n, 512)[:, -1], kv)
assert torch.equal(out, again) and bool((out != 0).any())
print("captured")
"""


@pytest.mark.parametrize("n", [128, 1024, 8192])
def test_the_first_calls_of_a_process_can_be_captured(n):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, n=n)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
