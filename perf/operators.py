"""The paged latent cache's operators as workloads: what a pass reads, writes and computes, the
operators in plain torch operations, and the library's calls.

A cache row is one 512-wide latent that serves as key and value of every head; dims 448..511 carry
the rotation of the row's position.  Pages hold page_rows rows each; a table maps a sequence's
logical pages to pages of the pool.
"""
import math

import torch

own = False

D, R0 = 512, 448
THETA = 160000.0


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of a decode batch's 64 sequences: latency
        append("append_decode", "bf16", B=64, lo=1, hi=1, hist=300, page=64),
        # the same token batch into FP8 rows, 16-row pages, as a serving engine's pool keeps them
        append("append_decode_fp8", "fp8_s128", B=64, lo=1, hi=1, hist=100, page=16),
        # a prefill chunk of 4096 tokens in ragged pieces of one to some thousand tokens
        append("append_chunk", "fp8_e8m0", B=3, lo=1, hi=2729, hist=77, page=64),
        # the whole prompts of four sequences of up to 65535 tokens
        append("append_prompt", "bf16", B=4, lo=16384, hi=65535, hist=0, page=64),
        # four short sequences (4096 tokens at ratio 2): the smallest decode batch
        attn("attn_tiny", "bf16", B=4, lo=2048, hi=2048, H=64, page=64, ratio=2),
        # one token of one sequence, a few pages of rows compressed 128 to 1
        attn("attn_one", "bf16", B=1, lo=513, hi=513, H=64, page=8, ratio=128),
        # the decode batch: 64 sequences of 16384 to 65536 tokens at ratio 2
        attn("attn_decode", "bf16", B=64, lo=8192, hi=32768, H=64, page=64, ratio=2),
        # the same batch on FP8 rows
        attn("attn_decode_fp8", "fp8_s128", B=64, lo=8192, hi=32768, H=64, page=64, ratio=2),
        # a long context on its own: 1048576 rows, split over the whole GPU
        attn("attn_long", "bf16", B=1, lo=1048576, hi=1048576, H=64, page=64, ratio=1),
        # a head shard of 16 heads, a wide ragged batch with padded queries, 48-row pages
        attn("attn_shard", "bf16", B=200, lo=1, hi=8191, H=16, page=48, ratio=1, pad=56),
        # four drafted tokens per sequence, E8M0 rows, 16-row pages
        attn("attn_draft", "fp8_e8m0", B=8, lo=1000, hi=20000, H=64, page=16, ratio=1, tokens=4),
        # a window of the last 128 rows kept in pages
        attn("attn_window", "bf16", B=32, lo=100, hi=60000, H=64, page=64, ratio=1, window=128),
    ]


def append(name, dtype, B, lo, hi, hist, page, ratio=1):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "lo": lo, "hi": hi, "hist": hist,
            "page": page, "ratio": ratio}


def attn(name, dtype, B, lo, hi, H, page, ratio, tokens=1, window=0, pad=0):
    return {"name": name, "op": "attn", "dtype": dtype, "B": B, "lo": lo, "hi": hi, "H": H,
            "page": page, "ratio": ratio, "tokens": tokens, "window": window, "pad": pad}


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp8_s128", "fp8_e8m0"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 64, 128, 256])
    if rng.random() < 0.35:
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, 150000 // B)
        lo = rng.randint(1, hi)
        c = append("", dtype, B, lo, hi, rng.randint(0, 300), page, rng.choice([1, 1, 2, 128]))
    else:
        H = rng.choice([64, 64, 64, rng.randint(1, 128), 8, 16, 32, 128])
        tokens = rng.choice([1, 1, 1, 2, 4])
        B = _log(rng, 1, 256)
        # rows of all queries together: at most the decode batch's
        hi = _log(rng, 1, 1000000 // (B * tokens))
        lo = rng.randint(max(1, hi // 8), hi)
        c = attn("", dtype, B, lo, hi, H, page, rng.choice([1, 1, 2, 128]), tokens,
                 rng.choice([0, 0, 0, 128, rng.randint(1, 2000)]), rng.choice([0, 0, rng.randint(1, 9)]))
    del c["name"]
    return c


def lengths(c):
    """The rows of each sequence, evenly spread from lo to hi (in ascending order)."""
    n = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) if n > 1 else c["hi"] for i in range(n)]


def row_bytes(c):
    return 1024 if c["dtype"] == "bf16" else 528


def work(c):
    ln = lengths(c)
    if c["op"] == "append":
        T = sum(ln)
        # per element about ten operations (two products and a sum in the rotated dims, the
        # quantiser's maximum and quotient)
        return {"bytes": T * (1024 + row_bytes(c)) + 12 * c["B"], "flops": 10 * T * D}
    n, w, H = c["tokens"], c["window"], c["H"]
    Q = n * c["B"]
    seen = [sum(min(w or x, x) for x in (max(0, y - n + 1 + i) for i in range(n))) for y in ln]
    once = [min(y, w + n - 1) if w else y for y in ln]
    return {"bytes": sum(once) * row_bytes(c) + Q * H * (2 * 1024 + 4) + 12 * Q + 4 * H,
            "flops": 4 * H * D * sum(seen)}


# ---- inputs -----------------------------------------------------------------------------------

def inv_freq():
    return THETA ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    B, page, ratio = c["B"], c["page"], c["ratio"]
    ln = torch.tensor(lengths(c))[torch.randperm(B, generator=h)]
    hist = torch.randint(0, c["hist"] + 1, (B,), generator=h) if c["op"] == "append" else torch.zeros(B, dtype=torch.int64)
    total = hist + ln
    pages = (total + page - 1) // page
    n_pages = 3 + sum(-(-(n + c.get("hist", 0)) // page) for n in lengths(c))
    ids = torch.randperm(n_pages, generator=h)[:int(pages.sum())].to(torch.int32)
    cols = torch.arange(int(pages.max()))
    table = torch.full((B, int(pages.max()) + 1), -1, dtype=torch.int32)
    table[:, :-1][cols < pages[:, None]] = ids
    s = {"c": c, "dtype": c["dtype"], "page": page, "ratio": ratio, "table": table.cuda(),
         "inv_freq": inv_freq().float().cuda()}
    rb = row_bytes(c)
    if c["dtype"] == "bf16":
        s["data"] = torch.empty((n_pages, page, D), dtype=torch.bfloat16, device="cuda")
        s["data"].normal_(generator=g)
        s["views"] = [s["data"]]
    else:
        d = s["data"] = torch.empty((n_pages, page, rb), dtype=torch.uint8, device="cuda")
        s["views"] = [d[..., :D].view(torch.float8_e4m3fn)]
        some = torch.randn((n_pages, page, D), generator=g, device="cuda", dtype=torch.bfloat16)
        if c["dtype"] == "fp8_s128":
            s["views"].append(d[..., D:].view(torch.float32))
        else:
            s["views"].append(d[..., D:].view(torch.float8_e8m0fnu))
        # codes of values near one in standard deviation: the largest of a group is coded near 448
        group = 128 if c["dtype"] == "fp8_s128" else 32
        store(s, some.reshape(-1, D), (torch.arange(n_pages * page, device="cuda") // page,
                                       torch.arange(n_pages * page, device="cuda") % page), group)
    if c["op"] == "append":
        T = int(ln.sum())
        s["kv"] = torch.randn((T, D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), ln.cumsum(0)]).to(torch.int32).cuda()
        s["start"] = hist.cuda()
    else:
        n, pad, H = c["tokens"], c["pad"], c["H"]
        last = (ln * ratio - 1)[:, None]  # the newest token's position: it sees ln rows
        pos = last - ratio * torch.arange(n - 1, -1, -1)
        s["q_pos"] = torch.cat([pos.reshape(-1), torch.zeros(pad, dtype=torch.int64)]).cuda()
        seq = torch.arange(B, dtype=torch.int32).repeat_interleave(n)
        s["q_seq"] = torch.cat([seq, torch.full((pad,), -1, dtype=torch.int32)]).cuda()
        Q = n * B + pad
        s["q"] = torch.randn((Q, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["sink"] = torch.randn((H,), generator=g, device="cuda")
        # rows of padded queries keep what they hold
        s["out"] = torch.full((Q, H, D), 2.0 ** -8, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.ones((Q, H), dtype=torch.float32, device="cuda")
        s["max_rows"] = c["hi"]
        s["window"] = c["window"]
    if own:
        import csa2_compressed_sparse_gb300 as csa2
        s["cache"] = csa2.Paged(s["data"], s["table"], fp8_dtype=2 if c["dtype"] == "fp8_e8m0" else 1)
        if c["op"] == "attn":
            size = csa2.csa2_paged_attn_workspace_size(Q, c["H"], s["max_rows"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    if s["c"]["op"] == "append":
        if own:
            import csa2_compressed_sparse_gb300 as csa2
            csa2.csa2_paged_append(s["kv"], s["cu"], s["start"], s["cache"], inv_freq=s["inv_freq"],
                                   ratio=s["ratio"])
        else:
            plain_append(s)
        return s["views"]
    if own:
        import csa2_compressed_sparse_gb300 as csa2
        csa2.csa2_paged_attn(s["q"], s["q_seq"], s["q_pos"], s["cache"], s["out"], s["ws"],
                             max_rows=s["max_rows"], ratio=s["ratio"], window=s["window"],
                             sink=s["sink"], lse=s["lse"], inv_freq=s["inv_freq"])
    else:
        plain_attn(s)
    return [s["out"], s["lse"]]


def turn(x, pos, freq, sign):
    """x [..., 512] in 32 bits with the pairs of dims 448.. times e^{sign i pos theta}; the angles
    and their cosines and sines in 64 bits."""
    a = pos.double()[..., None] * freq.double()
    co, si = a.cos().float(), sign * a.sin().float()
    e, o = x[..., R0::2], x[..., R0 + 1::2]
    rot = torch.stack([e * co - o * si, e * si + o * co], -1).flatten(-2)
    return torch.cat([x[..., :R0], rot], -1)


def store(s, y, at, group):
    """Rows y (32 bits) into the pool at (page, row): rounded to bf16, or quantised by group."""
    if s["dtype"] == "bf16":
        s["data"][at] = y.bfloat16()
        return
    v = y.float().reshape(y.shape[0], -1, group)
    top = v.abs().amax(-1, keepdim=True)
    if s["dtype"] == "fp8_s128":
        sc = torch.where(top > 0, top / 448, torch.ones_like(top))
        s["views"][1][at] = sc[..., 0]
    else:
        # the smallest power of two with top <= 448 * 2^e, from top / 448's exponent
        m, e = torch.frexp(top.double() / 448)
        e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
        e = torch.where(top > 0, e, torch.zeros_like(e))
        sc = torch.exp2(e.float())
        s["data"][..., D:][at] = (e[..., 0] + 127).to(torch.uint8)
    s["views"][0].view(torch.uint8)[at] = (v / sc).reshape(y.shape).to(torch.float8_e4m3fn).view(torch.uint8)


def plain_append(s):
    T = s["kv"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu"], t.to(torch.int32), right=True) - 1
    j = s["start"][b] + t - s["cu"][b]
    y = turn(s["kv"].float(), j * s["ratio"], s["inv_freq"], 1)
    page = s["table"][b, j // s["page"]].long()
    store(s, y, (page, j % s["page"]), 128 if s["dtype"] == "fp8_s128" else 32)


def plain_attn(s):
    live = s["q_seq"] >= 0
    seq, pos, q = s["q_seq"][live].long(), s["q_pos"][live], s["q"][live].float()
    hi = (pos + 1) // s["ratio"]
    lo = (hi - s["window"]).clamp(min=0) if s["window"] else torch.zeros_like(hi)
    n = s["window"] if s["window"] else s["max_rows"]
    j = lo[:, None] + torch.arange(min(n, s["max_rows"]), device="cuda")
    seen = j < hi[:, None]
    j = torch.where(seen, j, torch.zeros_like(j))
    page = s["table"][seq[:, None], j // s["page"]].long()
    page = torch.where(seen, page, torch.zeros_like(page))
    x = s["data"][page, j % s["page"]]
    if s["dtype"] == "bf16":
        x = x.float()
    else:
        tail = x[..., D:].contiguous()
        sc = tail.view(torch.float32) if s["dtype"] == "fp8_s128" else torch.exp2(tail.float() - 127)
        x = x[..., :D].contiguous().view(torch.float8_e4m3fn).float()
        x = (x.reshape(*sc.shape, -1) * sc[..., None]).reshape(x.shape)
    x = x.masked_fill_(~seen[..., None], 0.0)
    z = torch.matmul(q, x.transpose(1, 2)) * D ** -0.5
    z = z.masked_fill(~seen[:, None, :], -math.inf)
    sink = s["sink"][None, :, None]
    top = torch.maximum(z.amax(-1, keepdim=True), sink)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True) + torch.exp(sink - top)
    o = torch.matmul(p, x) / total
    o = turn(o, pos[:, None].expand(o.shape[:2]), s["inv_freq"], -1)
    s["out"][live] = o.bfloat16()
    s["lse"][live] = (top + torch.log(total))[..., 0]


# ---- the definition in 64 bits -----------------------------------------------------------------

def e4m3_table():
    """The 256 values of E4M3 from its fields: bias 7, no infinities, S.1111.111 is NaN."""
    v = []
    for k in range(256):
        e, m = (k >> 3) & 15, k & 7
        x = math.nan if (e, m) == (15, 7) else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if k & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def wide(s, rows):
    """Cache rows (bytes or bf16, [n, width]) as 64-bit values [n, 512]."""
    if s["dtype"] == "bf16":
        return rows.double()
    v = e4m3_table()[rows[:, :D].long()]
    if s["dtype"] == "fp8_s128":
        return v * rows[:, D:].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return v * torch.exp2(rows[:, D:].double() - 127).repeat_interleave(32, 1)


def rotate64(x, pos, sign):
    """x [n, 512] in 64 bits, row i rotated by sign * pos[i] * theta."""
    f = inv_freq().float().double().to(x.device)
    z = torch.view_as_complex(x[:, R0:].reshape(x.shape[0], 32, 2).contiguous())
    z = z * torch.polar(torch.ones_like(z.real), sign * pos.double()[:, None] * f)
    return torch.cat([x[:, :R0], torch.view_as_real(z).reshape(x.shape[0], 64)], 1)


def exact(c, seed):
    s = prepare(c, seed)
    page, table = s["page"], s["table"].cpu().tolist()
    if c["op"] == "append":
        # every row of the pool in 64 bits; what quantised rows hold is the definition's codes and
        # scales, whose quotient and maximum are taken in 64 bits
        flat = s["data"].reshape(-1, s["data"].shape[-1])
        cu, start = s["cu"].tolist(), s["start"].tolist()
        at, pos = [], []
        for b in range(c["B"]):
            js = torch.arange(start[b], start[b] + cu[b + 1] - cu[b])
            at.append(torch.tensor(table[b])[js // page].long() * page + js % page)
            pos.append(js * s["ratio"])
        at, pos = torch.cat(at).cuda(), torch.cat(pos).cuda()
        y = rotate64(s["kv"].double(), pos, 1)
        shape = s["data"].shape[:2]
        if c["dtype"] == "bf16":
            whole = flat.double()
            whole[at] = y
            return [whole.reshape(*shape, D)]
        group = 128 if c["dtype"] == "fp8_s128" else 32
        v = y.reshape(y.shape[0], -1, group)
        top = v.abs().amax(-1)
        if c["dtype"] == "fp8_s128":
            sc = torch.where(top > 0, top / 448, torch.ones_like(top))
            old = flat[:, D:].contiguous().view(torch.float32).double()
        else:
            e = torch.full_like(top, -127.0)
            for k in range(-126, 128):
                e = torch.where(top > 448 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
            sc = torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)))
            old = torch.exp2(flat[:, D:].double() - 127)
        codes = e4m3_table()[flat[:, :D].long()]
        codes[at] = (v / sc[..., None]).reshape(y.shape)
        old[at] = sc
        return [codes.reshape(*shape, D), old.reshape(*shape, -1)]
    out, lse = s["out"].double(), s["lse"].double()
    flat = s["data"].reshape(-1, s["data"].shape[-1])
    q_seq, q_pos = s["q_seq"].tolist(), s["q_pos"].tolist()
    for i, (b, p) in enumerate(zip(q_seq, q_pos)):
        if b < 0:
            continue
        hi = (p + 1) // s["ratio"]
        lo = max(0, hi - s["window"]) if s["window"] else 0
        sink = s["sink"].double()
        if hi <= lo:
            out[i], lse[i] = 0.0, sink
            continue
        js = torch.arange(lo, hi, device="cuda")
        x = wide(s, flat[s["table"][b].long()[js // page] * page + js % page])
        z = (s["q"][i].double() @ x.T) * D ** -0.5
        total = torch.logsumexp(torch.cat([z, sink[:, None]], 1), 1)
        o = torch.exp(z - total[:, None]) @ x
        out[i] = rotate64(o, torch.full((o.shape[0],), p, device="cuda"), -1)
        lse[i] = total
    return [out, lse]
