"""Operators around the paged latent cache as workloads: attention of chunks of new tokens, rows read
back, and the norm and rotation of queries and keys.  What a pass reads, writes and computes, the
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
        # sixteen tokens of one short conversation: latency
        chunk("chunk_one", "bf16", B=1, lo=16, hi=16, hist=284, H=64, page=64),
        # whole prompts of 100 to 2000 tokens in one packed batch, causal, nothing cached before
        chunk("chunk_prompt", "bf16", B=8, lo=100, hi=2000, hist=0, H=64, page=64),
        # a prefill chunk of 2048 tokens at the end of 65536, two tokens to a row
        chunk("chunk_long", "bf16", B=1, lo=2048, hi=2048, hist=63488, H=64, page=64, ratio=2),
        # chunks of four sequences over FP8 rows
        chunk("chunk_fp8", "fp8_s128", B=4, lo=100, hi=300, hist=16000, H=64, page=64),
        # a head shard of 16 heads, 24 ragged chunks with padded tokens, 48-row pages
        chunk("chunk_shard", "bf16", B=24, lo=1, hi=500, hist=3000, H=16, page=48, pad=37),
        # a ragged batch that sees a window of the last 128 rows, E8M0 rows in 16-row pages
        chunk("chunk_window", "fp8_e8m0", B=3, lo=1, hi=2729, hist=77, H=64, page=16, window=128),
        # eight drafted tokens over a long context
        chunk("chunk_few", "bf16", B=1, lo=8, hi=8, hist=262136, H=64, page=64),
        # one short sequence handed over: latency
        read("read_one", "fp8_s128", B=1, lo=300, hi=300, page=16),
        # the prompts of four sequences read back, rotated back on the way
        read("read_prompt", "fp8_e8m0", B=4, lo=16384, hi=65535, page=64, back=True),
        # the queries and the new latent of a decode batch of 64 tokens
        heads("heads_decode", T=64, H=64, K=1, dim=512, rope=64),
        # the same for a prefill chunk of 4096 tokens
        heads("heads_chunk", T=4096, H=64, K=1, dim=512, rope=64),
        # indexer queries and keys, 128 wide, halves rotated, a table and factor for long contexts
        heads("heads_index", T=1001, H=64, K=1, dim=128, rope=64, half=True, factor=1.25),
    ]


def chunk(name, dtype, B, lo, hi, hist, H, page, ratio=1, window=0, pad=0):
    return {"name": name, "op": "chunk", "dtype": dtype, "B": B, "lo": lo, "hi": hi, "hist": hist,
            "H": H, "page": page, "ratio": ratio, "window": window, "pad": pad}


def read(name, dtype, B, lo, hi, page, ratio=1, back=False):
    return {"name": name, "op": "read", "dtype": dtype, "B": B, "lo": lo, "hi": hi, "page": page,
            "ratio": ratio, "back": back}


def heads(name, T, H, K, dim, rope, half=False, factor=1.0, q_norm=True):
    return {"name": name, "op": "heads", "T": T, "H": H, "K": K, "dim": dim, "rope": rope,
            "half": half, "factor": factor, "q_norm": q_norm}


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp8_s128", "fp8_e8m0"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 64, 128, 256])
    ratio = rng.choice([1, 1, 2, 128])
    kind = rng.random()
    if kind < 0.6:
        H = rng.choice([64, 64, 64, rng.randint(1, 128), 8, 16, 32, 128])
        B = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, 131072 // (H * B)))  # of a sequence
        lo = rng.randint(1, tokens)
        # rows and products: at most what the largest listed case has
        rows = min(262144 // B, int(8.0e12 / (2048.0 * H * B * tokens)) + 1)
        hist = max(0, (_log(rng, 1, rows) - 1) * ratio - tokens + rng.randint(0, ratio))
        window = rng.choice([0, 0, 0, 128, rng.randint(1, 2000)])
        c = chunk("", dtype, B, lo, tokens, hist, H, page, ratio, window,
                  rng.choice([0, 0, rng.randint(1, 9)]))
    elif kind < 0.75:
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 150000 // B)
        c = read("", dtype, B, rng.randint(1, hi), hi, page, ratio, rng.random() < 0.5)
    else:
        dim = rng.choice([512, 512, 128, 128, 64, 192, 256, 8 * rng.randint(2, 64)])
        half = rng.random() < 0.5
        rope = min(rng.choice([16, 32, 64, 64, 64, 128, 512]), dim // 16 * 16)
        H = rng.choice([64, 64, 32, 16, rng.randint(1, 128)])
        K = rng.choice([0, 1, 1, 1, rng.randint(1, 16)])
        T = _log(rng, 1, 4096 * 65 * 512 // ((H + K) * dim))
        c = heads("", T, H, K, dim, rope, half, rng.choice([1.0, 1.0, 1.25, 0.1 * math.log(32) + 1]),
                  rng.random() < 0.8)
    del c["name"]
    return c


def lengths(c):
    """New tokens (or rows to read) of each sequence, evenly spread from lo to hi."""
    n = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) if n > 1 else c["hi"] for i in range(n)]


def row_bytes(c):
    return 1024 if c["dtype"] == "bf16" else 528


def seen(c, p):
    """Rows lo .. hi - 1 that the token at position p sees."""
    hi = (p + 1) // c["ratio"]
    return (max(0, hi - c["window"]) if c["window"] else 0), hi


def work(c):
    if c["op"] == "heads":
        n = c["T"] * (c["H"] + c["K"])
        return {"bytes": 4 * n * c["dim"] + 8 * c["T"], "flops": n * (4 * c["dim"] + 3 * c["rope"])}
    ln = lengths(c)
    if c["op"] == "read":
        T = sum(ln)
        return {"bytes": T * (row_bytes(c) + 2 * D) + 12 * c["B"], "flops": T * (D + 192)}
    pairs = once = 0
    for n in ln:
        first, last = seen(c, c["hist"]), seen(c, c["hist"] + n - 1)
        once += max(0, last[1] - first[0])
        pairs += sum(b - a for a, b in (seen(c, c["hist"] + i) for i in range(n)))
    T = sum(ln)
    return {"bytes": once * row_bytes(c) + T * c["H"] * (2 * 1024 + 4) + 12 * c["B"] + 4 * c["H"],
            "flops": 4 * c["H"] * D * pairs}


# ---- inputs -----------------------------------------------------------------------------------

def inv_freq(n=32, factor=1.0):
    """Rotation steps; beyond a factor of one the slow ones are slowed as for a longer context."""
    f = THETA ** (-torch.arange(0, n, dtype=torch.float64) / n)
    if factor != 1.0:
        slow = ((2 * math.pi / f) / 4096).clamp(0, 1)
        f = f * (1 - slow) + f / 16 * slow
    return f


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    if c["op"] == "heads":
        T, H, K, dim = c["T"], c["H"], c["K"], c["dim"]
        # one projection's output holds the queries and the keys of a token side by side
        x = torch.randn((T, H + K, dim), generator=g, device="cuda", dtype=torch.bfloat16)
        s = {"c": c, "x": x, "q": x[:, :H], "k": x[:, H:] if K else None,
             "q_out": torch.empty((T, H, dim), dtype=torch.bfloat16, device="cuda"),
             "k_out": torch.empty((T, K, dim), dtype=torch.bfloat16, device="cuda") if K else None,
             "pos": torch.randint(0, 1 << 20, (T,), generator=h).cuda(),
             "q_w": 1 + 0.2 * torch.randn((dim,), generator=g, device="cuda") if c["q_norm"] else None,
             "k_w": 1 + 0.2 * torch.randn((dim,), generator=g, device="cuda"),
             "inv_freq": inv_freq(c["rope"] // 2, c["factor"]).float().cuda()}
        return s
    B, page, ratio = c["B"], c["page"], c["ratio"]
    new = torch.tensor(lengths(c))[torch.randperm(B, generator=h)]
    if c["op"] == "chunk":
        start = torch.full((B,), c["hist"], dtype=torch.int64)  # position of the first new token
        total = (start + new) // ratio                          # rows of each sequence
    else:
        start = torch.randint(0, 100, (B,), generator=h)        # first row to read
        total = start + new
    pages = (total + page - 1) // page
    n_pages = 3 + sum(-(-(n + 100 if c["op"] == "read" else (c["hist"] + n) // ratio) // page)
                      for n in lengths(c))
    ids = torch.randperm(n_pages, generator=h)[:int(pages.sum())].to(torch.int32)
    cols = torch.arange(int(pages.max()))
    table = torch.full((B, int(pages.max()) + 1), -1, dtype=torch.int32)
    table[:, :-1][cols < pages[:, None]] = ids
    s = {"c": c, "table": table.cuda(), "inv_freq": inv_freq().float().cuda(),
         "lens": new.tolist(), "first": start.tolist(), "start": start.cuda(),
         "cu": torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).cuda()}
    if c["dtype"] == "bf16":
        s["data"] = torch.empty((n_pages, page, D), dtype=torch.bfloat16, device="cuda")
        s["data"].normal_(generator=g)
    else:
        # codes and scales of rows of deviation one, as the cache's writer leaves them
        x = torch.randn((n_pages * page, D), generator=g, device="cuda").bfloat16().float()
        v = x.reshape(x.shape[0], -1, 128 if c["dtype"] == "fp8_s128" else 32)
        top = v.abs().amax(-1, keepdim=True)
        if c["dtype"] == "fp8_s128":
            sc = top / 448
            tail = sc[..., 0].contiguous().view(torch.uint8)
        else:
            e = torch.ceil(torch.log2(top.double() / 448)).float()
            sc = torch.exp2(e)
            tail = (e[..., 0] + 127).to(torch.uint8)
        codes = (v / sc).reshape(x.shape).to(torch.float8_e4m3fn).view(torch.uint8)
        s["data"] = torch.cat([codes, tail], 1).reshape(n_pages, page, -1)
    T = int(new.sum())
    if c["op"] == "read":
        s["out"] = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    else:
        H = c["H"]
        s["q"] = torch.randn((T + c["pad"], H, D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["sink"] = torch.randn((H,), generator=g, device="cuda")
        # padded tokens keep what they hold
        s["out"] = torch.full((T + c["pad"], H, D), 2.0 ** -8, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.ones((T + c["pad"], H), dtype=torch.float32, device="cuda")
        s["max_rows"], s["total_rows"] = int(total.max()), int(total.sum())
    if own:
        import csa2_compressed_sparse_gb300 as csa2
        s["cache"] = csa2.Paged(s["data"], s["table"], fp8_dtype=2 if c["dtype"] == "fp8_e8m0" else 1)
        if c["op"] == "chunk":
            size = csa2.csa2_paged_chunk_attn_workspace_size(T + c["pad"], c["H"], s["cache"],
                                                             s["max_rows"], s["total_rows"])
            s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    c = s["c"]
    if c["op"] == "heads":
        if own:
            import csa2_compressed_sparse_gb300 as csa2
            csa2.csa2_qk_norm_rope(s["q"], s["q_out"], s["pos"], s["inv_freq"], k=s["k"],
                                   k_out=s["k_out"], q_norm=c["q_norm"], q_norm_w=s["q_w"],
                                   k_norm_w=s["k_w"] if c["K"] else None,
                                   layout=csa2.ROPE_HALVES if c["half"] else csa2.ROPE_PAIRS,
                                   factor=c["factor"])
        else:
            plain_heads(s)
        return [s["q_out"], s["k_out"]] if c["K"] else [s["q_out"]]
    if c["op"] == "read":
        if own:
            import csa2_compressed_sparse_gb300 as csa2
            csa2.csa2_paged_read(s["out"], s["cu"], s["start"], s["cache"],
                                 inv_freq=s["inv_freq"] if c["back"] else None, ratio=c["ratio"])
        else:
            plain_read(s)
        return [s["out"]]
    if own:
        import csa2_compressed_sparse_gb300 as csa2
        csa2.csa2_paged_chunk_attn(s["q"], s["cu"], s["start"], s["cache"], s["out"], s["ws"],
                                   max_rows=s["max_rows"], total_rows=s["total_rows"],
                                   ratio=c["ratio"], window=c["window"], sink=s["sink"],
                                   lse=s["lse"], inv_freq=s["inv_freq"])
    else:
        plain_chunk(s)
    return [s["out"], s["lse"]]


def turn(x, pos, freq, sign):
    """x [..., 512] in 32 bits with the pairs of dims 448.. times e^{sign i pos theta}; the angles
    and their cosines and sines in 64 bits."""
    a = pos.double()[..., None] * freq.double()
    co, si = a.cos().float(), sign * a.sin().float()
    e, o = x[..., R0::2], x[..., R0 + 1::2]
    rot = torch.stack([e * co - o * si, e * si + o * co], -1).flatten(-2)
    return torch.cat([x[..., :R0], rot], -1)


def rows(s, b, lo, hi):
    """Rows lo .. hi - 1 of sequence b in 32 bits."""
    c = s["c"]
    j = torch.arange(lo, hi, device="cuda")
    x = s["data"][s["table"][b][j // c["page"]].long(), j % c["page"]]
    if c["dtype"] == "bf16":
        return x.float()
    tail = x[:, D:].contiguous()
    sc = tail.view(torch.float32) if c["dtype"] == "fp8_s128" else torch.exp2(tail.float() - 127)
    v = x[:, :D].contiguous().view(torch.float8_e4m3fn).float()
    return (v.reshape(*sc.shape, -1) * sc[..., None]).reshape(v.shape)


def plain_read(s):
    at = 0
    for b, (n, first) in enumerate(zip(s["lens"], s["first"])):
        x = rows(s, b, first, first + n)
        if s["c"]["back"]:
            x = turn(x, torch.arange(first, first + n, device="cuda") * s["c"]["ratio"], s["inv_freq"], -1)
        s["out"][at:at + n] = x.bfloat16()
        at += n


def plain_chunk(s):
    c, at = s["c"], 0
    H, sink = c["H"], s["sink"][None, :, None]
    for b, (n, first) in enumerate(zip(s["lens"], s["first"])):
        base, end = seen(c, first)[0], seen(c, first + n - 1)[1]
        x = rows(s, b, base, end)
        step = max(1, (1 << 28) // (H * max(1, end - base)))  # tokens at a time
        for t in range(0, n, step):
            m = min(step, n - t)
            pos = first + t + torch.arange(m, device="cuda")
            hi = (pos + 1) // c["ratio"]
            lo = (hi - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(hi)
            a, e = seen(c, first + t)[0] - base, seen(c, first + t + m - 1)[1] - base
            j = base + torch.arange(a, e, device="cuda")
            y = x[a:e]
            q = s["q"][at + t:at + t + m].float()
            z = torch.matmul(q.reshape(m * H, D), y.T).reshape(m, H, -1) * D ** -0.5
            out = (j < lo[:, None]) | (j >= hi[:, None])
            z = z.masked_fill_(out[:, None, :], -math.inf)
            top = torch.maximum(z.amax(-1, keepdim=True), sink) if e > a else sink.expand(m, H, 1)
            p = torch.exp_(z.sub_(top))
            total = p.sum(-1, keepdim=True) + torch.exp(sink - top)
            o = torch.matmul(p.reshape(m * H, -1), y).reshape(m, H, D) / total
            o = turn(o, pos[:, None].expand(m, H), s["inv_freq"], -1)
            s["out"][at + t:at + t + m] = o.bfloat16()
            s["lse"][at + t:at + t + m] = (top + torch.log(total))[..., 0]
        at += n


def plain_heads(s):
    c = s["c"]
    dim, n = c["dim"], c["rope"] // 2
    r0 = dim - c["rope"]
    a = s["pos"].double()[:, None] * s["inv_freq"].double()
    co = (a.cos() * c["factor"]).float()[:, None]
    si = (a.sin() * c["factor"]).float()[:, None]
    for x, w, out, norm in ((s["q"], s["q_w"], s["q_out"], c["q_norm"]), (s["k"], s["k_w"], s["k_out"], True)):
        if x is None:
            continue
        y = x.float()
        if norm:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        if c["half"]:
            e, o = y[..., r0:r0 + n], y[..., r0 + n:]
            rot = torch.cat([e * co - o * si, e * si + o * co], -1)
        else:
            e, o = y[..., r0::2], y[..., r0 + 1::2]
            rot = torch.stack([e * co - o * si, e * si + o * co], -1).flatten(-2)
        out.copy_(torch.cat([y[..., :r0], rot], -1))


# ---- the definition in 64 bits -----------------------------------------------------------------

def e4m3_table():
    """The 256 values of E4M3 from its fields: bias 7, no infinities, S.1111.111 is NaN."""
    v = []
    for k in range(256):
        e, m = (k >> 3) & 15, k & 7
        x = math.nan if (e, m) == (15, 7) else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if k & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def wide(c, raw):
    """Cache rows (bytes or bf16, [n, width]) as 64-bit values [n, 512]."""
    if c["dtype"] == "bf16":
        return raw.double()
    v = e4m3_table()[raw[:, :D].long()]
    if c["dtype"] == "fp8_s128":
        return v * raw[:, D:].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return v * torch.exp2(raw[:, D:].double() - 127).repeat_interleave(32, 1)


def rotate64(x, pos, f, sign):
    """x [n, d] in 64 bits: pairs of its last dims times e^{sign i pos f}."""
    n = 2 * f.numel()
    z = torch.view_as_complex(x[:, x.shape[1] - n:].reshape(x.shape[0], n // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(z.real), sign * pos.double()[:, None] * f.double())
    return torch.cat([x[:, :x.shape[1] - n], torch.view_as_real(z).reshape(x.shape[0], n)], 1)


def exact(c, seed):
    if c["op"] == "chunk" and work(c)["flops"] > 1.0e13:
        return None
    s = prepare(c, seed)
    if c["op"] == "heads":
        outs = []
        for x, w, norm in ((s["q"], s["q_w"], c["q_norm"]), (s["k"], s["k_w"], True)):
            if x is None:
                continue
            y = x.double()
            if norm:
                y = y / (y.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * w.double()
            r0, n = c["dim"] - c["rope"], c["rope"] // 2
            if c["half"]:  # as pairs
                y = torch.cat([y[..., :r0], y[..., r0:].unflatten(-1, (2, n)).transpose(-1, -2).flatten(-2)], -1)
            pos = s["pos"][:, None].expand(y.shape[:2]).reshape(-1)
            y = rotate64(y.reshape(-1, c["dim"]), pos, s["inv_freq"], 1).reshape(y.shape)
            if c["half"]:
                y = torch.cat([y[..., :r0], y[..., r0:].unflatten(-1, (n, 2)).transpose(-1, -2).flatten(-2)], -1)
            y[..., r0:] *= c["factor"]
            outs.append(y)
        return outs
    page, at = c["page"], 0
    flat = s["data"].reshape(-1, s["data"].shape[-1])
    out = s["out"].double()
    lse = s["lse"].double() if c["op"] == "chunk" else None
    for b, (n, first) in enumerate(zip(s["lens"], s["first"])):
        end = first + n if c["op"] == "read" else (first + n) // c["ratio"]
        js = torch.arange(end, device="cuda")
        x = wide(c, flat[s["table"][b].long()[js // page] * page + js % page])
        if c["op"] == "read":
            y = x[first:]
            out[at:at + n] = rotate64(y, js[first:] * c["ratio"], s["inv_freq"], -1) if c["back"] else y
            at += n
            continue
        sink = s["sink"].double()
        for i in range(n):
            hi = (first + i + 1) // c["ratio"]
            lo = max(0, hi - c["window"]) if c["window"] else 0
            z = (s["q"][at + i].double() @ x[lo:hi].T) / math.sqrt(D)
            total = torch.logsumexp(torch.cat([z, sink[:, None]], 1), 1)
            o = torch.exp(z - total[:, None]) @ x[lo:hi]
            out[at + i] = rotate64(o, torch.full((o.shape[0],), first + i, device="cuda"), s["inv_freq"], -1)
            lse[at + i] = total
        at += n
    return [out] if c["op"] == "read" else [out, lse]
