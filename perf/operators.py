"""Cases that measure the paged-serving operators: the append of new keys and values (with the rotary embedding) to a
paged KV cache, attention of verify rows over it, the lm_head's logits and the rules applied to them.

Each operator has a plain form in elementary torch operations (``own`` false) and the library's call (``own`` true).
Lengths, rows and heads are those of the verify step (K rows per sequence, 128-wide heads, 151,936 tokens) for a batch
of sequences; per-sequence lengths follow from the case alone, the values from the seed."""
import math

import torch

own = False

HD = 128
LOG_LO, LOG_HI = 64, 131072


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request, one new token, a short odd-length cache: latency of the smallest call
        dict(name="decode one sequence", op="attention", seqs=1, rows=1, q_heads=32, kv_heads=8, page=64,
             len_lo=2011, len_hi=2011, window=0, prefix=0, softcap=0.0, slopes=False, docs=False),
        # the verify step's own attention: four drafted rows over 16,384 positions, now in pages
        dict(name="verify 4 rows at 16384", op="attention", seqs=1, rows=4, q_heads=32, kv_heads=8, page=64,
             len_lo=16384, len_hi=16384, window=0, prefix=0, softcap=0.0, slopes=False, docs=False),
        # a serving batch, one token each, very unequal lengths, small pages
        dict(name="ragged batch decode", op="attention", seqs=64, rows=1, q_heads=32, kv_heads=8, page=16,
             len_lo=500, len_hi=16000, window=0, prefix=0, softcap=0.0, slopes=False, docs=False),
        # sliding-window layers of a verify batch: 64 query heads, first positions kept, capped scores
        dict(name="windowed capped batch", op="attention", seqs=32, rows=4, q_heads=64, kv_heads=8, page=32,
             len_lo=100, len_hi=20000, window=512, prefix=16, softcap=30.0, slopes=False, docs=False),
        # full verify blocks of 16 rows over long caches (64 query rows a KV head)
        dict(name="long verify blocks", op="attention", seqs=2, rows=16, q_heads=32, kv_heads=8, page=128,
             len_lo=65003, len_hi=131001, window=0, prefix=0, softcap=0.0, slopes=False, docs=False),
        # packed documents with a distance bias, as many KV heads as query heads
        dict(name="documents with distance bias", op="attention", seqs=17, rows=3, q_heads=8, kv_heads=8, page=64,
             len_lo=30, len_hi=9000, window=0, prefix=0, softcap=0.0, slopes=True, docs=True),
        # the append of a verify batch's rows
        dict(name="append verify rows", op="append", seqs=64, rows_lo=1, rows_hi=4, q_heads=32, kv_heads=8, page=64,
             len_lo=100, len_hi=16000, rotary=128, yarn=0.0),
        # the append of prompts, partial rotary width with YaRN frequencies
        dict(name="append prompts", op="append", seqs=4, rows_lo=1501, rows_hi=2700, q_heads=48, kv_heads=8, page=64,
             len_lo=1, len_hi=5000, rotary=64, yarn=4.0),
        # one request's logits before its greedy token
        dict(name="one row of logits", op="logits", rows=1, vocab=151936, history=700, type="float32", bias=False,
             mask=False),
        # a serving batch's rows with histories, biases and grammar masks, an odd vocabulary
        dict(name="batch of ruled logits", op="logits", rows=256, vocab=128003, history=4000, type="bfloat16",
             bias=True, mask=True),
        # the vocabulary projection of a verify step
        dict(name="lm_head of 4 rows", op="lm_head", rows=4, hidden=2048, vocab=151936),
        # ... and of a full block over a small vocabulary
        dict(name="lm_head of 16 rows", op="lm_head", rows=16, hidden=1024, vocab=32003),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "logits", "lm_head"])
    if op == "attention":
        q_heads, kv_heads = rng.choice([(32, 8), (64, 8), (48, 8), (8, 8), (16, 2), (8, 1), (28, 4)])
        rows = rng.randint(1, min(16, 64 // (q_heads // kv_heads)))
        seqs = _log_int(rng, 1, 128)
        # at most 0.9 GB of keys and values, and no more products than the largest listed case
        most = min(0.9e9 / (512 * kv_heads), 4.5e10 / (512 * q_heads * rows)) / seqs
        hi = max(1, min(_log_int(rng, LOG_LO, LOG_HI), int(most)))
        lo = rng.choice([0, 1, hi, max(1, hi // 7), max(1, hi // 2)])
        return dict(op=op, seqs=seqs, rows=rows, q_heads=q_heads, kv_heads=kv_heads, page=rng.choice([16, 32, 64, 128]),
                    len_lo=min(lo, hi), len_hi=hi, window=rng.choice([0, 0, 0, 1, 129, 512, 2000]),
                    prefix=rng.choice([0, 0, 4, 70]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                    slopes=rng.random() < 0.25, docs=rng.random() < 0.25)
    if op == "append":
        q_heads, kv_heads = rng.choice([(32, 8), (64, 8), (48, 8), (4, 4), (16, 2), (8, 1)])
        seqs = _log_int(rng, 1, 200)
        hi = max(1, min(_log_int(rng, 1, 6000), 6000 // seqs))
        return dict(op=op, seqs=seqs, rows_lo=rng.choice([0, 1, hi]), rows_hi=hi, q_heads=q_heads, kv_heads=kv_heads,
                    page=rng.choice([16, 32, 64, 128]), len_lo=rng.choice([0, 1, 77]), len_hi=_log_int(rng, 100, 4000),
                    rotary=rng.choice([0, 32, 64, 128, 128, 20]), yarn=rng.choice([0.0, 0.0, 4.0]))
    if op == "logits":
        vocab = _log_int(rng, 1000, 160000)
        rows = max(1, min(_log_int(rng, 1, 256), int(2.5e7 / vocab)))
        return dict(op=op, rows=rows, vocab=vocab, history=_log_int(rng, 1, 8000),
                    type=rng.choice(["float32", "bfloat16"]), bias=rng.random() < 0.5, mask=rng.random() < 0.5)
    return dict(op=op, rows=rng.randint(1, 16), hidden=256 * rng.choice([1, 2, 4, 6, 8]),
                vocab=_log_int(rng, 1000, 151936))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced in their logarithm, in a fixed mixed order."""
    if n == 1:
        return [hi]
    v = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, n) == 1)
    return [v[(i * step) % n] for i in range(n)]


def _attention_shape(c):
    """Per sequence: committed length, rows, first visible position."""
    lens = _spread(c["len_lo"], c["len_hi"], c["seqs"])
    rows = [c["rows"] - (i * 5) % (1 + c["rows"] // 2) for i in range(c["seqs"])]
    first = [(n // 3 if i % 2 else 0) if c["docs"] else 0 for i, n in enumerate(lens)]
    return lens, rows, first


def _append_shape(c):
    return _spread(c["len_lo"], c["len_hi"], c["seqs"]), _spread(c["rows_lo"], c["rows_hi"], c["seqs"])


def work(c):
    if c["op"] == "attention":
        lens, rows, first = _attention_shape(c)
        seen = pairs = 0
        for n, r, f in zip(lens, rows, first):
            low = n + 1  # lowest position that some row sees beyond the prefix
            kept = 0
            for i in range(r):
                p = n + i
                w = max(f, p - c["window"] + 1) if c["window"] else f
                pre = max(0, min(c["prefix"], w) - f)
                pairs += p + 1 - w + pre
                low, kept = min(low, w), max(kept, min(c["prefix"], n + 1))
            seen += n + r - low + max(0, min(kept, low) - f)
        t = sum(rows)
        return {"bytes": seen * c["kv_heads"] * 4 * HD + t * c["q_heads"] * (4 * HD + 4),
                "flops": 4 * HD * c["q_heads"] * pairs}
    if c["op"] == "append":
        t = sum(_append_shape(c)[1])
        return {"bytes": max(1, t) * (c["q_heads"] + 2 * c["kv_heads"]) * 4 * HD, "flops": 0}
    if c["op"] == "logits":
        b = c["rows"] * c["vocab"] * (8 if c["type"] == "float32" else 4) + c["rows"] * 8
        b += -(-c["rows"] // 4) * c["history"] * 4
        b += 2 * c["vocab"] * 4 if c["bias"] else 0
        b += 4 * -(-c["vocab"] // 32) * 4 if c["mask"] else 0
        return {"bytes": b, "flops": 0}
    return {"bytes": 2 * c["hidden"] * (c["vocab"] + c["rows"]) + 4 * c["rows"] * c["vocab"],
            "flops": 2 * c["rows"] * c["hidden"] * c["vocab"]}


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def _pages(c, lens, rows, g, values):
    """The page pool (``values``: filled as a running server's, else empty) and the sequences' tables: pages in no
    order, entries past a sequence's own pages -1."""
    ps = c["page"]
    need = [-(-(n + r) // ps) for n, r in zip(lens, rows)]
    width, total = max(need + [1]), sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    rank = torch.arange(width, device="cuda").repeat(len(need), 1)
    n = torch.tensor(need, device="cuda")[:, None]
    at = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")[:, None] + rank
    table = torch.where(rank < n, order[at.clamp(max=total - 1)], torch.full_like(order[:1], -1))
    shape = (total, c["kv_heads"], ps, HD)
    if values:
        k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    else:
        k, v = (torch.zeros(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    return k, v, table.contiguous()


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("attention", "append"):
        if c["op"] == "attention":
            lens, rows, first = _attention_shape(c)
        else:
            lens, rows = _append_shape(c)
        t = sum(rows)
        s["k"], s["v"], s["table"] = _pages(c, lens, rows, g, c["op"] == "attention")
        s["len"], s["start"] = _ints(lens), _offsets(rows)
        s["o"] = torch.zeros(t, c["q_heads"] * HD, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "attention":
        # queries that make some positions stand out, as trained heads do
        s["q"] = (2.5 * torch.randn(t, c["q_heads"] * HD, generator=g, device="cuda")).bfloat16()
        s["lse"] = torch.zeros(t, c["q_heads"], dtype=torch.float32, device="cuda")
        s["first"] = _ints(first) if c["docs"] else None
        s["prefix"] = _ints([min(c["prefix"], n + 1) for n in lens]) if c["prefix"] else None
        s["slopes"] = (2.0 ** -(8.0 * torch.arange(1, c["q_heads"] + 1, device="cuda") / c["q_heads"])
                       if c["slopes"] else None)
    elif c["op"] == "append":
        # one fused projection's output: q, k and v are column ranges of its rows
        w = c["q_heads"] + 2 * c["kv_heads"]
        s["qkv"] = torch.randn(t, w * HD, generator=g, device="cuda", dtype=torch.bfloat16)
    elif c["op"] == "logits":
        r, vocab = c["rows"], c["vocab"]
        s["logits"] = (3 * torch.randn(r, vocab, generator=g, device="cuda")).to(getattr(torch, c["type"]))
        s["out"] = torch.empty_like(s["logits"])
        s["tok"] = torch.empty(r, dtype=torch.int32, device="cuda")
        s["best"] = torch.empty(r, dtype=torch.float32, device="cuda")
        # blocks of four rows: one history each, of which row i sees i tokens more (the drafts before it)
        each = c["history"] + 3
        blocks = -(-r // 4)
        u = torch.rand(blocks * each, generator=g, device="cuda")
        s["tokens"] = (u ** 4 * vocab).to(torch.int32).clamp(max=vocab - 1)
        s["begin"] = _ints([(i // 4) * each for i in range(r)])
        s["end"] = _ints([(i // 4) * each + (c["history"] if i // 4 != 1 else 0) + i % 4 for i in range(r)])
        s["repetition"] = 1 + 0.3 * torch.rand(r, generator=g, device="cuda")
        s["presence"] = torch.rand(r, generator=g, device="cuda")
        s["frequency"] = 0.5 * torch.rand(r, generator=g, device="cuda")
        s["bias"] = s["bias_row"] = s["allow"] = s["allow_row"] = None
        if c["bias"]:
            b = 4 * torch.randn(2, vocab, generator=g, device="cuda")
            s["bias"] = b * (torch.rand(2, vocab, generator=g, device="cuda") < 0.02)
            s["bias_row"] = _ints([i % 3 - 1 for i in range(r)])
        if c["mask"]:
            words = (4, -(-vocab // 32))
            bits = torch.randint(-2**31, 2**31, words, generator=g, device="cuda").to(torch.int32)
            for _ in range(4):  # the first mask lets few tokens through, as a grammar does
                bits[0] &= torch.randint(-2**31, 2**31, words[1:], generator=g, device="cuda").to(torch.int32)
            s["allow"], s["allow_row"] = bits, _ints([i % 5 - 1 for i in range(r)])
    else:
        s["x"] = torch.randn(c["rows"], c["hidden"], generator=g, device="cuda", dtype=torch.bfloat16)
        s["W"] = (0.02 * torch.randn(c["vocab"], c["hidden"], generator=g, device="cuda")).bfloat16()
        s["logits"] = torch.empty(c["rows"], c["vocab"], dtype=torch.float32, device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a server keeps between calls: the cache and rule descriptions and the workspace."""
    import moe_nvfp4_block_gb300 as M
    c = s["case"]
    s["M"] = M
    if c["op"] in ("attention", "append"):
        s["kv"] = M.PagedKV(s["k"], s["v"], s["table"], s["len"])
        s["ws"] = M.paged_workspace(s["kv"], c["rows"] if c["op"] == "attention" else 1, c["q_heads"])
    if c["op"] == "attention":
        s["scores"] = M.PagedScores(window=c["window"], softcap=c["softcap"], slopes=s["slopes"], first=s["first"],
                                    prefix=s["prefix"])
    elif c["op"] == "append":
        s["pos"] = M.attn_pos(rotary_dim=c["rotary"], rope_theta=_theta(c), yarn_factor=c["yarn"], yarn_orig_ctx=4096)
    elif c["op"] == "logits":
        s["rules"] = M.LogitRules(tokens=s["tokens"], begin=s["begin"], end=s["end"], repetition=s["repetition"],
                                  presence=s["presence"], frequency=s["frequency"], bias=s["bias"],
                                  bias_row=s["bias_row"], allow=s["allow"], allow_row=s["allow_row"])
        s["ws"] = M.logits_workspace(c["rows"], c["vocab"])
    else:
        s["ws"] = M.lm_head_workspace(c["rows"])


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"attention": _attention, "append": _append, "logits": _logits, "lm_head": _lm_head}[c["op"]](s, c)


def _own(s, c):
    M = s["M"]
    if c["op"] == "attention":
        M.moe_paged_attention(s["kv"], s["q"], s["start"], s["o"], s["ws"], max_rows=c["rows"], scores=s["scores"],
                              lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "append":
        q, k, v = _columns(s, c)
        M.moe_paged_kv_append(s["kv"], k, v, s["start"], s["ws"], q=q, q_out=s["o"], pos=s["pos"])
        return {"q": s["o"], "k": s["k"], "v": s["v"]}
    if c["op"] == "logits":
        M.moe_logits_constrain(s["logits"], s["rules"], s["ws"], out=s["out"], tok=s["tok"], best=s["best"])
        return {"out": s["out"], "tok": s["tok"], "best": s["best"]}
    M.moe_lm_head_logits(s["x"], s["W"], s["logits"], s["ws"])
    return s["logits"]


def _columns(s, c):
    a, b = c["q_heads"] * HD, (c["q_heads"] + c["kv_heads"]) * HD
    return s["qkv"][:, :a], s["qkv"][:, a:b], s["qkv"][:, b:]


def _rows_of(start, t):
    """The sequence of each of the t rows, and the row's place in it."""
    at = torch.arange(t, device="cuda")
    b = torch.searchsorted(start.long(), at, right=True) - 1
    return b, at - start.long()[b]


def _theta(c):
    return 500000.0 if c["yarn"] else 10000.0


def _frequencies(c):
    """Angle per position of each rotary pair, in 64 bits (with YaRN's ramp between 1 and 32 turns over 4096)."""
    rd = c["rotary"]
    f = torch.tensor(_theta(c), dtype=torch.float64, device="cuda") ** (
        -2.0 * torch.arange(rd // 2, dtype=torch.float64, device="cuda") / rd)
    if c["yarn"] > 1:
        ramp = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = (1 - ramp) * f / c["yarn"] + ramp * f
    return f


def _turn(x, cos, sin):
    """x [t][heads][128]: pairs (i, i + n) of the first 2 n dims turned by the row's angles."""
    n = cos.shape[-1]
    a, b, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _append(s, c):
    q, k, v = _columns(s, c)
    t, ps = q.shape[0], c["page"]
    b, i = _rows_of(s["start"], t)
    p = s["len"].long()[b] + i
    q, k, v = (x.reshape(t, -1, HD) for x in (q, k, v))
    if c["rotary"]:
        angle = p.double()[:, None] * _frequencies(c)
        cos, sin = angle.cos().float(), angle.sin().float()
        q, k = (_turn(x.float(), cos, sin).bfloat16() for x in (q, k))
    s["o"].copy_(q.reshape(t, -1))
    page = s["table"].long()[b, p // ps]
    s["k"][page, :, p % ps] = k
    s["v"][page, :, p % ps] = v
    return {"q": s["o"], "k": s["k"], "v": s["v"]}


def _attention(s, c):
    t, n_seq, kr, nq, nkv = s["q"].shape[0], c["seqs"], c["rows"], c["q_heads"], c["kv_heads"]
    group = nq // nkv
    b, i = _rows_of(s["start"], t)
    q = torch.zeros(n_seq, kr, nq, HD, device="cuda")
    q[b, i] = s["q"].float().reshape(t, nq, HD)
    q = q.reshape(n_seq, kr, nkv, group, HD).permute(0, 2, 1, 3, 4).reshape(n_seq, nkv, kr * group, HD)
    table = s["table"].long().clamp(min=0)
    k, v = (x[table].float().transpose(1, 2).reshape(n_seq, nkv, -1, HD) for x in (s["k"], s["v"]))
    x = q @ k.transpose(-1, -2) / math.sqrt(HD)
    del k
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.reshape(n_seq, nkv, kr, group, -1)
    p = torch.arange(x.shape[-1], device="cuda")
    pos = s["len"].long()[:, None, None] + torch.arange(kr, device="cuda")[:, None]
    if c["slopes"]:
        x = x + s["slopes"].reshape(nkv, 1, group, 1) * (p - pos)[:, None, :, None, :]
    see = p <= pos
    if c["window"]:
        near = p > pos - c["window"]
        see = see & (near | (p < s["prefix"].long()[:, None, None]) if c["prefix"] else near)
    if c["docs"]:
        see = see & (p >= s["first"].long()[:, None, None])
    x = torch.where(see[:, None, :, None, :], x, torch.full_like(x[:1, :1, :1, :1, :1], -math.inf))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(n_seq, nkv, kr * group, -1) @ v).reshape(n_seq, nkv, kr, group, HD)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(-1)
    s["o"].copy_(o.permute(0, 2, 1, 3, 4).reshape(n_seq, kr, nq * HD)[b, i].bfloat16())
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(n_seq, kr, nq)[b, i])
    return {"o": s["o"], "lse": s["lse"]}


def _logits(s, c):
    r, vocab = c["rows"], c["vocab"]
    n = (s["end"] - s["begin"]).long()
    row = torch.repeat_interleave(torch.arange(r, device="cuda"), n)
    at = torch.arange(row.numel(), device="cuda") - (n.cumsum(0) - n)[row] + s["begin"].long()[row]
    count = torch.zeros(r, vocab, device="cuda")
    count.index_put_((row, s["tokens"][at].long()), torch.ones((), device="cuda"), accumulate=True)
    x = s["logits"].float()
    rep = s["repetition"][:, None]
    hit = torch.where(x > 0, x / rep, x * rep) - (s["presence"][:, None] + count * s["frequency"][:, None])
    x = torch.where(count > 0, hit, x)
    if c["bias"]:
        b = s["bias_row"].long()
        x = torch.where((b >= 0)[:, None], x + s["bias"][b.clamp(min=0)], x)
    if c["mask"]:
        a = s["allow_row"].long()
        v = torch.arange(vocab, device="cuda")
        bit = (s["allow"][a.clamp(min=0)][:, v // 32] >> (v % 32).to(torch.int32)) & 1
        x = torch.where((bit == 1) | (a < 0)[:, None], x, torch.full_like(x[:1, :1], -math.inf))
    s["out"].copy_(x)
    best = x.amax(1)
    v = torch.arange(vocab, device="cuda", dtype=torch.int32)
    tok = torch.where(x == best[:, None], v, torch.full_like(v[:1], vocab)).amin(1)
    s["tok"].copy_(torch.where(best > -math.inf, tok, torch.full_like(tok, -1)))
    s["best"].copy_(best)
    return {"out": s["out"], "tok": s["tok"], "best": s["best"]}


def _lm_head(s, c):
    torch.matmul(s["x"].float(), s["W"].float().T, out=s["logits"])
    return s["logits"]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(c, seed):
    s = prepare(dict(c), seed)
    if c["op"] == "lm_head":
        return torch.cat([s["x"].double() @ w.double().T for w in s["W"].split(16384)], 1)
    if c["op"] == "logits":
        return _exact_logits(s, c)
    return _exact_append(s, c) if c["op"] == "append" else _exact_attention(s, c)


def _exact_logits(s, c):
    vocab = c["vocab"]
    out = s["logits"].double()
    begin, end = s["begin"].tolist(), s["end"].tolist()
    for r in range(c["rows"]):
        x = out[r]
        seen, count = torch.unique(s["tokens"][begin[r]:end[r]].long(), return_counts=True)
        y = x[seen]
        rep = s["repetition"][r].double()
        y = torch.where(y > 0, y / rep, y * rep)
        x[seen] = y - s["presence"][r].double() - count * s["frequency"][r].double()
        if c["bias"] and r % 3:
            x += s["bias"][r % 3 - 1].double()
        if c["mask"] and r % 5:
            word = s["allow"][r % 5 - 1].cpu().numpy().view("u4")
            bits = ((word[:, None] >> torch.arange(32).numpy().astype("u4")) & 1).reshape(-1)[:vocab]
            x[torch.from_numpy(bits == 0).cuda()] = -math.inf
    return {"out": out, "tok": None, "best": out.amax(1)}


def _exact_append(s, c):
    lens, rows = _append_shape(c)
    q, k, v = (x.double().unflatten(1, (-1, HD)) for x in _columns(s, c))
    rd = c["rotary"]
    pair = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    freq = torch.exp(-2 * pair / max(rd, 1) * math.log(_theta(c)))
    if c["yarn"] > 1:
        turns = 4096 * freq / (2 * math.pi)
        keep = torch.where(turns < 1, 0.0, torch.where(turns > 32, 1.0, (turns - 1) / 31))
        freq = freq * (keep + (1 - keep) / c["yarn"])
    kp, vp, at = s["k"].double(), s["v"].double(), 0
    q, k = q.clone(), k.clone()
    for b, (n, r) in enumerate(zip(lens, rows)):
        p = n + torch.arange(r, device="cuda")
        turn = torch.polar(torch.ones_like(p[:, None] * freq), p[:, None] * freq)[:, None]
        for x in (q, k):
            part = x[at:at + r]
            z = torch.complex(part[..., :rd // 2], part[..., rd // 2:rd]) * turn
            part[..., :rd // 2], part[..., rd // 2:rd] = z.real, z.imag
        page = s["table"][b].long()[p // c["page"]]
        kp[page, :, p % c["page"]] = k[at:at + r]
        vp[page, :, p % c["page"]] = v[at:at + r]
        at += r
    return {"q": q.flatten(1), "k": kp, "v": vp}


def _exact_attention(s, c):
    lens, rows, first = _attention_shape(c)
    group, at = c["q_heads"] // c["kv_heads"], 0
    o = torch.zeros(sum(rows), c["q_heads"], HD, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(rows), c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, r) in enumerate(zip(lens, rows)):
        pages = s["table"][b, :-(-(n + r) // c["page"])].long()
        for h in range(c["kv_heads"]):
            k = s["k"][pages, h].reshape(-1, HD)[:n + r].double()
            v = s["v"][pages, h].reshape(-1, HD)[:n + r].double()
            for i in range(r):
                lo = max(first[b], n + i + 1 - c["window"]) if c["window"] else first[b]
                pre = min(c["prefix"], n + 1)
                p = torch.arange(lo, n + i + 1, device="cuda")
                if pre > first[b] and lo > first[b]:
                    p = torch.cat([torch.arange(first[b], min(pre, lo), device="cuda"), p])
                heads = slice(h * group, (h + 1) * group)
                q = s["q"][at + i].reshape(-1, HD)[heads].double()
                kk, vv = (k, v) if p.numel() == n + r else (k[p], v[p])
                x = q @ kk.T * HD ** -0.5
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                if c["slopes"]:
                    x = x + s["slopes"][heads].double()[:, None] * (p - (n + i)).double()
                lse[at + i, heads] = torch.logsumexp(x, 1)
                o[at + i, heads] = torch.softmax(x, 1) @ vv
        at += r
    return {"o": o.flatten(1), "lse": lse}
