"""The paged-serving operators in 64 bits, row by row, for the tests."""
import math

import torch

HD = 128


def make_cache(lens, rows, nkv, ps, seed, device="cuda", extra_pages=5, spare=2, fill=None):
    """Pages in no order and the sequences' tables (``spare`` more entries
    than needed, -1).  ``fill``: what every slot past a sequence's positions
    holds (None: random)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    need = [-(-(n + r) // ps) for n, r in zip(lens, rows)]
    total = sum(need) + extra_pages
    order = torch.randperm(total, generator=g, device=device)
    table = torch.full((len(lens), max(need + [0]) + spare), -1, dtype=torch.int32, device=device)
    shape = (total, nkv, ps, HD)
    k = torch.randn(shape, generator=g, device=device).bfloat16()
    v = torch.randn(shape, generator=g, device=device).bfloat16()
    if fill is not None:
        keep = torch.zeros(total, ps, dtype=torch.bool, device=device)
    at = 0
    for b, (n, r, m) in enumerate(zip(lens, rows, need)):
        table[b, :m] = order[at:at + m].int()
        if fill is not None:
            p = torch.arange(n + r, device=device)
            keep[order[at:at + m][p // ps], p % ps] = True
        at += m
    if fill is not None:
        hide = ~keep[:, None, :, None].expand(shape)
        k[hide] = fill
        v[hide] = fill
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
    start = ints([sum(rows[:i]) for i in range(len(rows) + 1)])
    return k, v, table, ints(lens), start


def visible(pos, window=0, first=0, prefix=0, device="cuda"):
    p = torch.arange(pos + 1, device=device)
    see = p >= first
    if window:
        see &= (p > pos - window) | (p < prefix)
    return p[see]


def attention(q, k, v, table, lens, rows, nq, window=0, scale=0.0, softcap=0.0, slopes=None, first=None, prefix=None):
    """o, lse and a bound on each lse's error (float64) of every row."""
    nkv, ps = k.shape[1], k.shape[2]
    group, t = nq // nkv, 0
    dev = q.device
    o = torch.zeros(sum(rows), nq, HD, dtype=torch.float64, device=dev)
    lse = torch.full((sum(rows), nq), -math.inf, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(lse)
    scale = scale or HD ** -0.5
    for b, (n, r) in enumerate(zip(lens, rows)):
        for i in range(r):
            p = visible(n + i, window, first[b] if first else 0, prefix[b] if prefix else 0, dev)
            if p.numel():
                page, slot = table[b].long()[p // ps], p % ps
                for h in range(nkv):
                    hs = slice(h * group, (h + 1) * group)
                    kk, vv = k[page, h, slot].double(), v[page, h, slot].double()
                    qq = q[t].reshape(nq, HD)[hs].double()
                    s = qq @ kk.T * scale
                    # 128 products added in FP32 (a step 2^-23 where the sum is cut, not rounded), the
                    # few operations that make the score of it, and the exponential
                    err = (128 * 2.0 ** -23 * (qq.abs() @ kk.abs().T * scale).amax(1) + 2.0 ** -20
                           * (1 + s.abs().amax(1) + softcap))
                    if softcap:
                        s = softcap * torch.tanh(s / softcap)
                    if slopes is not None:
                        bias = slopes[hs].double()[:, None] * (p - (n + i)).double()
                        s = s + bias
                        err = err + 2.0 ** -22 * bias.abs().amax(1)
                    lse[t, hs] = torch.logsumexp(s, 1)
                    o[t, hs] = torch.softmax(s, 1) @ vv
                    bound[t, hs] = err + 2.0 ** -20 * lse[t, hs].abs()
            t += 1
    return o, lse, bound


def check_attention(o, lse, ref, what=""):
    """o to half a bf16 step of each value (2^-8) and, for the FP32 work before
    it, 2^-11 of the row's norm, in the norm of every row and head; rows with
    one or no visible position leave no other room.  lse to its bound."""
    ro, rl, bound = ref
    got = o.double().reshape(ro.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ro)), what
    d = (got - ro).norm(dim=-1)
    room = (2.0 ** -8 + 2.0 ** -11) * ro.norm(dim=-1)
    assert bool((d <= room).all()), f"{what}: o off by {(d / room.clamp(min=1e-30)).max().item():.3f} of its room"
    if lse is not None:
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all()), what
        e = ((lse.double() - rl).abs() / bound.clamp(min=1e-30))[~empty]
        assert e.numel() == 0 or e.max().item() <= 1, f"{what}: lse off by {e.max().item():.3f} of its bound"


def rotary_freqs(rd, theta, yarn=0.0, orig=0):
    f = theta ** (-2.0 * torch.arange(rd // 2, dtype=torch.float64) / max(rd, 1))
    if yarn > 1:
        ramp = ((orig * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = (1 - ramp) * f / yarn + ramp * f
    return f


def rotate(x, pos, freq):
    """x float64 [t, heads, 128] turned at positions pos [t]."""
    n = freq.numel()
    a = (pos.double()[:, None] * freq.to(x.device))[:, None]
    c, s = a.cos(), a.sin()
    lo, hi = x[..., :n], x[..., n:2 * n]
    return torch.cat([lo * c - hi * s, hi * c + lo * s, x[..., 2 * n:]], -1)


def logits(x, tokens=None, begin=None, end=None, repetition=None, presence=None, frequency=None, bias=None,
           bias_row=None, allow=None, allow_row=None):
    """The rules in FP32, operation by operation (each step is one correctly
    rounded FP32 operation, so the values are exact), on CPU tensors."""
    out = x.float().clone()
    R, V = out.shape
    for r in range(R):
        y = out[r]
        if tokens is not None:
            h = tokens[max(0, int(begin[r])):max(0, min(len(tokens), int(end[r])))].long()
            h = h[(h >= 0) & (h < V)]
            c = torch.bincount(h, minlength=V).float()
            rep = repetition[r] if repetition is not None else torch.tensor(1.0)
            pres = presence[r] if presence is not None else torch.tensor(0.0)
            freq = frequency[r] if frequency is not None else torch.tensor(0.0)
            hit = torch.where(y > 0, y / rep, y * rep) - (pres + c * freq)
            y = torch.where(c > 0, hit, y)
        if bias is not None and 0 <= int(bias_row[r]) < bias.shape[0]:
            y = y + bias[int(bias_row[r])]
        if allow is not None and 0 <= int(allow_row[r]) < allow.shape[0]:
            v = torch.arange(V)
            w = allow[int(allow_row[r])].view(torch.int32)[v // 32].long() & 0xFFFFFFFF
            y = torch.where((w >> (v % 32)) & 1 == 1, y, torch.full_like(y, -math.inf))
        out[r] = y
    z = torch.where(torch.isnan(out), torch.full_like(out, -math.inf), out)
    best = z.amax(1)
    tok = torch.where(z == best[:, None], torch.arange(V), torch.tensor(V)).amin(1)
    tok = torch.where(best > -math.inf, tok, torch.tensor(-1))
    return out, tok.int(), best
