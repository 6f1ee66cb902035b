"""Append to and attention over a paged cache of 8 bits, and the normed append to the bf16 cache, against 64 bits."""
import math

import pytest
import torch

import paged8_ref as R8
import paged_ref as R

pytestmark = pytest.mark.gpu

HD = 128
INVALID, TIMEOUT, CAPACITY = -1, -6, -7


@pytest.fixture(autouse=True)
def fp32_default():
    """The files of a run share torch's default type."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(old)


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_nvfp4_block_gb300 as M
    assert torch.cuda.is_available()
    return M


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).bfloat16()


# ---------------------------------------------------------------- append

ROTARY = {"none": None, "whole": dict(rotary_dim=128), "part": dict(rotary_dim=64, rope_theta=5e5, yarn_factor=4.0,
          yarn_orig_ctx=4096), "odd": dict(rotary_dim=20), "small": dict(rotary_dim=2)}


def freqs(name):
    kw = ROTARY[name] or {}
    return R.rotary_freqs(kw.get("rotary_dim", 0), kw.get("rope_theta", 10000.0), kw.get("yarn_factor", 0.0),
                          kw.get("yarn_orig_ctx", 0)).cuda()


def positions(lens, rows):
    return torch.cat([n + torch.arange(r) for n, r in zip(lens, rows)] + [torch.zeros(0, dtype=torch.long)]).cuda()


def check_rows(got, want, x, what):
    """bf16 rows: half a step, and FP32's operations, 16 roundings of a pair's magnitude."""
    room = 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True) + 2.0 ** -133
    d = (got.double() - want).abs()
    assert bool((d <= room).all()), f"{what}: off by {(d / room).max().item():.3f} of its room"


def check_pool(codes, scale, before, want_codes, want_scale, want, y, exact, what):
    """A pool after an append.  exact (no arithmetic before the store): codes and scales bit for bit.  Else a scale may
    differ where the block's largest value is within FP32's error of a border, and a code by the same error."""
    touched = ~torch.isnan(want)
    if exact:
        assert torch.equal(scale, want_scale), what
        assert torch.equal(codes, want_codes), what
        return
    near = (scale.int() - want_scale.int()).abs()
    assert int(near.max()) <= 1 and int((near > 0).sum()) <= 1, what
    same = (near == 0).repeat_interleave(16, -1)[..., None].expand(codes.shape)
    assert torch.equal(codes[~touched & same], want_codes[~touched & same]), what
    got = R8.decode(codes, scale)
    s = torch.exp2(scale.double() - 127).repeat_interleave(16, -1)[..., None].expand(codes.shape)
    big = torch.where(touched, want.abs(), 0).amax(-1, keepdim=True).expand(codes.shape)
    room = 2.0 ** -4 * want.abs() + 2.0 ** -10 * s + 2.0 ** -20 * big
    d = (got - want).abs()
    assert bool((d <= room)[touched].all()), f"{what}: off by {(d / room)[touched].max().item():.3f} of its room"


def append8(M, lens, rows, nq, nkv, ps, rotary="whole", norm=True, seed=0, scale=1.0, gains=True, strided=True,
            inplace=False, with_q=True, extra=0):
    kc, vc, ks, vs, table, length, start = R8.make_cache(lens, rows, nkv, ps, seed)
    T = sum(rows)
    w = nq + 2 * nkv
    qkv = randn(T + extra, w * HD, seed=seed + 7, scale=scale)
    q, k, v = qkv[:, :nq * HD], qkv[:, nq * HD:(nq + nkv) * HD], qkv[:, (nq + nkv) * HD:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    x = qkv.clone()
    qg, kg = (1 + 0.4 * randn(HD, seed=seed + 9).float()).bfloat16(), (1 + 0.4 * randn(HD, seed=seed + 8).float()).bfloat16()
    nm = M.QkNorm(qg if gains else None, kg if gains else None, 1e-5) if norm else None
    pos = M.attn_pos(**ROTARY[rotary]) if ROTARY[rotary] else None
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, nkv)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    out = q if inplace else torch.full((T + extra, nq * HD), 5.0, dtype=torch.bfloat16, device="cuda")
    M.moe_paged_kv8_append(kv, k, v, start, ws, q=q if with_q else None, q_out=out if with_q else None, norm=nm, pos=pos)
    assert M.moe_workspace_error(ws) == 0
    p, f = positions(lens, rows), freqs(rotary)
    eps = 1e-5 if norm else None
    xq, xk, xv = x[:T, :nq * HD], x[:T, nq * HD:(nq + nkv) * HD], x[:T, (nq + nkv) * HD:]
    wq = R8.new_rows(xq, p, f, qg if gains else None, eps)
    wk = R8.new_rows(xk, p, f, kg if gains else None, eps)
    wv = xv.double().unflatten(1, (-1, HD))
    if with_q:
        check_rows(out[:T].unflatten(1, (-1, HD)), wq, xq, "q")
        if extra:
            assert bool((out[T:] == (x[T:, :nq * HD] if inplace else 5.0)).all())
    plain = not norm and rotary == "none"
    ref = R8.store(before[0], before[1], table, lens, rows, ps, wk)
    check_pool(kc, ks, before[0], *ref, wk, plain, "keys")
    ref = R8.store(before[2], before[3], table, lens, rows, ps, wv)
    check_pool(vc, vs, before[2], *ref, wv, True, "values")


LENS = [([0], [1]), ([1], [1]), ([15], [1]), ([15], [2]), ([16], [1]), ([777], [3]), ([5], [16]), ([0], [16]), ([0], [17]),
        ([31], [33]), ([9], [130]), ([3, 0, 40, 16, 100], [1, 4, 0, 2, 3]), ([7, 15, 0], [0, 0, 0]), ([64, 1, 127], [5, 64, 1])]


@pytest.mark.parametrize("lens,rows", LENS)
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("norm", [False, True])
def test_append_lengths(M, lens, rows, ps, norm):
    append8(M, lens, rows, 4, 2, ps, norm=norm, seed=len(rows) + sum(lens))


@pytest.mark.parametrize("nq,nkv", [(32, 8), (1, 1), (3, 3), (48, 8), (10, 5), (8, 1), (6, 2)])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 9])
def test_append_heads(M, nq, nkv, rows):
    append8(M, [20, 33, 14], [rows, rows, rows], nq, nkv, 32, seed=nq + rows)


@pytest.mark.parametrize("rotary", list(ROTARY))
@pytest.mark.parametrize("norm,gains", [(False, True), (True, False), (True, True)])
def test_append_rotary_widths(M, rotary, norm, gains):
    append8(M, [30, 0, 4090], [5, 18, 2], 5, 2, 128, rotary=rotary, norm=norm, gains=gains, seed=3)


@pytest.mark.parametrize("kw", [dict(strided=False), dict(inplace=True), dict(inplace=True, rotary="odd"), dict(with_q=False),
                                dict(extra=5), dict(extra=5, inplace=True), dict(scale=1e-30), dict(scale=1e30, norm=False),
                                dict(scale=3e-38, norm=False, rotary="none"), dict(scale=1e15), dict(ps=16), dict(ps=32)])
def test_append_forms(M, kw):
    kw = dict(ps=64) | kw
    append8(M, [12, 45, 3], [4, 7, 20], 6, 3, kw.pop("ps"), seed=11, **kw)


@pytest.mark.parametrize("n", [1000, 700])
def test_append_of_many_sequences(M, n):
    lens = [(37 * i) % 90 for i in range(n)]
    append8(M, lens, [(i * 7) % 3 for i in range(n)], 2, 1, 16, seed=n)


def test_append_of_prompts(M):
    append8(M, [3, 1000, 0], [2001, 1503, 900], 4, 2, 64, seed=2)


def one_block(M, com, com_byte, new, ps=16):
    """Appends `new` [r, 128] (bf16) behind `com` committed positions (codes i % 120, scale `com_byte`) of one block;
    the page's codes, its scale, and what they should be."""
    codes = (torch.arange(16 * HD, device="cuda") % 120).to(torch.uint8).reshape(1, 1, 16, HD)
    scale = torch.full((1, 1, 1), com_byte, dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = codes.clone(), codes.clone(), scale.clone(), scale.clone()
    table, start, length = ints([[0]]), ints([0, new.shape[0]]), ints([com])
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 1)
    M.moe_paged_kv8_append(kv, new, new, start, ws)
    assert M.moe_workspace_error(ws) == 0
    want = R8.store(codes, scale, table, [com], [new.shape[0]], 16, new.double().unflatten(1, (-1, HD)))
    assert torch.equal(kc, vc) and torch.equal(ks, vs)
    return kc, ks, want


@pytest.mark.parametrize("com", [0, 1, 7, 15])
@pytest.mark.parametrize("byte", [1, 100, 119, 121, 128, 160, 254])
def test_a_scale_grows_and_never_shrinks(M, com, byte):
    kc, ks, want = one_block(M, com, byte, randn(1, HD, seed=byte))
    assert torch.equal(ks, want[1]) and torch.equal(kc, want[0])
    if com == 0:
        assert int(ks) in (119, 120, 121)
    else:
        assert int(ks) >= byte


@pytest.mark.parametrize("big", [448.0, 449.0, 464.0, 1.75, 1.7578125, 2.0 ** -133, 3.3895313892515355e38, 0.0])
def test_scales_at_borders(M, big):
    x = torch.zeros(2, HD, dtype=torch.bfloat16, device="cuda")
    x[1, 77] = -big
    x[0, 3] = big / 1000
    kc, ks, want = one_block(M, 0, 7, x)
    assert torch.equal(ks, want[1]) and torch.equal(kc, want[0])


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("com", [0, 5])
def test_infinite_and_nan_values_become_nan_alone(M, what, com):
    x = randn(3, HD, seed=4)
    x[1, 9] = what
    kc, ks, want = one_block(M, com, 119, x)
    got = kc.view(torch.float8_e4m3fn).double()
    ref = want[0].view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and bool(torch.isnan(got[0, 0, com + 1, 9]))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref)) and torch.equal(ks, want[1])
    x[:] = what  # nothing finite
    kc, ks, _ = one_block(M, 0, 200, x)
    assert int(ks) == 1 and bool(torch.isnan(kc.view(torch.float8_e4m3fn).double()[0, 0, :3]).all())


def test_a_nan_scale_stays(M):
    kc, ks, _ = one_block(M, 4, 255, randn(2, HD))
    assert int(ks) == 255 and bool(torch.isnan(kc.view(torch.float8_e4m3fn).double()[0, 0, 4:6]).all())


def test_norm_of_zeros_and_of_infinities(M):
    q = torch.zeros(3, HD, dtype=torch.bfloat16, device="cuda")
    q[1, 5] = math.inf
    q[2, 6] = math.nan
    for form in (8, 16):
        if form == 8:
            c = torch.zeros(1, 1, 16, HD, dtype=torch.uint8, device="cuda")
            s = torch.zeros(1, 1, 1, dtype=torch.uint8, device="cuda")
            kv = M.PagedKV8(c, c.clone(), s, s.clone(), ints([[0]]), ints([0]))
        else:
            c = torch.zeros(1, 1, 16, HD, dtype=torch.bfloat16, device="cuda")
            kv = M.PagedKV(c, c.clone(), ints([[0]]), ints([0]))
        ws, o = M.paged_workspace(kv, 1, 1), torch.empty_like(q)
        f = dict(q=q, q_out=o, pos=M.attn_pos(rotary_dim=64))
        nm = M.QkNorm(eps=1e-6)
        if form == 8:
            M.moe_paged_kv8_append(kv, q, q, ints([0, 3]), ws, norm=nm, **f)
        else:
            M.moe_paged_kv_append_norm(kv, nm, q, q, ints([0, 3]), ws, **f)
        assert bool((o[0] == 0).all()) and bool(torch.isnan(o[1]).any()) and bool(torch.isnan(o[2]).any())


@pytest.mark.parametrize("kind", ["capacity", "page", "page2", "length", "rows", "fall"])
def test_append_of_bad_sequences(M, kind):
    """What is wrong in a sequence is recorded; the others are stored."""
    lens, rows = [20, 33, 14], [3, 4, 2]
    kc, vc, ks, vs, table, length, start = R8.make_cache(lens, rows, 2, 16, 1, spare=0)
    x = randn(9, 4 * HD, seed=5)
    err = INVALID
    if kind == "capacity":
        length[1] = table.shape[1] * 16
        err = CAPACITY
    elif kind == "page":
        table[1, 2] = -1
    elif kind == "page2":
        table[1, 2] = kc.shape[0]
    elif kind == "length":
        length[1] = -4
    elif kind == "rows":
        start[3] = 40
    else:
        start = ints([0, 7, 3, 5])
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 2)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    o = torch.full_like(x, 5.0)
    M.moe_paged_kv8_append(kv, x[:, :2 * HD], x[:, 2 * HD:], start, ws, q=x, q_out=o)
    assert M.moe_workspace_error(ws) == err
    at = {"rows": [0, 3, 7], "fall": [0, -1, 3]}.get(kind, [0, 3, 7])
    n = {"rows": [3, 4, 0], "fall": [7, 0, 2]}.get(kind, [3, 0, 2])
    if kind == "fall":  # rows 3 and 4 are the third sequence's; the first one has the others
        return
    k = x[:, :2 * HD].double().unflatten(1, (-1, HD))
    y = torch.cat([k[a:a + m] for a, m in zip(at, n)])
    want = R8.store(before[0], before[1], table, lens, n, 16, y)
    assert torch.equal(kc, want[0]) and torch.equal(ks, want[1])
    if kind == "rows":
        assert bool((o[7:] == 5.0).all()) and torch.equal(o[:7], x[:7])
    else:  # queries go through all the same
        assert torch.equal(o, x)


def test_row_starts_that_overlap_stay_in_bounds(M):
    kc, vc, ks, vs, table, length, _ = R8.make_cache([20, 33, 14], [30, 30, 30], 2, 16, 1)
    x = randn(40, 4 * HD, seed=5)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 2)
    runs = []
    for _ in range(2):
        o = torch.zeros_like(x)
        M.moe_paged_kv8_append(kv, x[:, :2 * HD], x[:, 2 * HD:], ints([0, 30, 10, 40]), ws, q=x, q_out=o,
                               pos=M.attn_pos(rotary_dim=128))
        runs.append((o, kc.clone(), ks.clone()))
        assert M.moe_workspace_error(ws) == INVALID
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_appends_in_steps_and_again(M):
    """Row by row, and the same rows once more (a rejected draft's place): what the cache stands for stays near."""
    kc, vc, ks, vs, table, length, _ = R8.make_cache([0], [40], 2, 16, 1)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 2)
    x = randn(40, 2 * HD, seed=5)
    x *= torch.exp2(torch.arange(40, device="cuda") % 7)[:, None].bfloat16()
    for t in range(40):
        length.fill_(t)
        for _ in range(2):
            M.moe_paged_kv8_append(kv, x[t:t + 1], x[t:t + 1], ints([0, 1]), ws)
    page, slot = table[0].long()[torch.arange(40, device="cuda") // 16], torch.arange(40, device="cuda") % 16
    got = R8.decode(kc, ks)[page, :, slot].flatten(1)
    s = torch.exp2(ks.double() - 127)[page, :, slot // 16].repeat_interleave(HD, -1)
    # a rounding to E4M3, and where the scale grew more of them, each at most half a step of the last scale's subnormals
    room = 2.0 ** -4 * x.double().abs() + 7 * 2.0 ** -10 * s
    assert bool(((got - x.double()).abs() <= room).all())


def test_row_starts_that_fall(M):
    """The second sequence's rows are wrong; the third's two lie within the first's seven, which has the other five."""
    lens = [20, 33, 14]
    kc, vc, ks, vs, table, length, _ = R8.make_cache(lens, [7, 4, 2], 2, 16, 1, spare=0)
    x = randn(9, 4 * HD, seed=5)
    x[3] *= 64  # (the largest: not the first sequence's)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 2)
    before = [t.clone() for t in (kc, ks, vc, vs)]
    o = torch.full_like(x, 5.0)
    M.moe_paged_kv8_append(kv, x[:, :2 * HD], x[:, 2 * HD:], ints([0, 7, 3, 5]), ws, q=x, q_out=o)
    assert M.moe_workspace_error(ws) == INVALID
    assert torch.equal(o[:7], x[:7]) and bool((o[7:] == 5.0).all())
    pos = 20 + torch.arange(3, 5, device="cuda")
    gap = table[0].long()[pos // 16], slice(None), pos % 16
    for codes, scale, old, old_scale, cols in ((kc, ks, before[0], before[1], slice(0, 2 * HD)),
                                               (vc, vs, before[2], before[3], slice(2 * HD, 4 * HD))):
        y = x[:, cols].double().unflatten(1, (-1, HD))
        first = y[:7].clone()
        first[3:5] = 0
        want, want_scale, _ = R8.store(old, old_scale, table, lens, [7, 0, 2], 16, torch.cat([first, y[3:5]]))
        want[gap] = old[gap]  # what the first sequence's rows leave free stays
        assert torch.equal(codes, want) and torch.equal(scale, want_scale)


@pytest.mark.parametrize("big", [1.0, 64.0, 2.0 ** 14, 2.0 ** 30])
def test_rounds_of_rejected_outliers(M, big):
    """Three of four rows are rejected each round, `big` times the committed ones: the cache is what the rule gives, and
    what is committed is off by its rounding and, of blocks whose scale has grown, by half a step of the last scale's
    smallest at each growth."""
    kc, vc, ks, vs, table, length, _ = R8.make_cache([0], [70], 2, 16, 1)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, 1, 2)
    x = randn(64, 4, 2 * HD, seed=5)
    x[:, 1:] *= big
    for t in range(64):
        length.fill_(t)
        before = kc.clone(), ks.clone()
        M.moe_paged_kv8_append(kv, x[t], x[t], ints([0, 4]), ws)
        want = R8.store(*before, table, [t], [4], 16, x[t].double().unflatten(1, (-1, HD)))
        assert torch.equal(kc, want[0]) and torch.equal(ks, want[1])
    assert M.moe_workspace_error(ws) == 0
    p = torch.arange(64, device="cuda")
    page, slot = table[0].long()[p // 16], p % 16
    got, y = R8.decode(kc, ks)[page, :, slot].flatten(1), x[:, 0].double()
    s = torch.exp2(ks.double() - 127)[page, :, slot // 16].repeat_interleave(HD, -1)
    # (a scale grows by whole powers of two: roundings of half steps 2^-10 s, s/2, s/4 .. add up to less than 2^-9 s)
    assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -9 * s).all())


# ---------------------------------------------------------------- the normed append to the bf16 cache

@pytest.mark.parametrize("nq,nkv", [(32, 8), (1, 1), (48, 8), (10, 5), (6, 2)])
@pytest.mark.parametrize("rotary", ["whole", "part", "odd", "none"])
@pytest.mark.parametrize("gains", [False, True])
def test_normed_append(M, nq, nkv, rotary, gains):
    lens, rows, ps = [20, 0, 33, 14], [3, 0, 17, 1], 32
    k0, v0, table, length, start = R.make_cache(lens, rows, nkv, ps, 3)
    T = sum(rows)
    qkv = randn(T + 2, (nq + 2 * nkv) * HD, seed=nq)
    q, k, v = qkv[:, :nq * HD], qkv[:, nq * HD:(nq + nkv) * HD], qkv[:, (nq + nkv) * HD:]
    kc, vc = k0.clone(), v0.clone()
    qg, kg = (1 + 0.4 * randn(HD, seed=1).float()).bfloat16(), (1 + 0.4 * randn(HD, seed=2).float()).bfloat16()
    if not gains:
        qg = kg = None
    kv = M.PagedKV(kc, vc, table, length)
    ws = M.paged_workspace(kv, 1, nkv)
    out = torch.full((T + 2, nq * HD), 5.0, dtype=torch.bfloat16, device="cuda")
    pos = M.attn_pos(**ROTARY[rotary]) if ROTARY[rotary] else None
    M.moe_paged_kv_append_norm(kv, M.QkNorm(qg, kg, 1e-5), k, v, start, ws, q=q, q_out=out, pos=pos)
    assert M.moe_workspace_error(ws) == 0
    p, f = positions(lens, rows), freqs(rotary)
    check_rows(out[:T].unflatten(1, (-1, HD)), R8.new_rows(q[:T], p, f, qg, 1e-5), q, "q")
    assert bool((out[T:] == 5.0).all())
    at = 0
    for b, (n, r) in enumerate(zip(lens, rows)):
        pp = n + torch.arange(r, device="cuda")
        page = table[b].long()[pp // ps]
        want = R8.new_rows(k[at:at + r], pp, f, kg, 1e-5)
        check_rows(kc[page, :, pp % ps], want, k, "k")
        assert torch.equal(vc[page, :, pp % ps].flatten(1), v[at:at + r])
        k0[page, :, pp % ps] = kc[page, :, pp % ps]
        v0[page, :, pp % ps] = vc[page, :, pp % ps]
        at += r
    assert torch.equal(k0, kc) and torch.equal(v0, vc)
    # over the queries
    M.moe_paged_kv_append_norm(kv, M.QkNorm(qg, kg, 1e-5), k, v, start, ws, q=q, q_out=q, pos=pos)
    assert torch.equal(q[:T], out[:T])


# ---------------------------------------------------------------- attention

def attend(M, lens, rows, nq, nkv, ps, seed=0, max_rows=None, cache=None, q=None, qscale=2.5, want_lse=True, ref=True,
           scale=0.0, softcap=0.0, window=0, slopes=False, first=None, prefix=None, inplace=False, extra=0):
    kc, vc, ks, vs, table, length, start = cache or R8.make_cache(lens, rows, nkv, ps, seed)
    T = sum(rows)
    if q is None:
        q = randn(T + extra, nq * HD, seed=seed + 5, scale=qscale)
    sl = torch.exp2(-8.0 * torch.arange(1, nq + 1, device="cuda") / nq) if slopes else None
    sc = M.PagedScores(window=window, scale=scale, softcap=softcap, slopes=sl, first=None if first is None else ints(first),
                       prefix=None if prefix is None else ints(prefix))
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    mr = max_rows or max(rows + [1])
    ws = M.paged_workspace(kv, mr, nq)
    q0 = q.clone()
    o = q if inplace else torch.full((T + extra, nq * HD), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + extra, nq), 5.0, device="cuda") if want_lse else None
    M.moe_paged_kv8_attention(kv, q, start, o, ws, mr, scores=sc, lse=lse)
    assert M.moe_workspace_error(ws) == 0
    if extra:
        assert bool((o[T:] == (q0[T:] if inplace else 5.0)).all()) and bool((lse[T:] == 5.0).all())
    if ref:
        want = R8.attention(q0[:T], R8.decode(kc, ks), R8.decode(vc, vs), R8.scales(vs), table, lens, rows, nq, window=window, scale=scale,
                            softcap=softcap, slopes=sl, first=first, prefix=prefix)
        R8.check_attention(o[:T], None if lse is None else lse[:T], want, f"{lens} {rows} {nq}/{nkv} {ps}")
    return o, lse, (kv, ws, q0, start, sc)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 63, 127, 128, 129, 255, 256, 300, 2011])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_attention_lengths(M, n, ps):
    attend(M, [n], [1], 8, 2, ps, seed=n)


@pytest.mark.parametrize("nq,nkv,rows", [(32, 8, 1), (32, 8, 4), (8, 8, 1), (1, 1, 16), (4, 1, 4), (4, 1, 5), (4, 1, 8),
                                         (64, 8, 4), (64, 8, 8), (32, 8, 16), (28, 4, 3), (12, 4, 11), (5, 1, 9), (7, 7, 16)])
def test_attention_heads_and_rows(M, nq, nkv, rows):
    attend(M, [700, 3, 0, 161], [rows, 1, rows, max(1, rows - 1)], nq, nkv, 32, seed=rows)


FORMS = [dict(window=1), dict(window=17), dict(window=128), dict(window=200, prefix=[4, 0, 70, 1]),
         dict(window=64, prefix=[300, 300, 300, 300]), dict(softcap=20.0), dict(softcap=1e4), dict(slopes=True),
         dict(slopes=True, softcap=30.0, window=100), dict(first=[0, 10, 600, 40]), dict(first=[800, 800, 800, 800]),
         dict(first=[5, 0, 130, 161], window=50, prefix=[20, 3, 140, 170]), dict(scale=0.3), dict(scale=1e-3),
         dict(first=[-5, 2 ** 31 - 1, 0, 3])]


@pytest.mark.parametrize("kw", FORMS)
@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, 3), (16, 2, 4), (16, 1, 4)])
def test_attention_masks_and_scores(M, kw, nq, nkv, rows):
    ref = dict(kw)
    if "first" in kw:
        kw = kw | dict(first=[max(-5, x) for x in kw["first"]])
    attend(M, [700, 30, 640, 161], [rows, rows, 1, rows], nq, nkv, 32, seed=2, **ref)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, 1), (8, 2, 8), (8, 1, 8)])
def test_attention_over_many_cut_units(M, ps, nq, nkv, rows):
    lens = [(977 * i) % 3001 + 1 for i in range(23)]
    attend(M, lens, [1 + i % rows for i in range(23)], nq, nkv, ps, seed=ps, max_rows=rows)


@pytest.mark.parametrize("nq,nkv,rows", [(8, 8, 1), (32, 8, 4), (64, 8, 8)])
def test_attention_over_long_caches(M, nq, nkv, rows):
    attend(M, [40001], [rows], nq, nkv, 64, seed=1)


def wide(cache, n_max):
    """The cache with a table of n_max pages a sequence (beyond what they hold: no page)."""
    table = torch.full((cache[4].shape[0], n_max), -1, dtype=torch.int32, device="cuda")
    table[:, :cache[4].shape[1]] = cache[4]
    return cache[:4] + (table,) + cache[5:]


@pytest.mark.parametrize("nq,nkv,rows", [(4, 1, 5), (8, 1, 4), (32, 8, 8), (17, 1, 1), (10, 5, 16), (24, 8, 7)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(slopes=True), dict(first=[3, 700, 0], prefix=[0, 710, 4])])
def test_17_to_32_rows_in_wide_tables(M, nq, nkv, rows, kw):
    """The form that 17 to 32 query rows a KV head have over tables with room for long sequences."""
    lens, rows = [2500, 700, 0], [rows, max(1, rows - 1), rows]
    attend(M, lens, rows, nq, nkv, 32, seed=nq, cache=wide(R8.make_cache(lens, rows, nkv, 32, nq), 40000), **kw)


@pytest.mark.parametrize("rows", [5, 8])
def test_17_to_32_rows_over_long_caches(M, rows):
    lens = [40001, 77]
    attend(M, lens, [rows, 2], 32, 8, 64, seed=2, max_rows=rows)
    lens = [(977 * i) % 3001 + 1 for i in range(19)]
    rows = [1 + i % rows for i in range(19)]
    attend(M, lens, rows, 32, 8, 64, seed=3, max_rows=8, cache=wide(R8.make_cache(lens, rows, 8, 64, 3), 300))


@pytest.mark.parametrize("rows", [5, 8, 16])
def test_a_call_again_and_in_place_gives_the_same_bits(M, rows):
    """Units that are whole and units that several CTAs share, many segments a CTA."""
    lens = [(977 * i) % 3001 for i in range(40)] + [30001]
    n = [1 + (i * 7) % rows for i in range(40)] + [rows]
    cache = wide(R8.make_cache(lens, n, 4, 64, rows), 500)
    q = randn(sum(n), 16 * HD, seed=rows, scale=2.5)
    first = attend(M, lens, n, 16, 4, 64, max_rows=rows, cache=cache, q=q.clone())[:2]
    for inplace in (False, True):
        again = attend(M, lens, n, 16, 4, 64, max_rows=rows, cache=cache, q=q.clone(), inplace=inplace, ref=False)[:2]
        assert all(torch.equal(x, y) for x, y in zip(first, again)), inplace


def test_attention_over_more_sequences_than_threads(M):
    lens = [(13 * i) % 150 for i in range(1024)]
    attend(M, lens, [i % 2 for i in range(1024)], 2, 1, 16, seed=1)


@pytest.mark.parametrize("kw", [dict(inplace=True), dict(extra=3), dict(extra=3, inplace=True), dict(want_lse=False)])
def test_attention_forms(M, kw):
    for nq, rows in ((8, 2), (16, 4), (16, 8)):
        attend(M, [300, 9, 0, 45], [rows, 1, 0, rows], nq, 2, 32, seed=3, **kw)


@pytest.mark.parametrize("rows,nq", [(1, 4), (4, 8), (8, 8)])
def test_hidden_positions_may_hold_anything(M, rows, nq):
    """Codes and scales of NaN behind and before what the rows see (and between, under a window)."""
    lens, ps = [200, 37], 16
    cache = R8.make_cache(lens, [rows] * 2, 1, ps, 4)
    q = randn(2 * rows, nq * HD, seed=5)
    kw = dict(window=40, prefix=[5, 3], cache=cache, q=q, ref=False)
    o, lse, _ = attend(M, lens, [rows] * 2, nq, 1, ps, **kw)
    kc, vc, ks, vs, table, _, _ = cache
    for b, n in enumerate(lens):
        last = n + rows
        p = torch.arange(table.shape[1] * ps, device="cuda")
        low = n - 40 + 1
        hide = (p >= last) | ((p >= kw["prefix"][b]) & (p < low))
        ok = table[b].long()[p // ps] >= 0
        hp = p[hide & ok]
        page = table[b].long()[hp // ps]
        kc[page, :, hp % ps] = 0x7F
        vc[page, :, hp % ps] = 0xFF
        whole = [a for a in range(0, len(p), 16) if bool(hide[a:a + 16].all()) and bool(ok[a])]
        for a in whole:
            pg = int(table[b, a // ps])
            ks[pg, :, a % ps // 16] = 255
            vs[pg, :, a % ps // 16] = 255
    # (slices with such values are summed position by position, so that a last bit of o may differ)
    o2, lse2, _ = attend(M, lens, [rows] * 2, nq, 1, ps, **(kw | dict(ref=True)))
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("kw", [dict(), dict(window=300, prefix=[20 + 7 * i for i in range(17)]), dict(softcap=20.0)])
@pytest.mark.parametrize("rows,ps", [(9, 16), (16, 64), (16, 128)])
def test_nan_behind_long_sequences_stays_hidden(M, rows, ps, kw):
    """Codes of NaN in every position that no row sees, in units of one to 32 chunks, several segments a CTA: the last
    chunks (and, under a window, the first) are looked over after many whose values every row sees."""
    lens = [(977 * i) % 4001 + 1 for i in range(17)]
    n = [1 + (i * 5) % rows for i in range(17)]
    n[3] = rows
    cache = R8.make_cache(lens, n, 4, ps, rows)
    kc, vc, _, _, table, _, _ = cache
    for b, (m, r) in enumerate(zip(lens, n)):
        p = torch.arange(-(-(m + r) // ps) * ps, device="cuda")
        hide = p >= m + r
        if "window" in kw:
            hide |= (p >= kw["prefix"][b]) & (p <= m - kw["window"])
        p = p[hide]
        page = table[b].long()[p // ps]
        kc[page, :, p % ps] = 0x7F
        vc[page, :, p % ps] = 0xFF
    q = randn(sum(n), 16 * HD, seed=rows, scale=2.5)
    first = attend(M, lens, n, 16, 4, ps, max_rows=rows, cache=cache, q=q, **kw)[:2]
    for _ in range(20):
        again = attend(M, lens, n, 16, 4, ps, max_rows=rows, cache=cache, q=q, ref=False, **kw)[:2]
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("rows,nq", [(4, 4), (4, 8), (8, 8)])
@pytest.mark.parametrize("what", ["value", "value scale", "key", "key scale"])
def test_nan_is_seen_by_those_that_see_it(M, rows, nq, what):
    """NaN at the last row's own position: the rows before it must not notice."""
    n, ps = 130, 16
    cache = R8.make_cache([n], [rows], 1, ps, 4)
    kc, vc, ks, vs, table, _, _ = cache
    q = randn(rows, nq * HD, seed=5)
    clean, lse0, _ = attend(M, [n], [rows], nq, 1, ps, cache=cache, q=q)
    p = n + rows - 1
    page, slot = int(table[0, p // ps]), p % ps
    if what == "value":
        vc[page, 0, slot, 7] = 0x7F
    elif what == "key":
        kc[page, 0, slot, 7] = 0x7F
    o, lse, _ = attend(M, [n], [rows], nq, 1, ps, cache=cache, q=q, ref="scale" not in what)
    if what == "value":
        assert torch.equal(torch.isnan(o[-1].reshape(nq, HD)[:, 7]), torch.ones(nq, dtype=torch.bool, device="cuda"))
        assert torch.equal(lse, lse0)
    if what == "key":
        assert bool(torch.isnan(o[-1]).all()) and bool(torch.isnan(lse[-1]).all())
    if "scale" not in what:
        assert torch.equal(torch.isnan(o[:-1]), torch.zeros_like(o[:-1], dtype=torch.bool))
        return
    # a whole block of NaN that only the last rows see: its first position is the last row's
    n = 144 - rows + 1
    cache = R8.make_cache([n], [rows], 1, ps, 4)
    kc, vc, ks, vs, table, _, _ = cache
    (vs if what.startswith("value") else ks)[int(table[0, 9]), 0, 0] = 255
    o, lse, _ = attend(M, [n], [rows], nq, 1, ps, cache=cache, q=q)
    assert bool(torch.isnan(o[-1]).all()) and not bool(torch.isnan(o[:-1]).any())


@pytest.mark.parametrize("kb,vb", [(1, 1), (30, 236), (127, 236), (100, 3), (150, 127), (0, 0)])
@pytest.mark.parametrize("rows", [1, 8, 16])
def test_attention_scales_of_any_size(M, kb, vb, rows):
    """Scales from the smallest (and byte 0) to the largest whose 316 values' sum stays in FP32: 448 * 2^109 * 316 < 2^127."""
    lens = [300]
    cache = list(R8.make_cache(lens, [rows], 1, 32, 4))
    cache[2] = torch.full_like(cache[2], kb)
    cache[3] = torch.full_like(cache[3], vb)
    q = randn(rows, 4 * HD, seed=5, scale=2.0 ** max(-100, min(20, 118 - kb)))
    attend(M, lens, [rows], 4, 1, 32, cache=tuple(cache), q=q)


@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("spread", [7, 12, 40, 100])
@pytest.mark.parametrize("n", [40, 300, 3000])
def test_attention_value_scales_apart(M, rows, spread, n):
    """Blocks of values whose scales differ by up to 2^spread either way, one of 0 and the smallest scale among them."""
    cache = list(R8.make_cache([n, 70], [rows, 1], 1, 32, 4))
    g = torch.Generator(device="cuda")
    g.manual_seed(spread)
    cache[3] = (119 + torch.randint(-spread, spread + 1, cache[3].shape, generator=g, device="cuda")).to(torch.uint8)
    cache[3][:, :, 1] = cache[3][:, :, 1].clamp(max=119)
    cache[3][1] = 1
    cache[1][1] = 0
    attend(M, [n, 70], [rows, 1], 4, 1, 32, cache=tuple(cache), seed=spread)


@pytest.mark.parametrize("rows", [1, 8, 16])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e4, 1e25])
def test_queries_of_any_size(M, rows, scale):
    lens = [150]
    cache = R8.make_cache(lens, [rows], 1, 32, 4)
    q = randn(rows, 4 * HD, seed=5, scale=scale)
    attend(M, lens, [rows], 4, 1, 32, cache=cache, q=q, scale=0.1 / max(scale, 1e-20))


@pytest.mark.parametrize("rows", [1, 8, 16])
def test_infinite_queries_give_what_the_formula_gives(M, rows):
    cache = R8.make_cache([50], [rows], 1, 32, 4)
    q = randn(rows, 4 * HD, seed=5)
    q[0, 3] = math.inf
    q[0, HD + 5] = math.nan
    o, lse, _ = attend(M, [50], [rows], 4, 1, 32, cache=cache, q=q, ref=False)
    assert bool(torch.isnan(o[0, :2 * HD]).all()) and not bool(torch.isnan(o[0, 2 * HD:]).any())
    assert not bool(torch.isnan(o[1:]).any())


@pytest.mark.parametrize("what", ["page", "capacity", "length", "rows", "many"])
@pytest.mark.parametrize("nq", [4, 8, 16])
def test_attention_of_bad_sequences(M, what, nq):
    lens, rows = [200, 100, 50], [2, 3, 4]
    cache = list(R8.make_cache(lens, rows, 1, 16, 4, spare=0))
    q = randn(9, nq * HD, seed=5)
    clean, lse0, _ = attend(M, lens, rows, nq, 1, 16, cache=tuple(cache), q=q)
    table, length, start = cache[4:]
    err, mr = INVALID, 4
    if what == "page":
        table[1, 3] = 10 ** 6
    elif what == "capacity":
        length[1] = table.shape[1] * 16 - 1
        err = CAPACITY
    elif what == "length":
        length[1] = -7
    elif what == "rows":
        start[3] = 30
    else:
        mr = 3
    kv = M.PagedKV8(*cache[:4], table, length)
    ws = M.paged_workspace(kv, mr, nq)
    o, lse = torch.full_like(clean, 5.0), torch.full_like(lse0, 5.0)
    M.moe_paged_kv8_attention(kv, q, start, o, ws, mr, lse=lse)
    assert M.moe_workspace_error(ws) == err
    bad = slice(5, 9) if what in ("rows", "many") else slice(2, 5)
    good = [i for i in range(9) if not bad.start <= i < bad.stop]
    if what != "page":
        assert bool((o[bad] == 5.0).all()) and bool((lse[bad] == 5.0).all())
    # the others' sums may be cut in other places: two roundings, and 2^-11 of each weight times a mean |v| below 8
    assert bool(((o[good].double() - clean[good].double()).abs() <= 2.0 ** -7 * clean[good].double().abs() + 2.0 ** -7).all())
    # the workspace serves the next call
    kv = M.PagedKV8(*R8.make_cache(lens, rows, 1, 16, 4, spare=0)[:6])
    M.moe_paged_kv8_attention(kv, q, ints([0, 2, 5, 9]), o, M.paged_workspace(kv, 4, nq), 4)


@pytest.mark.parametrize("nq", [4, 8, 16])
def test_a_wait_that_runs_out_is_recorded(M, nq):
    cache = R8.make_cache([3000, 70], [4, 4], 1, 32, 4)
    q = randn(8, nq * HD, seed=5)
    o, lse, (kv, ws, _, start, sc) = attend(M, [3000, 70], [4, 4], nq, 1, 32, cache=cache, q=q)
    M.moe_debug_set_wait_limit_ns(0)
    try:
        M.moe_paged_kv8_attention(kv, q, start, torch.empty_like(o), ws, 4)
        assert M.moe_workspace_error(ws) == TIMEOUT
    finally:
        M.moe_debug_set_wait_limit_ns(2_000_000_000)
    ws.zero_()
    again = torch.empty_like(o)
    M.moe_paged_kv8_attention(kv, q, start, again, ws, 4, scores=sc)
    assert M.moe_workspace_error(ws) == 0 and torch.equal(again, o)


@pytest.mark.parametrize("nq", [4, 8, 16])
def test_attention_captured_replayed_and_on_two_streams(M, nq):
    lens, rows = [900, 100, 37], [4, 4, 2]
    cache = R8.make_cache(lens, rows, 2, 32, 4)
    q = randn(10, 2 * nq * HD, seed=5)
    o, lse, (kv, ws, _, start, sc) = attend(M, lens, rows, 2 * nq, 2, 32, cache=cache, q=q)
    ws2 = M.paged_workspace(kv, 4, 2 * nq)
    a, b = torch.empty_like(o), torch.empty_like(o)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1):
        M.moe_paged_kv8_attention(kv, q, start, a, ws, 4)
    with torch.cuda.graph(g2):  # the same workspace, another length
        M.moe_paged_kv8_attention(kv, q, start, b, ws, 4)
    for _ in range(3):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(b, o)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.zero_()
    b.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        M.moe_paged_kv8_attention(kv, q, start, a, ws, 4, stream=s1)
        M.moe_paged_kv8_attention(kv, q, start, b, ws2, 4, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(b, o) and M.moe_workspace_error(ws) == 0


def test_equal_calls_give_equal_bits(M):
    for nq in (8, 16, 32):
        x = [attend(M, [5000, 33, 2100], [4, 2, 1], nq, 2, 64, seed=9, ref=False)[0] for _ in range(3)]
        assert torch.equal(x[0], x[1]) and torch.equal(x[0], x[2])


@pytest.mark.parametrize("nq,rows", [(4, 3), (8, 4), (16, 4)])
def test_caches_past_four_gigabytes(M, nq, rows):
    """Pages whose codes lie beyond 2^32 bytes: appended to and attended over."""
    ps, n_pages, lens = 128, 290_000, [260, 100]
    shape = (n_pages, 1, ps, HD)  # 4.75e9 bytes each
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(shape[:2] + (ps // 16,), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = ints([[n_pages - 1, 5, n_pages - 9], [n_pages - 4, -1, -1]])
    length = ints([0, 0])
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, rows, nq)
    x = randn(sum(lens) + 2 * rows, 2 * HD, seed=3)
    M.moe_paged_kv8_append(kv, x[:, :HD], x[:, HD:], ints([0, lens[0] + rows, x.shape[0]]), ws)
    length.copy_(ints(lens))
    used = table.long().clamp(min=0).flatten().unique()
    small = torch.searchsorted(used, table.long().clamp(min=0)).int()  # the same pages in a small pool
    y = x.double().unflatten(1, (-1, HD))
    empty = torch.zeros((len(used),) + shape[1:], dtype=torch.uint8, device="cuda"), torch.zeros((len(used), 1, ps // 16), dtype=torch.uint8, device="cuda")
    n = [m + rows for m in lens]
    for codes, scale, z in ((kc, ks, y[:, :1]), (vc, vs, y[:, 1:])):
        want = R8.store(*empty, small, [0, 0], n, ps, z)
        assert torch.equal(codes[used], want[0]) and torch.equal(scale[used], want[1])
    attend(M, lens, [rows] * 2, nq, 1, ps, cache=(kc[used], vc[used], ks[used], vs[used], small, length, ints([0, rows, 2 * rows])))
    q = randn(2 * rows, nq * HD, seed=5, scale=2.5)
    o, p = torch.empty_like(q), torch.empty_like(q)
    M.moe_paged_kv8_attention(kv, q, ints([0, rows, 2 * rows]), o, ws, rows)
    kv2 = M.PagedKV8(kc[used], vc[used], ks[used], vs[used], small, length)
    M.moe_paged_kv8_attention(kv2, q, ints([0, rows, 2 * rows]), p, M.paged_workspace(kv2, rows, nq), rows)
    assert torch.equal(o, p) and M.moe_workspace_error(ws) == 0


@pytest.mark.parametrize("nq,rows", [(4, 3), (8, 4), (16, 4)])
def test_a_padded_batch_and_strided_rows(M, nq, rows):
    """Rows behind the last sequence's stay as they were; q and o are column ranges of wider rows."""
    lens = [300, 40]
    kc, vc, ks, vs, table, length, start = R8.make_cache(lens, [rows] * 2, 1, 32, 4)
    wide = randn(2 * rows + 5, (nq + 3) * HD, seed=5, scale=2.5)
    out = torch.full_like(wide, 7.0)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, rows, nq)
    q, o = wide[:, HD:(nq + 1) * HD], out[:, 2 * HD:(nq + 2) * HD]
    M.moe_paged_kv8_attention(kv, q, start, o, ws, rows)
    want = R8.attention(q[:2 * rows], R8.decode(kc, ks), R8.decode(vc, vs), R8.scales(vs), table, lens, [rows] * 2, nq)
    R8.check_attention(o[:2 * rows], None, want)
    assert bool((out[2 * rows:] == 7.0).all()) and bool((out[:, :2 * HD] == 7.0).all()) and bool((out[:, (nq + 2) * HD:] == 7.0).all())


def test_both_caches_of_one_workspace_in_turn(M):
    """Calls of every form, and of the pool, share a workspace in one stream."""
    lens, ps = [500, 20], 32
    c8 = R8.make_cache(lens, [4, 4], 1, ps, 4)
    c16 = R.make_cache(lens, [4, 4], 1, ps, 4)
    kv8, kv16 = M.PagedKV8(*c8[:6]), M.PagedKV(*c16[:4])
    ws = M.paged_workspace(kv8, 4, 16)
    start, free = ints([0, 4, 8]), ints([0, 1, 2, 3])
    pool = M.PagePool(ints([[-1] * 4] * 2), ints([0, 0]), free, ints([4]), ps)
    first = {}
    for turn in range(3):
        for nq in (4, 8, 16):
            q = randn(8, nq * HD, seed=nq)
            for kv, f in ((kv8, M.moe_paged_kv8_attention), (kv16, M.moe_paged_attention)):
                o = torch.empty_like(q)
                f(kv, q, start, o, ws, 4)
                assert torch.equal(first.setdefault((nq, f), o), o)
            M.moe_paged_reserve(pool, ints([0, 0]), ints([40, 3]), ints([0] * 3), ws)
            M.moe_paged_release(pool, ints([0, 0]), ws)
    assert M.moe_workspace_error(ws) == 0 and free.tolist() == [0, 1, 2, 3]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("nq", [8, 16])
def test_serving_rounds(M, ps, nq):
    """Reserve, append, attend, commit and release, in a captured step with a padded batch, as a server runs them."""
    nkv, n, K, width = 2, 5, 4, 40
    lens, T = [0, 30, 200, 15, 64], n * K
    pages = 200
    kc, vc = (torch.zeros(pages, nkv, ps, HD, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, nkv, ps // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    length, held, free = ints([0] * n), ints([0] * n), torch.randperm(pages, device="cuda").int()
    n_free, rows, start = ints([pages]), ints(lens), ints([0] * (n + 1))
    granted = ints([0] * n)
    pool = M.PagePool(table, held, free, n_free, ps)
    kv = M.PagedKV8(kc, vc, ks, vs, table, length)
    ws = M.paged_workspace(kv, K, nq)
    gain = (1 + 0.3 * randn(HD, seed=3).float()).bfloat16()
    nm, pos = M.QkNorm(gain, gain, 1e-6), M.attn_pos(rotary_dim=HD)
    # the prompts
    qkv = randn(sum(lens), (nq + 2 * nkv) * HD, seed=1)
    keys = [[] for _ in range(n)]
    values = [[] for _ in range(n)]
    M.moe_paged_reserve(pool, length, rows, start, ws, granted=granted)
    M.moe_paged_kv8_append(kv, qkv[:, nq * HD:(nq + nkv) * HD], qkv[:, (nq + nkv) * HD:], start, ws, norm=nm, pos=pos)
    assert granted.tolist() == [1] * n
    at = 0
    for b, r in enumerate(lens):
        x = qkv[at:at + r]
        keys[b].append(R8.new_rows(x[:, nq * HD:(nq + nkv) * HD], torch.arange(r, device="cuda"), freqs("whole"), gain, 1e-6))
        values[b].append(x[:, (nq + nkv) * HD:].double().unflatten(1, (-1, HD)))
        at += r
    length.copy_(rows)
    # the captured step
    x = torch.zeros(T + 3, (nq + 2 * nkv) * HD, dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :nq * HD], x[:, nq * HD:(nq + nkv) * HD], x[:, (nq + nkv) * HD:]
    qt, o = torch.zeros(T + 3, nq * HD, dtype=torch.bfloat16, device="cuda"), torch.zeros(T + 3, nq * HD, dtype=torch.bfloat16, device="cuda")
    slot = ints([0] * (T + 3))

    def step():
        M.moe_paged_reserve(pool, length, rows, start, ws, slot=slot)
        M.moe_paged_kv8_append(kv, k, v, start, ws, q=q, q_out=qt, norm=nm, pos=pos)
        M.moe_paged_kv8_attention(kv, qt, start, o, ws, K)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    cur = list(lens)
    for t in range(6):
        r = [(b + t) % (K + 1) for b in range(n)]
        rows.copy_(ints(r))
        x.copy_(randn(*x.shape, seed=50 + t))
        g.replay()
        assert M.moe_workspace_error(ws) == 0
        st = start.tolist()
        f = freqs("whole")
        for b in range(n):
            p = cur[b] + torch.arange(r[b], device="cuda")
            mine = slice(st[b], st[b] + r[b])
            assert slot[mine].tolist() == (table[b].long()[p // ps] * ps + p % ps).tolist()
            nk = R8.new_rows(k[mine], p, f, gain, 1e-6)
            nv = v[mine].double().unflatten(1, (-1, HD))
            # the cache against what was appended: E4M3's half step, and of what its scale leaves
            pp = torch.arange(cur[b] + r[b], device="cuda")
            page = table[b].long()[pp // ps]
            for pool8, sc8, past, new in ((kc, ks, keys[b], nk), (vc, vs, values[b], nv)):
                want = torch.cat(past + [new])
                got = R8.decode(pool8, sc8)[page, :, pp % ps]
                s = torch.exp2(sc8.double() - 127)[page, :, pp % ps // 16][..., None]
                room = 2.0 ** -4 * want.abs() + 6 * 2.0 ** -10 * s + 2.0 ** -20 * want.abs().amax(-1, keepdim=True)
                assert bool(((got - want).abs() <= room).all())
            take = min(r[b], 1 + (b * t) % 3)  # accepted rows
            keys[b].append(nk[:take])
            values[b].append(nv[:take])
            cur[b] += take
        want = R8.attention(qt[:st[n]], R8.decode(kc, ks), R8.decode(vc, vs), R8.scales(vs), table, length.tolist(), r, nq)
        R8.check_attention(o[:st[n]], None, want, f"step {t}")
        assert slot[st[n]:].tolist() == [-1] * (T + 3 - st[n])
        length.copy_(ints(cur))
        M.moe_paged_release(pool, length, ws)
        assert held.tolist() == [-(-c // ps) for c in cur]
    M.moe_paged_release(pool, ints([0] * n), ws)
    assert n_free.tolist() == [pages] and sorted(free.tolist()) == list(range(pages))
    assert bool((table == -1).all()) and M.moe_workspace_error(ws) == 0


@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("nq", [8, 16])
def test_serving_with_a_pool_that_runs_short(M, ps, nq):
    """A captured step (reserve, append, attention) in which two of four sequences get no page: the others are served and
    every cache is as it should be; with pages back, the same step serves all."""
    nkv, width, pages, K = 2, 8, 40, 4
    lens, T, w = [2 * ps - 2, 4 * ps - 2, 3 * ps - 2, ps + 4], 16, nq + 2 * nkv
    kc, vc = (torch.zeros(pages, nkv, ps, HD, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, nkv, ps // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    length, held, free = ints([0] * 4), ints([0] * 4), torch.randperm(pages, device="cuda").int()
    n_free, rows, start, granted = ints([pages]), ints(lens), ints([0] * 5), ints([0] * 4)
    pool, kv = M.PagePool(table, held, free, n_free, ps), M.PagedKV8(kc, vc, ks, vs, table, length)
    ws, f = M.paged_workspace(kv, K, nq), freqs("whole")
    gain = (1 + 0.3 * randn(HD, seed=3).float()).bfloat16()
    nm, pos = M.QkNorm(gain, gain, 1e-6), M.attn_pos(rotary_dim=HD)
    x0 = randn(sum(lens), w * HD, seed=1)
    M.moe_paged_reserve(pool, length, rows, start, ws, granted=granted)
    M.moe_paged_kv8_append(kv, x0[:, nq * HD:(nq + nkv) * HD], x0[:, (nq + nkv) * HD:], start, ws, norm=nm, pos=pos)
    assert granted.tolist() == [1] * 4 and held.tolist() == [2, 4, 3, 2] and M.moe_workspace_error(ws) == 0
    length.copy_(ints(lens))
    rows.fill_(K)
    x = randn(T, w * HD, seed=2)
    q, k, v = x[:, :nq * HD], x[:, nq * HD:(nq + nkv) * HD], x[:, (nq + nkv) * HD:]
    qt, o, slot = torch.zeros(T, nq * HD, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, nq * HD, dtype=torch.bfloat16, device="cuda"), ints([0] * T)

    def step():
        M.moe_paged_reserve(pool, length, rows, start, ws, slot=slot, granted=granted)
        M.moe_paged_kv8_append(kv, k, v, start, ws, q=q, q_out=qt, norm=nm, pos=pos)
        M.moe_paged_kv8_attention(kv, qt, start, o, ws, K)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    nk = R8.new_rows(k, torch.cat([n + torch.arange(K, device="cuda") for n in lens]), f, gain, 1e-6)
    nv = v.double().unflatten(1, (-1, HD))
    left = int(n_free)
    for have, ok in ((1, [1, 0, 0, 1]), (left - 1, [1, 1, 1, 1])):
        n_free.fill_(have)
        before = [t.clone() for t in (kc, ks, vc, vs)]
        g.replay()
        assert M.moe_workspace_error(ws) == (0 if all(ok) else CAPACITY)
        assert granted.tolist() == ok and start.tolist() == [0, 4, 8, 12, 16]
        # a sequence without its page: its rows go as far as the pages it holds
        stored = [K if y else 2 for y in ok]
        mine = torch.cat([4 * b + torch.arange(r, device="cuda") for b, r in enumerate(stored)])
        check_pool(kc, ks, before[0], *R8.store(before[0], before[1], table, lens, stored, ps, nk[mine]), nk, False, "keys")
        check_pool(vc, vs, before[2], *R8.store(before[2], before[3], table, lens, stored, ps, nv[mine]), nv, True, "values")
        want = R8.attention(qt, R8.decode(kc, ks), R8.decode(vc, vs), R8.scales(vs), table, lens, [K] * 4, nq)
        served = torch.cat([4 * b + torch.arange(K, device="cuda") for b in range(4) if ok[b]])
        R8.check_attention(o[served], None, tuple(t[served] for t in want), f"{ok}")
        for b in range(4):
            p = lens[b] + torch.arange(K, device="cuda")
            assert slot[4 * b:4 * b + 4].tolist() == ((table[b].long()[p // ps] * ps + p % ps).tolist() if ok[b] else [-1] * K)
        if have == 1:
            assert n_free.tolist() == [0] and held.tolist() == [3, 4, 3, 2]
            free.copy_(torch.roll(free, -1))  # the others come back
    assert held.tolist() == [3, 5, 4, 2]
