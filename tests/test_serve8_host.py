"""The operators around a paged cache of 8 bits on the host (no GPU needed): the arguments they refuse before anything
is enqueued, and the references of the GPU tests against themselves."""
import ctypes

import pytest
import torch

import paged8_ref as R8
from test_serve_host import BAD_CACHES, fp32_default, kv, M  # noqa: F401

OK, INVALID, SHAPE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4


def kv8(M, **kw):
    d = dict(kpages=16, vpages=16, kscale=16, vscale=16, table=16, kv_len=16, n_pages=10, page_size=64, nkv=8,
             head_dim=128, n_seqs=3, max_pages=4)
    d.update(kw)
    return M.moe_paged_kv8(**d)


def norm(M, **kw):
    return M.moe_qk_norm(**(dict(q_gain=16, k_gain=16, eps=1e-6) | kw))


def append8(M, c=None, nm=None, q=16, qs=1024, k=16, ks=1024, v=16, vs=1024, n=5, nq=8, start=16, pos=None, qo=16,
            qos=1024, ws=16, wsb=256):
    c = c if c is not None else kv8(M)
    return M.lib.moe_paged_kv8_append(ctypes.byref(c), None if nm is None else ctypes.byref(nm), q, qs, k, ks, v, vs, n,
                                      nq, start, None if pos is None else ctypes.byref(pos), qo, qos, ws, wsb, None)


def append_norm(M, c=None, nm=None, q=16, qs=1024, k=16, ks=1024, v=16, vs=1024, n=5, nq=8, start=16, pos=None, qo=16,
                qos=1024, ws=16, wsb=256):
    c = c if c is not None else kv(M)
    return M.lib.moe_paged_kv_append_norm(ctypes.byref(c), None if nm is None else ctypes.byref(nm), q, qs, k, ks, v, vs,
                                          n, nq, start, None if pos is None else ctypes.byref(pos), qo, qos, ws, wsb, None)


def attention8(M, c=None, q=16, qs=4096, n=5, max_rows=2, nq=32, start=16, sc=None, o=16, os_=4096, lse=None, ws=16,
               wsb=1 << 30):
    c = c if c is not None else kv8(M)
    return M.lib.moe_paged_kv8_attention(ctypes.byref(c), q, qs, n, max_rows, nq, start,
                                         None if sc is None else ctypes.byref(sc), o, os_, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES + [(dict(kscale=None), INVALID), (dict(vscale=None), INVALID),
                                                    (dict(kscale=17), ALIGN), (dict(vscale=24), ALIGN)])
def test_bad_caches_are_refused(M, kw, status):
    assert append8(M, kv8(M, **kw)) == status
    if kw != dict(nkv=0):
        assert attention8(M, kv8(M, **kw)) == status
    else:
        assert attention8(M, kv8(M, **kw)) != OK
    if "kscale" not in kw and "vscale" not in kw:
        assert append_norm(M, kv(M, **kw), norm(M)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(start=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(n=-1), INVALID), (dict(nq=0), INVALID),
    (dict(ks=1000), INVALID), (dict(qs=512), INVALID), (dict(ks=1028), ALIGN), (dict(k=20), ALIGN),
    (dict(q=8), ALIGN), (dict(qo=18), ALIGN), (dict(start=18), ALIGN), (dict(ws=8), ALIGN), (dict(wsb=255), WORKSPACE),
    (dict(qos=2048), INVALID)])
def test_append_refusals(M, kw, status):
    assert append8(M, **kw) == status
    assert append8(M, nm=norm(M), **kw) == status
    assert append_norm(M, nm=norm(M), **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                                       (dict(eps=float("inf")), INVALID), (dict(q_gain=8), ALIGN), (dict(k_gain=18), ALIGN)])
def test_bad_norms_are_refused(M, kw, status):
    assert append8(M, nm=norm(M, **kw)) == status
    assert append_norm(M, nm=norm(M, **kw)) == status


def test_the_normed_append_wants_a_norm(M):
    assert append_norm(M) == INVALID
    assert append_norm(M, nm=norm(M, q_gain=None, k_gain=None), n=0) == OK


@pytest.mark.parametrize("kw,status", [(dict(rotary_dim=129), SHAPE), (dict(rotary_dim=7), SHAPE),
                                       (dict(rotary_dim=64, rope_theta=1.0), INVALID),
                                       (dict(rotary_dim=64, yarn_factor=4.0, yarn_orig_ctx=0), INVALID)])
def test_append_refuses_bad_rotary(M, kw, status):
    assert append8(M, pos=M.attn_pos(**kw)) == status
    assert append_norm(M, nm=norm(M), pos=M.attn_pos(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(start=None), INVALID), (dict(ws=None), INVALID),
    (dict(n=-1), INVALID), (dict(nq=0), INVALID), (dict(nq=12), SHAPE), (dict(max_rows=0), INVALID),
    (dict(max_rows=17), SHAPE), (dict(max_rows=9, nq=64), SHAPE), (dict(qs=4088), INVALID), (dict(os_=4100), ALIGN),
    (dict(q=24), ALIGN), (dict(o=8), ALIGN), (dict(lse=18), ALIGN), (dict(wsb=1000), WORKSPACE),
    (dict(q=16, o=16, os_=4104), INVALID)])
def test_attention_refusals(M, kw, status):
    assert attention8(M, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(softcap=float("inf")), INVALID), (dict(slopes=18), ALIGN), (dict(first=18), ALIGN), (dict(prefix=18), ALIGN)])
def test_attention_refuses_bad_scores(M, kw, status):
    assert attention8(M, sc=M.moe_paged_scores(**kw)) == status


def test_no_rows_is_no_work(M):
    assert append8(M, n=0, q=None, qo=None, k=None, v=None) == OK
    assert attention8(M, n=0, q=None, o=None) == OK
    assert append_norm(M, nm=norm(M), n=0, q=None, qo=None, k=None, v=None) == OK


def pool(M, **kw):
    d = dict(table=16, held=16, free_pages=16, n_free=16, n_pages=10, page_size=64, n_seqs=3, max_pages=4)
    d.update(kw)
    return M.moe_page_pool(**d)


def reserve(M, p=None, kv_len=16, rows=16, n=5, start=16, slot=16, pos=16, granted=16, ws=16, wsb=256):
    p = p if p is not None else pool(M)
    return M.lib.moe_paged_reserve(ctypes.byref(p), kv_len, rows, n, start, slot, pos, granted, ws, wsb, None)


def release(M, p=None, keep=16, shared=None, ws=16, wsb=256):
    p = p if p is not None else pool(M)
    return M.lib.moe_paged_release(ctypes.byref(p), keep, shared, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), INVALID), (dict(held=None), INVALID), (dict(free_pages=None), INVALID), (dict(n_free=None), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_seqs=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_seqs=1025), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=100), SHAPE), (dict(page_size=256), SHAPE), (dict(page_size=0), SHAPE),
    (dict(n_pages=1 << 25), SHAPE), (dict(max_pages=1 << 25), SHAPE), (dict(table=18), ALIGN), (dict(held=17), ALIGN),
    (dict(free_pages=19), ALIGN), (dict(n_free=18), ALIGN)])
def test_bad_pools_are_refused(M, kw, status):
    assert reserve(M, pool(M, **kw)) == status
    assert release(M, pool(M, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kv_len=None), INVALID), (dict(rows=None), INVALID), (dict(start=None), INVALID), (dict(n=-1), INVALID),
    (dict(n=0), INVALID), (dict(n=0, slot=None), INVALID), (dict(ws=None), INVALID), (dict(ws=24), ALIGN),
    (dict(wsb=255), WORKSPACE), (dict(kv_len=18), ALIGN), (dict(rows=18), ALIGN), (dict(start=18), ALIGN),
    (dict(slot=18), ALIGN), (dict(pos=18), ALIGN), (dict(granted=18), ALIGN)])
def test_reserve_refusals(M, kw, status):
    assert reserve(M, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(keep=None), INVALID), (dict(ws=None), INVALID), (dict(ws=24), ALIGN),
                                       (dict(wsb=255), WORKSPACE), (dict(keep=18), ALIGN), (dict(shared=18), ALIGN)])
def test_release_refusals(M, kw, status):
    assert release(M, **kw) == status


def test_pool_calls_refuse_arrays_that_overlap(M):
    n, wide, pages, rows = 3, 4, 10, 5
    size = dict(table=n * wide, held=n, free_pages=pages, n_free=1, kv_len=n, rows=n, start=n + 1, slot=rows, pos=rows, granted=n)
    buf = (ctypes.c_int32 * 1000)()
    base = (ctypes.addressof(buf) + 63) & ~63

    def call(over=None, by=0):
        """A reserve whose arrays lie apart, but for one that begins `by` ints behind another's begin."""
        at, addr = base, {}
        for name, k in size.items():
            addr[name], at = at, at + 4 * (k + 2)
        if over:
            addr[over[0]] = addr[over[1]] + 4 * by
        p = pool(M, n_seqs=n, max_pages=wide, n_pages=pages, **{k: addr.pop(k) for k in ("table", "held", "free_pages", "n_free")})
        return (reserve(M, p, n=rows, **addr), release(M, p, keep=addr["kv_len"], shared=addr["rows"]))

    for x in size:
        for y in size:
            reads = {x, y} <= {"kv_len", "rows", "free_pages"}
            if x == y or reads:
                continue
            assert call((x, y), size[y] - 1)[0] == INVALID, (x, y)
            assert call((x, y))[0] == INVALID, (x, y)
    for x, y in [("kv_len", "held"), ("rows", "table"), ("kv_len", "n_free"), ("rows", "free_pages"), ("held", "table")]:
        assert call((x, y))[1] == INVALID, (x, y)


def test_binding_refuses_tensors_it_would_misread(M):
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    k, sc = torch.zeros(6, 2, 32, 128, dtype=u8), torch.zeros(6, 2, 2, dtype=u8)
    table, n = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    c = M.PagedKV8(k, k.clone(), sc, sc.clone(), table, n)
    M.PagedKV8(k.view(torch.float8_e4m3fn), k, sc.view(torch.float8_e8m0fnu), sc, table, n)
    for bad in (dict(kpages=k.view(torch.float8_e5m2)), dict(vpages=k[:5]), dict(kscale=sc[:, :, :1]),
                dict(vscale=sc.float()), dict(kscale=torch.zeros(6, 2, 4, dtype=u8)[:, :, ::2]), dict(table=table.long()),
                dict(kv_len=n[:2])):
        with pytest.raises(ValueError):
            M.PagedKV8(**(dict(kpages=k, vpages=k, kscale=sc, vscale=sc, table=table, kv_len=n) | bad))
    rows, start, ws = torch.zeros(5, 256, dtype=bf), torch.zeros(4, dtype=i32), torch.zeros(1 << 20, dtype=u8)
    kb = torch.zeros(6, 2, 16, 128, dtype=bf)
    cb = M.PagedKV(kb, kb.clone(), table, n)
    with pytest.raises(ValueError):
        M.moe_paged_kv8_append(cb, rows, rows, start, ws)  # a cache of the other kind
    with pytest.raises(ValueError):
        M.moe_paged_kv_append(c, rows, rows, start, ws)
    with pytest.raises(ValueError):
        M.moe_paged_attention(c, rows, start, rows, ws, 2)
    with pytest.raises(ValueError):
        M.moe_paged_kv8_attention(cb, rows, start, rows, ws, 2)
    with pytest.raises(ValueError):
        M.moe_paged_kv8_append(c, rows, rows, start, ws)  # not on a GPU
    with pytest.raises(ValueError):
        M.moe_paged_kv_append_norm(cb, None, rows, rows, start, ws)
    for bad in (dict(q_gain=torch.ones(128)), dict(k_gain=torch.ones(64, dtype=bf)),
                dict(q_gain=torch.ones(256, dtype=bf)[::2])):
        with pytest.raises(ValueError):
            M.QkNorm(**bad)
    ints = lambda *s: torch.zeros(s, dtype=i32)
    for bad in (dict(table=ints(3, 4).long()), dict(held=ints(2)), dict(n_free=ints(2)), dict(free_pages=ints(10).float()),
                dict(free_pages=ints(20)[::2])):
        with pytest.raises(ValueError):
            M.PagePool(**(dict(table=ints(3, 4), held=ints(3), free_pages=ints(10), n_free=ints(1), page_size=16) | bad))
    p = M.PagePool(ints(3, 4), ints(3), ints(10), ints(1), 16)
    for bad in (dict(kv_len=ints(2)), dict(rows=ints(3).long()), dict(row_start=ints(3)), dict(granted=ints(4)),
                dict(slot=ints(5), pos=ints(6))):
        with pytest.raises(ValueError):
            M.moe_paged_reserve(**(dict(pool=p, kv_len=ints(3), rows=ints(3), row_start=ints(4), ws=ws) | bad))
    with pytest.raises(ValueError):
        M.moe_paged_release(p, ints(2), ws)


def test_a_cache_class_of_the_callers_own_is_taken(M, monkeypatch):
    """The calls on a bf16 cache use a few attributes of it, so that any class with these will do."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(6, 2, 16, 128, dtype=bf)
    real = M.PagedKV(k, k.clone(), torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32))

    class Own:
        _ref, nkv, n_seqs, index, device = real._ref, real.nkv, real.n_seqs, real.index, real.device

    calls = []
    monkeypatch.setattr(M, "_call", lambda what, index, stream, f, *args: calls.append((what, args[0])))
    rows, q, start, ws = (torch.zeros(5, 256, dtype=bf), torch.zeros(5, 512, dtype=bf), torch.zeros(4, dtype=i32),
                          torch.zeros(1 << 20, dtype=torch.uint8))
    M.moe_paged_kv_append(Own(), rows, rows, start, ws)
    M.moe_paged_attention(Own(), q, start, q, ws, 2)
    M.moe_paged_kv_append_norm(Own(), M.QkNorm(), rows, rows, start, ws)
    assert calls == [(n, real._ref) for n in ("moe_paged_kv_append", "moe_paged_attention", "moe_paged_kv_append_norm")]

    class Own8(Own):  # a description that the bf16 calls would misread, and one that the 8-bit calls would
        c = M.moe_paged_kv8()

    for f in (lambda: M.moe_paged_kv_append(Own8(), rows, rows, start, ws), lambda: M.moe_paged_attention(Own8(), q, start, q, ws, 2),
              lambda: M.moe_paged_kv8_append(Own(), rows, rows, start, ws), lambda: M.moe_paged_kv8_append(real, rows, rows, start, ws),
              lambda: M.moe_paged_kv8_attention(Own(), q, start, q, ws, 2)):
        with pytest.raises(ValueError):
            f()
    assert len(calls) == 3


def test_slots_and_positions_of_different_lengths_are_refused(M, monkeypatch):
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)
    p = M.PagePool(ints(3, 4), ints(3), ints(10), ints(1), 16)
    calls = []
    monkeypatch.setattr(M, "_call", lambda what, index, stream, f, *args: calls.append(args[3:7]))
    ws = torch.zeros(256, dtype=torch.uint8)
    go = lambda **kw: M.moe_paged_reserve(p, ints(3), ints(3), ints(4), ws, **kw)
    some, none = ints(5), ints(0)
    for bad in (dict(slot=none, pos=some), dict(slot=some, pos=none), dict(slot=ints(4), pos=some), dict(slot=none.float()),
                dict(pos=none.long()), dict(slot=none, pos=none.long()), dict(slot=ints(1, 5))):
        with pytest.raises(ValueError):
            go(**bad)
    assert not calls
    for ok, n in ((dict(slot=some, pos=some), 5), (dict(slot=some), 5), (dict(pos=some), 5), (dict(slot=none, pos=none), 0),
                  (dict(pos=none), 0), (dict(), 0)):
        go(**ok)
        rows, _, slot, pos = calls.pop()
        assert rows == n and (slot is None) == (not n or "slot" not in ok) and (pos is None) == (not n or "pos" not in ok)


def test_references_round_as_the_type():
    x = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    assert torch.equal(R8.encode(R8.round_e4m3(x)), x.float().to(torch.float8_e4m3fn).view(torch.uint8))
    every = torch.arange(256, dtype=torch.uint8)
    y = every.view(torch.float8_e4m3fn).double()
    fine = ~torch.isnan(y)
    assert torch.equal(R8.round_e4m3(y[fine]), y[fine])


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (448.0001, 128), (224.0, 126), (1.0, 119), (0.0, 1), (1e-45, 1),
                                       (3.3895313892515355e38, 247), (1.75, 119), (1.7500001, 120)])
def test_references_scale(amax, byte):
    assert int(R8.block_byte(torch.tensor(amax, dtype=torch.float64))) == byte


def test_a_release_undoes_a_reserve_in_the_reference():
    table = [[3, 5, -1, -1], [7, -1, -1, -1], [-1, -1, -1, -1]]
    held, free, lens, rows, ps = [2, 1, 0], [9, 8, 6, 4, 2, 1, 0, -1, -1, -1], [30, 16, 0], [4, 17, 1], 16
    t, h, n, start, slot, pos, ok = R8.reserve(table, held, free, 7, lens, rows, ps, 25)
    assert h == [3, 3, 1] and n == 3 and ok == [1, 1, 1] and start == [0, 4, 21, 22]
    assert t[0][2] == 0 and t[1][1:3] == [1, 2] and t[2][0] == 4 and slot[2] == 0 and pos[22:] == [-1] * 3
    assert R8.release(t, h, free, n, lens, None, ps) == (table, held, free, 7)
