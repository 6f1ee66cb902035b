"""The serving operators on the host (no GPU needed): workspace sizes and the
arguments they refuse before anything is enqueued."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4


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
    return M


def kv(M, **kw):
    d = dict(kpages=16, vpages=16, table=16, kv_len=16, n_pages=10, page_size=64, nkv=8, head_dim=128, n_seqs=3,
             max_pages=4)
    d.update(kw)
    return M.moe_paged_kv(**d)


BAD_CACHES = [(dict(kpages=None), INVALID), (dict(vpages=None), INVALID), (dict(table=None), INVALID),
              (dict(kv_len=None), INVALID), (dict(n_pages=0), INVALID), (dict(nkv=0), INVALID),
              (dict(n_seqs=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_seqs=1025), SHAPE),
              (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=256), SHAPE),
              (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE), (dict(head_dim=64), SHAPE),
              (dict(n_pages=1 << 22, page_size=64), SHAPE), (dict(max_pages=1 << 25), SHAPE),
              (dict(kpages=8), ALIGN), (dict(vpages=24), ALIGN), (dict(table=18), ALIGN), (dict(kv_len=17), ALIGN)]


def append(M, c=None, q=16, qs=1024, k=16, ks=1024, v=16, vs=1024, n=5, nq=8, start=16, pos=None, qo=16, qos=1024,
           ws=16, wsb=256):
    c = c if c is not None else kv(M)
    return M.lib.moe_paged_kv_append(ctypes.byref(c), q, qs, k, ks, v, vs, n, nq, start,
                                     None if pos is None else ctypes.byref(pos), qo, qos, ws, wsb, None)


def attention(M, c=None, q=16, qs=4096, n=5, max_rows=2, nq=32, start=16, sc=None, o=16, os_=4096, lse=None, ws=16,
              wsb=1 << 30):
    c = c if c is not None else kv(M)
    return M.lib.moe_paged_attention(ctypes.byref(c), q, qs, n, max_rows, nq, start,
                                     None if sc is None else ctypes.byref(sc), o, os_, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(M, kw, status):
    assert append(M, kv(M, **kw)) == status
    if kw != dict(nkv=0):
        assert attention(M, kv(M, **kw)) == status
    else:
        assert attention(M, kv(M, **kw)) != OK


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(start=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(n=-1), INVALID), (dict(nq=0), INVALID),
    (dict(ks=1000), INVALID), (dict(qs=512), INVALID), (dict(ks=1028), ALIGN), (dict(k=20), ALIGN),
    (dict(q=8), ALIGN), (dict(qo=18), ALIGN), (dict(start=18), ALIGN), (dict(ws=8), ALIGN), (dict(wsb=255), WORKSPACE),
    (dict(qos=2048), INVALID)])
def test_append_refusals(M, kw, status):
    assert append(M, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(rotary_dim=129), SHAPE), (dict(rotary_dim=7), SHAPE),
                                       (dict(rotary_dim=-2), SHAPE), (dict(rotary_dim=64, rope_theta=1.0), INVALID),
                                       (dict(rotary_dim=64, yarn_factor=4.0, yarn_orig_ctx=0), INVALID)])
def test_append_refuses_bad_rotary(M, kw, status):
    assert append(M, pos=M.attn_pos(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(start=None), INVALID), (dict(ws=None), INVALID),
    (dict(n=-1), INVALID), (dict(nq=0), INVALID), (dict(nq=12), SHAPE), (dict(max_rows=0), INVALID),
    (dict(max_rows=17), SHAPE), (dict(max_rows=9, nq=64), SHAPE), (dict(qs=4088), INVALID), (dict(os_=4100), ALIGN),
    (dict(q=24), ALIGN), (dict(o=8), ALIGN), (dict(lse=18), ALIGN), (dict(wsb=1000), WORKSPACE)])
def test_attention_refusals(M, kw, status):
    assert attention(M, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(softcap=-2.0), INVALID), (dict(softcap=float("nan")), INVALID),
    (dict(softcap=float("inf")), INVALID), (dict(slopes=18), ALIGN), (dict(first=18), ALIGN), (dict(prefix=18), ALIGN)])
def test_attention_refuses_bad_scores(M, kw, status):
    assert attention(M, sc=M.moe_paged_scores(**kw)) == status


@pytest.mark.parametrize("what", ["scale", "softcap"])
def test_attention_scores_may_be_large_but_not_out_of_range(M, what):
    # no rows: nothing is enqueued for what passes
    assert attention(M, n=0, sc=M.moe_paged_scores(**{what: 2.0 ** 126})) == OK
    assert attention(M, n=0, sc=M.moe_paged_scores(**{what: 1e-45})) == OK
    assert attention(M, n=0, sc=M.moe_paged_scores(**{what: 1.0001 * 2.0 ** 126})) == INVALID


def test_no_rows_is_no_work(M):
    assert append(M, n=0) == OK and attention(M, n=0) == OK


def test_no_rows_need_no_matrices(M):
    # an empty tensor has no address
    assert append(M, n=0, q=None, qo=None, k=None, v=None) == OK and attention(M, n=0, q=None, o=None) == OK


def test_output_over_the_queries_wants_their_stride(M):
    assert attention(M, q=16, o=16, os_=4104) == INVALID


def test_binding_refuses_rules_it_would_misread(M):
    with pytest.raises(ValueError):
        M.LogitRules(bias=torch.zeros(50), bias_row=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        M.LogitRules(allow=torch.zeros(2, dtype=torch.int32), allow_row=torch.zeros(3, dtype=torch.int32))
    empty, row = torch.zeros(0, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    c = M.LogitRules(tokens=empty, begin=row, end=row, repetition=torch.ones(3)).c
    assert c.tokens is None and c.begin is None and c.end is None


def test_binding_refuses_tensors_of_the_wrong_place(M):
    bf, i32 = torch.bfloat16, torch.int32
    k, table, n = torch.zeros(6, 2, 16, 128, dtype=bf), torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    c, rows, start, ws = M.PagedKV(k, k.clone(), table, n), torch.zeros(5, 256, dtype=bf), torch.zeros(4, dtype=i32), \
        torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        M.moe_paged_kv_append(c, rows, rows, start, ws)
    with pytest.raises(ValueError):
        M.moe_paged_attention(c, rows, start, rows, ws, 2)
    w = torch.zeros(30, 256, dtype=bf)
    for bad in (dict(logits=torch.zeros(5, 30, dtype=bf)), dict(logits=torch.zeros(4, 30)), dict(W=w.float()),
                dict(W=w[:, :128]), dict(x_norm=rows.float()), dict(logits=torch.zeros(30, 5).T)):
        with pytest.raises(ValueError):
            M.moe_lm_head_logits(**(dict(x_norm=rows, W=w, logits=torch.zeros(5, 30), ws=ws) | bad))


def test_paged_workspace_sizes(M):
    f = M.lib.moe_paged_workspace_size
    assert f(0, 32, 8) == 0 and f(17, 8, 8) == 0 and f(2, 12, 8) == 0 and f(16, 64, 8) == 0 and f(1, 8, 0) == 0
    sizes = [f(r, 32, 8) for r in (1, 4, 5, 8, 9, 16)]
    assert sizes[0] > 0 and sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)


def constrain(M, x=16, type_=0, s=100, R=3, V=100, rules=None, out=16, os_=100, tok=16, best=16, ws=16, wsb=1 << 30):
    return M.lib.moe_logits_constrain(x, type_, s, R, V, None if rules is None else ctypes.byref(rules), out, os_, tok,
                                      best, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(ws=None), INVALID), (dict(out=None, tok=None, best=None), INVALID),
    (dict(type_=2), INVALID), (dict(type_=-1), INVALID), (dict(R=0), INVALID), (dict(V=0), INVALID),
    (dict(R=4097), SHAPE), (dict(V=(1 << 24) + 1, s=1 << 25, os_=1 << 25), SHAPE), (dict(s=99), INVALID),
    (dict(os_=99), INVALID), (dict(os_=128), INVALID), (dict(x=24), ALIGN), (dict(out=20), ALIGN), (dict(tok=17), ALIGN),
    (dict(best=18), ALIGN), (dict(ws=8), ALIGN), (dict(wsb=100), WORKSPACE)])
def test_logits_refusals(M, kw, status):
    assert constrain(M, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=16), INVALID), (dict(tokens=16, begin=16), INVALID), (dict(begin=16), INVALID),
    (dict(tokens=16, begin=16, end=16, n_tokens=-1), INVALID), (dict(bias=16, n_bias=1), INVALID),
    (dict(bias=16, bias_row=16), INVALID), (dict(allow=16, n_allow=1), INVALID), (dict(allow=16, allow_row=16), INVALID),
    (dict(repetition=17), ALIGN), (dict(bias=17, bias_row=16, n_bias=1), ALIGN)])
def test_logits_refuse_bad_rules(M, kw, status):
    assert constrain(M, rules=M.moe_logit_rules(**kw)) == status


def test_lm_head_logits_refusals(M):
    f = M.lib.moe_lm_head_logits
    n = M.lib.moe_lm_head_workspace_size(4)
    assert f(16, 4, 2048, 16, 1000, None, 16, n, None) == INVALID
    assert f(16, 4, 2048, 16, 1000, 24, 16, n, None) == ALIGN
    assert f(16, 17, 2048, 16, 1000, 16, 16, n, None) == INVALID
    assert f(16, 4, 4096, 16, 1000, 16, 16, n, None) == SHAPE
    assert f(16, 4, 2048, 16, 1000, 16, 16, n - 1, None) == WORKSPACE
    # the argmax still wants its tokens
    assert M.lib.moe_lm_head_argmax(16, 4, 2048, 16, 1000, None, None, 16, n, None) == INVALID


def test_binding_refuses_tensors_it_would_misread(M):
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(6, 2, 16, 128, dtype=bf)
    table, n = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    c = M.PagedKV(k, k.clone(), table, n)
    with pytest.raises(ValueError):
        M.PagedKV(k, k[:5], table, n)
    with pytest.raises(ValueError):
        M.PagedKV(k.float(), k, table, n)
    with pytest.raises(ValueError):
        M.PagedKV(k, k, table.long(), n)
    with pytest.raises(ValueError):
        M.PagedKV(k, k, table, n[:2])
    with pytest.raises(ValueError):
        M.PagedKV(k.transpose(1, 2), k.transpose(1, 2), table, n)
    start, ws = torch.zeros(4, dtype=i32), torch.zeros(256, dtype=torch.uint8)
    rows = torch.zeros(5, 256, dtype=bf)
    for bad in (dict(k_new=rows.float()), dict(k_new=rows[:, :128]), dict(v_new=rows[:4]), dict(row_start=start[:3]),
                dict(row_start=start.long()), dict(q=rows), dict(q=rows[:, :200], q_out=rows[:, :200]),
                dict(k_new=torch.zeros(256, 5, dtype=bf).T)):
        args = dict(k_new=rows, v_new=rows, row_start=start, ws=ws) | bad
        with pytest.raises(ValueError):
            M.moe_paged_kv_append(c, **args)
    for bad in (dict(q=rows.half()), dict(o=rows[:, :128]), dict(lse=torch.zeros(5, 3)),
                dict(scores=M.PagedScores(slopes=torch.zeros(3))), dict(scores=M.PagedScores(first=n[:2]))):
        args = dict(q=rows, row_start=start, o=rows, ws=ws, max_rows=2) | bad
        with pytest.raises(ValueError):
            M.moe_paged_attention(c, **args)
    with pytest.raises(ValueError):
        M.LogitRules(repetition=torch.ones(3), presence=torch.ones(4))
    with pytest.raises(ValueError):
        M.LogitRules(tokens=torch.zeros(3))
