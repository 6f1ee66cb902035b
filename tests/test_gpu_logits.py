"""The logit rules and the lm_head's logits on the GPU.  The rules are a fixed
sequence of FP32 operations, so their values are compared bit for bit with the
same sequence in torch."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_ref as ref
import synthgen
from helpers import to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp32_default():
    """The files of a run share torch's default type."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(old)


@pytest.fixture(scope="module")
def M(cuda_ok):
    import moe_nvfp4_block_gb300 as M
    return M


def rules_for(R, V, seed, history=60, penalties=True, bias=True, mask=True):
    g = torch.Generator()
    g.manual_seed(seed)
    d = {}
    if penalties:
        d["tokens"] = torch.randint(-2, V + 2, (R * history + 5,), generator=g, dtype=torch.int32)
        hot = torch.randint(0, V, (7,), generator=g, dtype=torch.int32)
        pick = torch.rand(d["tokens"].shape, generator=g) < 0.4
        d["tokens"][pick] = hot[torch.randint(0, 7, (int(pick.sum()),), generator=g)]
        d["begin"] = torch.tensor([r * history - (3 if r == 0 else 0) for r in range(R)], dtype=torch.int32)
        d["end"] = torch.tensor([(r + 1) * history + (99 if r == R - 1 else 0) if r % 3 != 1 else r * history - 2
                                 for r in range(R)], dtype=torch.int32)
        d["repetition"] = 0.7 + torch.rand(R, generator=g)
        d["presence"] = torch.randn(R, generator=g)
        d["frequency"] = torch.randn(R, generator=g)
    if bias:
        d["bias"] = 3 * torch.randn(3, V, generator=g)
        d["bias"][0, ::5] = -math.inf
        d["bias_row"] = torch.tensor([(r + 1) % 5 - 1 if (r + 1) % 5 < 4 else -7 for r in range(R)], dtype=torch.int32)
    if mask:
        d["allow"] = torch.randint(-2**31, 2**31, (2, (V + 31) // 32), generator=g).to(torch.int32)
        d["allow_row"] = torch.tensor([r % 3 - 1 for r in range(R)], dtype=torch.int32)
    return d


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check(M, x, d, in_place=False, ws=None, out_stride=None):
    R, V = x.shape
    dev = M.LogitRules(**{k: v.cuda() for k, v in d.items()}) if d is not None else None
    xd = x.cuda()
    if x.stride(0) != V:
        wide = torch.zeros(R, x.stride(0), dtype=x.dtype, device="cuda")
        wide[:, :V] = xd
        xd = wide[:, :V]
    out = xd if in_place else torch.full((R, out_stride or V), 7.0, dtype=x.dtype, device="cuda")[:, :V]
    tok = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    best = torch.zeros(R, device="cuda")
    ws = ws if ws is not None else M.logits_workspace(R, V)
    M.moe_logits_constrain(xd, dev, ws, out=out, tok=tok, best=best)
    assert M.moe_workspace_error(ws) == 0
    want, wtok, wbest = ref.logits(x, **(d or {}))
    got = out.cpu()
    w = want.to(x.dtype)
    nan = torch.isnan(w)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(bits(got.contiguous())[~nan], bits(w.contiguous())[~nan])
    assert torch.equal(tok.cpu(), wtok)
    assert torch.equal(best.cpu(), wbest)
    return ws


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 1), (1, 2), (2, 7), (3, 31), (5, 33), (4, 1000), (7, 1025), (3, 8191), (2, 8200),
                                 (1, 151936), (9, 32003)])
def test_sizes(M, dtype, R, V):
    x = (3 * torch.randn(R, V, generator=torch.Generator().manual_seed(V))).to(dtype)
    check(M, x, rules_for(R, V, V + R))
    check(M, x, None)


@pytest.mark.parametrize("parts", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_each_rule_alone(M, parts):
    x = torch.randn(6, 5000, generator=torch.Generator().manual_seed(1))
    check(M, x, rules_for(6, 5000, 2, 300, *parts))


@pytest.mark.parametrize("missing", ["repetition", "presence", "frequency"])
def test_a_missing_penalty_is_neutral(M, missing):
    d = rules_for(4, 3001, 3, bias=False, mask=False)
    del d[missing]
    check(M, torch.randn(4, 3001, generator=torch.Generator().manual_seed(1)), d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,stride,out_stride", [(1003, 1003, 1003), (1003, 1024, 1003), (1003, 1005, 1040), (2048, 2051, None)])
def test_strides_and_in_place(M, dtype, V, stride, out_stride):
    x = torch.randn(5, stride, generator=torch.Generator().manual_seed(1)).to(dtype)[:, :V]
    d = rules_for(5, V, 4)
    check(M, x, d, out_stride=out_stride)
    check(M, x, d, in_place=True)


def test_ties_go_to_the_lowest_index(M):
    x = torch.zeros(4, 20000)
    x[1, 15000] = x[1, 3] = x[1, 19999] = 2.0
    x[2] = -math.inf
    x[3] = -math.inf
    x[3, 12345] = -3e38
    check(M, x, None)


def test_nan_and_infinite_logits(M):
    x = torch.randn(5, 3000, generator=torch.Generator().manual_seed(1))
    x[0, 5] = x[0, 2999] = math.nan
    x[1] = math.nan
    x[2, 70] = math.inf
    x[2, 100] = math.inf
    x[3] = -math.inf
    x[4, 7] = math.nan
    x[4, 8:] = -math.inf
    check(M, x, None)
    check(M, x, rules_for(5, 3000, 9, bias=False))


def test_a_mask_that_leaves_nothing(M):
    d = rules_for(3, 500, 5, bias=False)
    d["allow"].zero_()
    check(M, torch.randn(3, 500, generator=torch.Generator().manual_seed(1)), d)


def test_many_rows_and_one_workspace(M):
    big = M.logits_workspace(4096, 3000)
    for R, V in ((300, 777), (4096, 100), (3, 3000), (600, 41)):
        x = torch.randn(R, V, generator=torch.Generator().manual_seed(R))
        check(M, x, rules_for(R, V, R, history=11), ws=big)


def test_long_history_of_one_token(M):
    d = dict(tokens=torch.full((100000,), 17, dtype=torch.int32), begin=torch.tensor([0, 1], dtype=torch.int32),
             end=torch.tensor([100000, 70001], dtype=torch.int32), frequency=torch.tensor([1e-3, 2e-3]))
    check(M, torch.randn(2, 9000, generator=torch.Generator().manual_seed(1)), d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_repeated_tokens_than_a_list_holds(M, dtype):
    # every token of a row once and some thousands of them again, over long tiles (many rows)
    R, V = 700, 14001
    g = torch.Generator().manual_seed(3)
    tokens = torch.cat([torch.randperm(V, generator=g), torch.randint(0, 9000, (5000,), generator=g)]).int()
    begin = torch.tensor([(r * 37) % 3000 for r in range(R)], dtype=torch.int32)
    end = torch.tensor([len(tokens) - (r % 11) * 900 for r in range(R)], dtype=torch.int32)
    check(M, torch.randn(R, V, generator=g).to(dtype),
          dict(tokens=tokens, begin=begin, end=end, repetition=torch.full((R,), 1.25),
               frequency=torch.rand(R, generator=g)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_long_list_in_place(M, dtype):
    # the stretches of a tile one after another, each over what it read
    R, V = 700, 14001
    g = torch.Generator().manual_seed(4)
    d = rules_for(R, V, 5, history=1)
    d["tokens"] = torch.cat([torch.randperm(V, generator=g), torch.randint(0, 9000, (5000,), generator=g)]).int()
    d["begin"] = torch.tensor([(r * 41) % 3000 for r in range(R)], dtype=torch.int32)
    d["end"] = torch.tensor([len(d["tokens"]) - (r % 7) * 900 for r in range(R)], dtype=torch.int32)
    check(M, torch.randn(R, V, generator=g).to(dtype), d, in_place=True)


def test_whole_rows_of_a_large_vocabulary(M):
    # as many rows as SMs and more: a CTA takes up to 131,072 tokens
    R, V = 256, 128003
    g = torch.Generator().manual_seed(6)
    d = rules_for(R, V, 7, history=40)
    d["end"][::5] = d["begin"][::5].clamp(min=0) + 9000
    check(M, torch.randn(R, V, generator=g).bfloat16(), d)
    check(M, torch.randn(R, V, generator=g).bfloat16(), d, in_place=True)


def test_an_empty_history(M):
    x = torch.randn(3, 900, generator=torch.Generator().manual_seed(1))
    e = torch.zeros(0, dtype=torch.int32)
    check(M, x, dict(tokens=e, begin=torch.zeros(3, dtype=torch.int32), end=torch.ones(3, dtype=torch.int32),
                     repetition=torch.full((3,), 2.0)))


def test_two_streams_at_once(M):
    xs = [torch.randn(40, 30011, device="cuda") for _ in range(2)]
    d = [rules_for(40, 30011, s) for s in (1, 2)]
    rules = [M.LogitRules(**{k: v.cuda() for k, v in q.items()}) for q in d]
    ws, outs = [M.logits_workspace(40, 30011) for _ in xs], [torch.empty_like(x) for x in xs]
    toks = [torch.empty(40, dtype=torch.int32, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            M.moe_logits_constrain(xs[i], rules[i], ws[i], out=outs[i], tok=toks[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        want, wtok, _ = ref.logits(xs[i].cpu(), **d[i])
        assert torch.equal(outs[i].cpu(), want) and torch.equal(toks[i].cpu(), wtok)


def test_rows_past_the_tables_are_recorded(M):
    R, V = 3, 900
    x = torch.randn(R, V, generator=torch.Generator().manual_seed(1))
    for name, n in (("bias", 2), ("allow", 1)):
        d = rules_for(R, V, 5, penalties=False, bias=name == "bias", mask=name == "allow")
        d[name] = d[name][:n].contiguous()
        d[name + "_row"] = torch.tensor([0, n, 2**31 - 1], dtype=torch.int32)
        ws = M.logits_workspace(R, V)
        out = torch.empty(R, V, device="cuda")
        M.moe_logits_constrain(x.cuda(), M.LogitRules(**{k: v.cuda() for k, v in d.items()}), ws, out=out)
        assert M.moe_workspace_error(ws) == M.MOE_ERR_INVALID_ARG
        assert torch.equal(out.cpu(), ref.logits(x, **d)[0])


def test_argmax_or_logits_alone(M):
    x = torch.randn(3, 4001, generator=torch.Generator().manual_seed(1))
    d = rules_for(3, 4001, 6)
    dev = M.LogitRules(**{k: v.cuda() for k, v in d.items()})
    want, wtok, wbest = ref.logits(x, **d)
    ws = M.logits_workspace(3, 4001)
    out, tok, best = torch.empty(3, 4001, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda")
    M.moe_logits_constrain(x.cuda(), dev, ws, out=out)
    assert torch.equal(out.cpu(), want)
    M.moe_logits_constrain(x.cuda(), dev, ws, tok=tok)
    assert torch.equal(tok.cpu(), wtok)
    M.moe_logits_constrain(x.cuda(), dev, ws, best=best)
    assert torch.equal(best.cpu(), wbest)


def test_graph_replay(M):
    x = torch.randn(2, 5000, device="cuda")
    ws = M.logits_workspace(2, 5000)
    tok = torch.empty(2, dtype=torch.int32, device="cuda")
    M.moe_logits_constrain(x, None, ws, tok=tok)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_logits_constrain(x, None, ws, tok=tok)
    for i in range(3):
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok.long(), x.argmax(1))


@pytest.mark.parametrize("K,H,V", [(1, 256, 300), (3, 512, 1001), (4, 2048, 5003), (8, 2048, 2500), (16, 2048, 1700),
                                   (16, 256, 40), (5, 1024, 1)])
def test_lm_head_logits(M, K, H, V):
    x = synthgen.normal_bf16(K, 0, synthgen.T_X, 0, K * H, 0.0, 1.0).reshape(K, H)
    W = synthgen.normal_bf16(K, 0, synthgen.T_LM_HEAD, 0, V * H, 0.0, 0.02).reshape(V, H)
    xd, Wd = to_dev_bf16(x), to_dev_bf16(W)
    logits = torch.full((K + 1, V), 7.0, device="cuda")
    ws = M.lm_head_workspace(K)
    tok, best = torch.empty(K, dtype=torch.int32, device="cuda"), torch.empty(K, device="cuda")
    for _ in range(2):
        M.moe_lm_head_logits(xd, Wd, logits[:K], ws)
        M.moe_lm_head_argmax(xd, Wd, tok, ws, best_logit=best)
    assert M.moe_workspace_error(ws) == 0
    want = xd.double() @ Wd.double().T
    # H products added in FP32, at most H / 32 of them one after another and five joins
    room = (H / 32 + 6) * 2.0 ** -24 * (xd.double().abs() @ Wd.double().abs().T)
    assert bool(((logits[:K].double() - want).abs() <= room).all())
    assert bool((logits[K] == 7).all())
    # the argmax's own values: same bits, same token
    assert torch.equal(logits[:K].amax(1), best)
    first = torch.where(logits[:K] == best[:, None], torch.arange(V, device="cuda"), V).amin(1)
    assert torch.equal(first.int(), tok)


@pytest.mark.parametrize("K", [2, 5, 7, 9, 12, 13])
def test_lm_head_logits_of_any_row_count(M, K):
    # the bits are a row's own, whatever rows are beside it
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(16, 768, generator=g, device="cuda").bfloat16()
    W = torch.randn(1303, 768, generator=g, device="cuda").bfloat16()
    ws = torch.zeros(M.lib.moe_lm_head_workspace_size(16), dtype=torch.uint8, device="cuda")
    all_, some = torch.empty(16, 1303, device="cuda"), torch.empty(K, 1303, device="cuda")
    M.moe_lm_head_logits(x, W, all_, ws)
    M.moe_lm_head_logits(x[:K], W, some, ws)
    assert torch.equal(some, all_[:K])
    want = x.double() @ W.double().T
    bound = 768 * 2.0 ** -24 * (x.double().abs() @ W.double().abs().T)  # a rounding a term
    assert bool(((all_.double() - want).abs() <= bound).all())


def test_lm_head_logits_wait_limit(M):
    K, H, V = 4, 2048, 4096
    x = torch.randn(K, H, device="cuda").bfloat16()
    W = torch.randn(V, H, device="cuda").bfloat16()
    logits, ws = torch.empty(K, V, device="cuda"), M.lm_head_workspace(K)
    try:
        M.moe_debug_set_wait_limit_ns(0)
        M.moe_lm_head_logits(x, W, logits, ws)
        torch.cuda.synchronize()
    finally:
        M.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_DEVICE_TIMEOUT
    M.moe_lm_head_logits(x, W, logits, ws)
    assert M.moe_workspace_error(ws) == 0
    want = x.double() @ W.double().T
    assert bool(((logits.double() - want).abs() <= (H / 32 + 6) * 2.0 ** -24 * (x.double().abs() @ W.double().abs().T)).all())
