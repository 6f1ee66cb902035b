"""The paged append and attention on the GPU against their 64-bit definition:
lengths around every tile and page edge, empty rows and sequences, score
forms, strides, hidden NaNs, bad pages, graphs, streams and workspaces."""
import math

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu
HD = 128


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


def queries(t, nq, seed, strided=False, scale=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (scale * torch.randn(t, (nq + 3 if strided else nq) * HD, generator=g, device="cuda")).bfloat16()
    return q[:, HD:(nq + 1) * HD] if strided else q


def run(M, k, v, table, n, start, q, nq, max_rows, strided=False, ws=None, stream=None, **kw):
    kv = M.PagedKV(k, v, table, n)
    t = q.shape[0]
    o = torch.full((t, (nq + 2 if strided else nq) * HD), 7.0, dtype=torch.bfloat16, device="cuda")
    o = o[:, HD:(nq + 1) * HD] if strided else o
    lse = torch.full((t, nq), 7.0, device="cuda")
    ws = ws if ws is not None else M.paged_workspace(kv, max_rows, nq)
    M.moe_paged_attention(kv, q, start, o, ws, max_rows, scores=M.PagedScores(**kw) if kw else None, lse=lse,
                          stream=stream)
    return o, lse, ws


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(M, lens, rows, nq, nkv, ps, seed=0, max_rows=None, strided=False, fill=float("nan"), first=None, prefix=None,
          **kw):
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, ps, seed, fill=fill)
    q = queries(sum(rows), nq, seed + 1, strided)
    dev = dict(kw)
    if first:
        dev["first"] = ints(first)
    if prefix:
        dev["prefix"] = ints(prefix)
    o, lse, ws = run(M, k, v, table, n, start, q, nq, max_rows or max(rows), strided, **dev)
    assert M.moe_workspace_error(ws) == 0
    want = ref.attention(q, k, v, table, lens, rows, nq, first=first, prefix=prefix, **kw)
    ref.check_attention(o, lse, want, f"lens {lens} rows {rows} heads {nq}/{nkv} page {ps} {kw}")


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, [1] * 9), (4, 4, [3, 1, 2, 0, 4, 1, 1, 2, 3]), (16, 2, [4] * 9),
                                         (8, 1, [8, 1, 5, 0, 7, 2, 8, 3, 6]), (16, 4, [16] * 9)])
def test_lengths_around_tiles_and_pages(M, nq, nkv, rows, ps):
    check(M, [0, 1, 15, 16, 47, 63, 64, 130, 255], rows, nq, nkv, ps, seed=ps + nq)


def test_one_token_of_an_empty_cache(M):
    check(M, [0], [1], 2, 1, 16)


@pytest.mark.parametrize("lens,rows", [([5000], [1]), ([3000, 1, 20000], [4, 4, 2]), ([100] * 40, [2] * 40),
                                       ([9000, 0, 0, 700], [0, 16, 0, 16])])
def test_long_and_unequal_lengths(M, lens, rows):
    check(M, lens, rows, 8, 2, 64, seed=3)


@pytest.mark.parametrize("kw", [dict(), dict(window=2000, prefix=[0, 7, 3000]), dict(softcap=20.0, first=[4000, 1, 0])])
@pytest.mark.parametrize("rows,nq,nkv", [([8, 5, 7], 8, 2), ([16, 11, 1], 4, 2), ([5, 6, 4], 10, 2)])
def test_middling_rows_over_long_tables(M, rows, nq, nkv, kw):
    # 17 to 32 query rows a KV head where the tables have room for long sequences
    check(M, [26000, 3, 9000], rows, nq, nkv, 64, seed=8, **kw)


def test_middling_rows_with_distance_bias(M):
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda").float()
    check(M, [26000, 20, 300], [8, 5, 7], 8, 2, 32, seed=9, slopes=slopes)


@pytest.mark.parametrize("kw", [
    dict(window=1), dict(window=5), dict(window=64), dict(window=200), dict(window=10**6), dict(softcap=5.0),
    dict(softcap=30.0, window=33), dict(scale=0.02), dict(window=17, prefix=[0, 3, 100, 17, 2000]),
    dict(first=[0, 70, 5, 64, 1000]), dict(first=[3, 2, 129, 0, 900], window=40, prefix=[10, 1, 140, 9, 901])])
@pytest.mark.parametrize("rows,nq,nkv", [([2, 1, 4, 3, 4], 8, 2), ([1] * 5, 4, 4), ([8, 7, 3, 8, 1], 8, 1)])
def test_score_forms(M, kw, rows, nq, nkv):
    check(M, [3, 77, 200, 64, 1100], rows, nq, nkv, 32, seed=5, **kw)


FORMS = [([4, 3], 8, 2), ([8, 5], 8, 2), ([16, 11], 8, 2)]  # up to 16, 32 and 64 query rows a KV head


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1.0, 9.0, 100.0, 1e3, 1e4, 1e6, 1e9, 1e20, 2.0 ** 126])
def test_softcaps_of_any_size(M, cap, rows, nq, nkv):
    # the cap's error is to the score, not to the cap: the room is that of the uncapped scores
    # (|d tanh| <= |d z|, and tanh's own 6e-7 of the score is below the 2^-20 of it there)
    lens = [200, 90]
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1, fill=float("nan"))
    q = queries(sum(rows), nq, 2)
    o, lse, _ = run(M, k, v, table, n, start, q, nq, max(rows), softcap=cap)
    want = ref.attention(q, k, v, table, lens, rows, nq, softcap=cap)
    bound = ref.attention(q, k, v, table, lens, rows, nq)[2]
    ref.check_attention(o, lse, (want[0], want[1], bound), f"softcap {cap}")


@pytest.mark.parametrize("kw", [dict(scale=2.0 ** 120, softcap=20.0), dict(scale=2.0 ** -120, softcap=2.0 ** 60),
                                dict(scale=2.0 ** -100, softcap=2.0 ** 100)])
def test_softcaps_far_from_the_scale(M, kw):
    # scores at the cap's two ends (or zero), or all but equal
    for rows, nq, nkv in FORMS:
        lens = [200, 90]
        k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1)
        q = queries(sum(rows), nq, 2)
        q[0] = 0
        o, lse, _ = run(M, k, v, table, n, start, q, nq, max(rows), **kw)
        want = ref.attention(q, k, v, table, lens, rows, nq, **kw)
        bound = 2.0 ** -20 * (1 + 20 + want[1].abs())  # scores of at most 20 and their sums
        ref.check_attention(o, lse, (want[0], want[1], bound), f"{kw}")


@pytest.mark.parametrize("rows", [[2, 1, 3], [1, 1, 1]])
def test_distance_bias(M, rows):
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda").float()
    check(M, [500, 20, 3000], rows, 8, 4, 16, seed=6, slopes=slopes)
    check(M, [500, 20, 3000], rows, 8, 4, 16, seed=6, slopes=-slopes / 64, softcap=20.0, window=300)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(window=300), dict(softcap=20.0, window=70, prefix=[5, 0, 40])])
def test_distance_bias_of_many_rows(M, kw):
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda").float()
    check(M, [500, 20, 3000], [16, 9, 12], 8, 2, 32, seed=6, slopes=slopes, **kw)
    check(M, [500, 20, 3000], [16, 9, 12], 8, 2, 32, seed=7, slopes=-slopes / 64, **kw)


@pytest.mark.parametrize("group,rows", [(3, [16, 11, 5]), (5, [12, 7, 1]), (7, [9, 8, 2]), (7, [5, 6, 7]), (9, [7, 3, 4]),
                                        (11, [5, 4, 3]), (13, [4, 3, 1]), (64, [1, 1, 1]), (21, [3, 2, 1]), (3, [10, 9, 6]),
                                        (7, [4, 3, 1]), (5, [3, 1, 2]), (17, [1, 1, 1]), (33, [1, 1, 1])])
def test_odd_head_groups(M, group, rows):
    for lens in ([700, 3, 64], [26000, 100, 0]):  # short and long tables
        check(M, lens, rows, 2 * group, 2, 32, seed=group, window=0)
    check(M, [300, 90, 8], rows, 3 * group, 3, 16, seed=group, window=65, prefix=[3, 70, 0], softcap=25.0)


def test_rows_that_see_nothing(M):
    # first past the rows' positions: o = 0, lse = -inf; some rows of a sequence only
    check(M, [10, 40, 5, 300], [3, 2, 4, 1], 8, 2, 16, first=[11, 1000, 7, 2**31 - 1])


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
@pytest.mark.parametrize("kw", [dict(), dict(window=30), dict(window=7, prefix=[9, 200])])
def test_rows_that_see_nothing_need_no_pages(M, rows, nq, nkv, kw):
    lens = [10, 40]
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1)
    table.fill_(-1)
    q, dev = queries(sum(rows), nq, 2), {x: ints(y) if x == "prefix" else y for x, y in kw.items()}
    for first in ([1000, 2**31 - 1], [lens[0] + rows[0], lens[1] + rows[1]]):
        o, lse, ws = run(M, k, v, table, n, start, q, nq, max(rows), first=ints(first), **dev)
        assert M.moe_workspace_error(ws) == 0
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
def test_limits_at_the_ends_of_their_type(M, rows, nq, nkv):
    # below zero: as zero; past the rows: as far as there are positions
    lens, low, high = [200, 90], -2**31, 2**31 - 1
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1, fill=float("nan"))
    q = queries(sum(rows), nq, 2)
    for window, prefix, first, wp, wf in ((20, [low, low + 3], [low, -1], [0, 0], [0, 0]),
                                          (20, [high, -1], [70, low], [10**6, 0], [70, 0]),
                                          (high, [high, low], [0, 1], [0, 0], [0, 1])):
        o, lse, ws = run(M, k, v, table, n, start, q, nq, max(rows), window=window, prefix=ints(prefix), first=ints(first))
        assert M.moe_workspace_error(ws) == 0
        ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, nq, window=window, prefix=wp, first=wf))


def test_strided_rows(M):
    check(M, [33, 129], [4, 3], 8, 2, 64, strided=True)


@pytest.mark.parametrize("fill", [0.0, float("inf"), float("-inf"), 3e38])
def test_hidden_slots_hold_anything(M, fill):
    check(M, [17, 90, 64], [2, 5, 1], 4, 2, 32, fill=fill, window=30)


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(window=170, prefix=[50, 60]), dict(first=[19, 20])])
@pytest.mark.parametrize("lens", [[200, 90], [20000, 90], [0, 17]])
def test_visible_infinite_values_are_what_the_formula_gives(M, rows, nq, nkv, equal, kw, lens):
    # infinite, opposite and NaN values, seen by every row or by some; with equal scores the weights are exact in bf16
    inf = math.inf
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1, fill=float("nan"))
    if equal:
        k.zero_()
    for b in range(2):
        def put(p, dim, x):
            if p < lens[b] + rows[b]:
                v[table[b, p // 16].long(), :, p % 16, dim] = x
        for p, dim, x in ((20, 3, inf), (40, 4, -inf), (20, 5, inf), (70, 5, -inf), (33, 6, math.nan), (3, 10, inf),
                          (lens[b], 11, -inf), (lens[b] + 2, 12, inf), (lens[b] - 100, 13, inf)):
            put(max(p, 0), dim, x)
        for p in range(16, 32):
            put(p, 8, inf)
            put(p, 9, -inf)
    q, dev = queries(sum(rows), nq, 2), {x: ints(y) if x != "window" else y for x, y in kw.items()}
    o, lse, _ = run(M, k, v, table, n, start, q, nq, max(rows), **dev)
    ro, rl, _ = ref.attention(q, k, v, table, lens, rows, nq, **kw)
    got = o.double().reshape(ro.shape)
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got), kind(ro)), kind.__name__
    fine = torch.isfinite(ro)
    assert bool(((got - ro)[fine].abs() <= 2.0 ** -8 * ro[fine].abs() + 2.0 ** -11 * 4).all())


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
@pytest.mark.parametrize("seqs", [2, 200])
@pytest.mark.parametrize("gain", [2.0, 5.0, 60.0])
def test_weights_do_not_take_values_out_of_range(M, rows, nq, nkv, seqs, gain):
    # a position in the middle outweighs those before by e^gain; its value times that passes FP32's
    # range, the row's output does not
    lens, rows = [700] * seqs, [rows[i % 2] for i in range(seqs)]
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 64, 1)
    k.zero_()
    v.zero_()
    big = min(3e38 / math.exp(gain) * 3, 1e38)
    for b in range(seqs):
        k[table[b, 400 // 64].long(), :, 400 % 64, 0] = 1
        v[table[b, 400 // 64].long(), :, 400 % 64] = big
    q = torch.zeros(sum(rows), nq * HD, device="cuda")
    q[:, ::HD] = gain * HD ** 0.5
    q = q.bfloat16()
    o, lse, _ = run(M, k, v, table, n, start, q, nq, max(rows))
    ro, rl, bound = ref.attention(q[:sum(rows[:2])], k, v, table, lens[:2], rows[:2], nq)
    t = sum(rows[:2])
    ref.check_attention((o[:t].double() / big), lse[:t], (ro / big, rl, bound))
    assert bool(torch.isfinite(o).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 20])
def test_a_rows_own_bad_value_stays_its_own(M, bad, window):
    # position 100 + 2 (row 2's own) holds a bad value, hidden from rows 0 and 1; with the
    # window position 85 too is hidden from rows 5 on
    lens, rows, nq, nkv = [100], [8], 8, 1
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 16, 1, fill=float("nan"))
    for p in (102, 85) if window else (102,):
        v[table[0, p // 16].long(), 0, p % 16, 5:9] = bad
    q = queries(8, nq, 2)
    o, lse, _ = run(M, k, v, table, n, start, q, nq, 8, window=window)
    ro, rl, _ = ref.attention(q, k, v, table, lens, rows, nq, window=window)
    got = o.double().reshape(ro.shape)
    fine = torch.isfinite(ro)
    assert bool((torch.isfinite(got) == fine).all())
    assert bool(fine[:2].all()) if not window else bool(fine[6:, :, :5].all())
    d = (got - ro)[fine].abs()
    assert bool((d <= 2.0 ** -8 * ro[fine].abs() + 2.0 ** -11 * 4).all())
    assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("nq", [1, 2, 4, 8])
def test_a_bad_value_of_some_rows_in_every_form(M, bad, window, nq):
    # as above for 8 to 64 query rows, and inf and NaN told apart
    lens, rows = [100], [8]
    k, v, table, n, start = ref.make_cache(lens, rows, 1, 16, 1, fill=float("nan"))
    for p in (102, 85) if window else (102,):
        v[table[0, p // 16].long(), 0, p % 16, 5:9] = bad
    q = queries(8, nq, 2)
    o, lse, _ = run(M, k, v, table, n, start, q, nq, 8, window=window)
    ro, rl, bound = ref.attention(q, k, v, table, lens, rows, nq, window=window)
    got = o.double().reshape(ro.shape)
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got), kind(ro))
    fine = torch.isfinite(ro)
    assert bool(((got - ro)[fine].abs() <= 2.0 ** -8 * ro[fine].abs() + 2.0 ** -11 * 4).all())
    assert bool(((lse.double() - rl).abs() <= bound).all())


def test_keys_of_infinite_score(M):
    # a visible score of -inf counts for nothing; all of them: an empty row
    k, v, table, n, start = ref.make_cache([2], [1], 1, 16, 1)
    page = table[0, 0].long()
    k[page, 0, :2] = 0
    k[page, 0, :2, 0] = float("-inf")
    q = torch.ones(1, HD, dtype=torch.bfloat16, device="cuda")
    o, lse, _ = run(M, k, v, table, n, start, q, 1, 1)
    assert torch.equal(o[0], v[page, 0, 2])
    k[page, 0, 2] = k[page, 0, 1]
    o, lse, _ = run(M, k, v, table, n, start, q, 1, 1)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_rows_of_no_sequence_are_left_alone(M):
    k, v, table, n, start = ref.make_cache([40, 9], [2, 1], 2, 16, 0)
    q = queries(8, 4, 1)
    o, lse, ws = run(M, k, v, table, n, start + 2, q, 4, 2)
    want = ref.attention(q[2:5], k, v, table, [40, 9], [2, 1], 4)
    ref.check_attention(o[2:5], lse[2:5], want)
    for x in (o, lse):
        assert bool((x[:2] == 7).all()) and bool((x[5:] == 7).all())
    assert M.moe_workspace_error(ws) == 0


def test_shared_prompt_pages(M):
    k, v, table, n, start = ref.make_cache([64, 70], [1, 1], 2, 32, 0)
    table[1, :2] = table[0, :2]
    q = queries(2, 4, 1)
    o, lse, _ = run(M, k, v, table, n, start, q, 4, 1)
    ref.check_attention(o, lse, ref.attention(q, k, v, table, [64, 70], [1, 1], 4))


def test_wrong_sequences_are_skipped_and_recorded(M):
    lens, rows = [40, 30, 20], [1, 2, 1]
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 16, 0, spare=0)
    q = queries(4, 4, 1)
    want = ref.attention(q, k, v, table, lens, rows, 4)
    for what, code in (("negative", M.MOE_ERR_INVALID_ARG), ("long", M.MOE_ERR_CAPACITY), ("huge", M.MOE_ERR_CAPACITY),
                       ("rows", M.MOE_ERR_INVALID_ARG), ("outside", M.MOE_ERR_INVALID_ARG)):
        m, s, mr = n.clone(), start.clone(), 2
        if what == "rows":
            mr = 1
        elif what == "outside":
            s[1] = -1
        else:
            m[1] = {"negative": -1, "long": 16 * table.shape[1] - 1, "huge": 2**31 - 1}[what]
        o, lse, ws = run(M, k, v, table, m, s, q, 4, mr)
        assert M.moe_workspace_error(ws) == code, what
        assert M.moe_workspace_error(ws) == 0
        skipped = slice(1, 3)
        if what != "outside":
            assert bool((o[skipped] == 7).all()) and bool((lse[skipped] == 7).all())
            ref.check_attention(o[:1], lse[:1], [x[:1] for x in want])
        ref.check_attention(o[3:], lse[3:], [x[3:] for x in want])
        o, lse, _ = run(M, k, v, table, n, start, q, 4, 2, ws=ws)  # the workspace stays usable
        ref.check_attention(o, lse, want)


@pytest.mark.parametrize("page", [-1, 10**6, 2**31 - 1, -2**31])
def test_bad_page_ids_are_recorded(M, page):
    lens, rows = [40, 50], [1, 2]
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 16, 0)
    q = queries(3, 4, 1)
    want = ref.attention(q, k, v, table, lens, rows, 4)
    bad = table.clone()
    bad[0, 1] = page
    o, lse, ws = run(M, k, v, bad, n, start, q, 4, 2)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_INVALID_ARG
    ref.check_attention(o[1:], lse[1:], [x[1:] for x in want])
    # a page that holds no visible position is not looked at
    o, lse, ws = run(M, k, v, bad, n, start, q, 4, 2, window=5)
    assert M.moe_workspace_error(ws) == 0
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, 4, window=5))


def test_same_bits_again_in_any_workspace(M):
    lens, rows = [7000, 300, 4000], [4, 2, 4]
    k, v, table, n, start = ref.make_cache(lens, rows, 4, 32, 0)
    q = queries(10, 16, 1)
    o, lse, ws = run(M, k, v, table, n, start, q, 16, 4)
    big = M.paged_workspace(M.PagedKV(k, v, table, n), 16, 16)
    big[256:].random_(0, 255)  # whatever other calls left
    for w in (ws, ws, big, big):
        o2, lse2, _ = run(M, k, v, table, n, start, q, 16, 4, ws=w)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_graph_replay_follows_the_lengths(M):
    lens, rows = [700, 30], [2, 2]
    k, v, table, n, start = ref.make_cache([l + 600 for l in lens], rows, 2, 64, 0)
    kv = M.PagedKV(k, v, table, n)
    q, o, lse = queries(4, 8, 1), torch.zeros(4, 8 * HD, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 8, device="cuda")
    ws = M.paged_workspace(kv, 2, 8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        M.moe_paged_attention(kv, q, start, o, ws, 2, lse=lse)
    side.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, one workspace
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            M.moe_paged_attention(kv, q, start, o, ws, 2, lse=lse)
    for step, add in enumerate((0, 1, 64, 555)):
        n.copy_(ints([l + add for l in lens]))
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        ref.check_attention(o, lse, ref.attention(q, k, v, table, [l + add for l in lens], rows, 8))


def test_another_stream(M):
    lens, rows = [500, 30], [2, 1]
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 64, 0)
    q = queries(3, 8, 1)
    want = ref.attention(q, k, v, table, lens, rows, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o, lse, _ = run(M, k, v, table, n, start, q, 8, 2)
        ref.check_attention(o, lse, want)
    kv, o2 = M.PagedKV(k, v, table, n), torch.zeros_like(o)
    ws = M.paged_workspace(kv, 2, 8)
    torch.cuda.synchronize()
    M.moe_paged_attention(kv, q, start, o2, ws, 2, stream=s)
    s.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("nq,rows", [(8, [2, 1]), (8, [8, 5]), (8, [16, 9])])
def test_output_over_the_queries(M, nq, rows):
    lens = [5000, 40]
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 64, 0)
    q = queries(sum(rows), nq, 1)
    o, lse, ws = run(M, k, v, table, n, start, q, nq, 16)
    kv, got = M.PagedKV(k, v, table, n), q.clone()
    M.moe_paged_attention(kv, got, start, got, ws, 16)
    assert torch.equal(got, o)


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
@pytest.mark.parametrize("more", [0, 1])
def test_output_over_the_queries_in_every_form(M, rows, nq, nkv, more):
    lens, most = [5000, 40], min(16, max(rows) + more)
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 64, 0)
    q = queries(sum(rows), nq, 1, strided=True)
    o, lse, ws = run(M, k, v, table, n, start, q, nq, most)
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, nq))
    wide = torch.full((sum(rows), q.stride(0)), 3.0, dtype=torch.bfloat16, device="cuda")
    got = wide[:, HD:(nq + 1) * HD]
    got.copy_(q)
    M.moe_paged_attention(M.PagedKV(k, v, table, n), got, start, got, ws, most)
    assert torch.equal(got, o)
    assert bool((wide[:, :HD] == 3).all()) and bool((wide[:, (nq + 1) * HD:] == 3).all())


def test_no_rows(M):
    k, v, table, n, start = ref.make_cache([5], [0], 2, 16, 0)
    kv = M.PagedKV(k, v, table, n)
    ws, q = M.paged_workspace(kv, 1, 4), queries(0, 4, 1)
    M.moe_paged_kv_append(kv, queries(0, 2, 2), queries(0, 2, 3), start, ws, q=q, q_out=q)
    M.moe_paged_attention(kv, q, start, q, ws, 1)
    assert M.moe_workspace_error(ws) == 0


@pytest.mark.parametrize("nq,rows", [(8, [2, 1]), (8, [16, 9])])
def test_two_streams_at_once(M, nq, rows):
    lens = [[6000, 300], [100, 9000]]
    caches = [ref.make_cache(l, rows, 2, 64, i) for i, l in enumerate(lens)]
    kvs, qs = [M.PagedKV(*c[:4]) for c in caches], [queries(sum(rows), nq, i) for i in range(2)]
    ws, os_ = [M.paged_workspace(kv, 16, nq) for kv in kvs], [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in kvs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            M.moe_paged_attention(kvs[i], qs[i], caches[i][4], os_[i], ws[i], 16, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        k, v, table = caches[i][:3]
        ref.check_attention(os_[i], None, ref.attention(qs[i], k, v, table, lens[i], rows, nq))


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
def test_two_streams_at_once_in_every_form(M, rows, nq, nkv):
    lens = [[6000, 300], [100, 9000]]
    caches = [ref.make_cache(l, rows, nkv, 64, i) for i, l in enumerate(lens)]
    kvs, qs = [M.PagedKV(*c[:4]) for c in caches], [queries(sum(rows), nq, i) for i in range(2)]
    ws, os_ = [M.paged_workspace(kv, max(rows), nq) for kv in kvs], [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in kvs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            M.moe_paged_attention(kvs[i], qs[i], caches[i][4], os_[i], ws[i], max(rows), stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        k, v, table = caches[i][:3]
        ref.check_attention(os_[i], None, ref.attention(qs[i], k, v, table, lens[i], rows, nq))


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
def test_graphs_of_every_form_share_a_workspace(M, rows, nq, nkv):
    lens = [[700, 30], [5, 4000]]
    caches = [ref.make_cache([l + 400 for l in ls], rows, nkv, 64, i) for i, ls in enumerate(lens)]
    kvs, qs = [M.PagedKV(*c[:4]) for c in caches], [queries(sum(rows), nq, i) for i in range(2)]
    os_, ws = [torch.empty_like(q) for q in qs], M.paged_workspace(kvs[0], max(rows), nq)
    call = lambda i: M.moe_paged_attention(kvs[i], qs[i], caches[i][4], os_[i], ws, max(rows))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(0)
    side.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i)
    for add in (0, 63, 399):
        for i in range(2):
            kvs[i].kv_len.copy_(ints([l + add for l in lens[i]]))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            k, v, table = caches[i][:3]
            ref.check_attention(os_[i], None, ref.attention(qs[i], k, v, table, [l + add for l in lens[i]], rows, nq))
    assert M.moe_workspace_error(ws) == 0


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
def test_idle_sequences_between_long_ones(M, rows, nq, nkv):
    # a server's slots: most have no rows this time, some of them long histories all the same
    lens = [3000] + [(i * 13) % 200 for i in range(500)] + [2000] + [(i * 7) % 90 for i in range(400)]
    all_rows = [rows[0]] + [0] * 500 + [rows[1]] + [0] * 400
    k, v, table, n, start = ref.make_cache(lens, all_rows, nkv, 64, 0)
    n[7], n[600] = -5, 2**31 - 1  # nobody looks at the length of a sequence without rows
    q = queries(sum(rows), nq, 1)
    o, lse, ws = run(M, k, v, table, n, start, q, nq, max(rows))
    assert M.moe_workspace_error(ws) == 0
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, all_rows, nq))


def test_a_captured_step_appends_and_attends(M):
    # append, attention and commit as one graph: each replay sees what the one before appended
    lens, K, nq, nkv, ps = [60, 3, 250], 3, 8, 2, 64
    k, v, table, n, start = ref.make_cache([l + 5 * K for l in lens], [K] * 3, nkv, ps, 0)
    n.copy_(ints(lens))
    kv, pos = M.PagedKV(k, v, table, n), M.attn_pos(rotary_dim=128)
    qkv = queries(3 * K, nq + 2 * nkv, 1)
    a, b = nq * HD, (nq + nkv) * HD
    q, o, ws = torch.empty(3 * K, a, dtype=torch.bfloat16, device="cuda"), torch.empty(3 * K, a, dtype=torch.bfloat16, device="cuda"), \
        M.paged_workspace(kv, K, nq)
    step = lambda: (M.moe_paged_kv_append(kv, qkv[:, a:b], qkv[:, b:], start, ws, q=qkv[:, :a], q_out=q, pos=pos),
                    M.moe_paged_attention(kv, q, start, o, ws, K))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        qkv.normal_()
        n.copy_(ints([l + i * K for l in lens]))
        g.replay()
        torch.cuda.synchronize()
        ref.check_attention(o, None, ref.attention(q, k, v, table, [l + i * K for l in lens], [K] * 3, nq))
        for s, l in enumerate(lens):  # the values as they came
            for j in range(K):
                p = l + i * K + j
                assert torch.equal(v[table[s, p // ps].long(), :, p % ps].flatten(), qkv[s * K + j, b:])
    assert M.moe_workspace_error(ws) == 0


def test_offsets_past_32_bits(M):
    # a pool of 2^31 + elements: the last pages lie past 2^32 bytes and 2^31 elements
    nkv, ps = 8, 128
    pages = 2**31 // (nkv * ps * HD) + 40
    k, v = (torch.zeros(pages, nkv, ps, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(pages - 6, pages, dtype=torch.int32, device="cuda").reshape(2, 3)
    k[pages - 6:].normal_()
    v[pages - 6:].normal_()
    n, start = ints([300, 200]), ints([0, 1, 3])
    q = queries(3, 8, 1)
    o, lse, _ = run(M, k, v, table, n, start, q, 8, 2)
    ref.check_attention(o, lse, ref.attention(q, k, v, table, [300, 200], [1, 2], 8))
    kv = M.PagedKV(k, v, table, n)
    rows = torch.randn(3, nkv * HD, device="cuda").bfloat16()
    M.moe_paged_kv_append(kv, rows, -rows, start, M.paged_workspace(kv, 1, 8))
    assert torch.equal(k[pages - 6 + 2, :, 300 - 256].reshape(-1), rows[0])
    assert torch.equal(v[pages - 6 + 4, :, 201 - 128].reshape(-1), -rows[2])


# ---------------------------------------------------------------- append

def append_case(M, lens, rows, nq, nkv, ps, rd=0, theta=10000.0, yarn=0.0, in_place=False, with_q=True, lead=0, seed=0):
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, ps, seed)
    t = sum(rows) + 2 * lead
    start = start + lead
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    qkv = torch.randn(t, (nq + 2 * nkv + 1) * HD, generator=g, device="cuda").bfloat16()
    q, kn, vn = qkv[:, :nq * HD], qkv[:, nq * HD:(nq + nkv) * HD], qkv[:, (nq + nkv) * HD:(nq + 2 * nkv) * HD]
    q0, k0, v0, was_k, was_v = q.clone(), kn.clone(), vn.clone(), k.clone(), v.clone()
    kv = M.PagedKV(k, v, table, n)
    ws = M.paged_workspace(kv, 1, nkv)
    pos = M.attn_pos(rotary_dim=rd, rope_theta=theta, yarn_factor=yarn, yarn_orig_ctx=4096)
    out = (q if in_place else torch.full((t, nq * HD), 7.0, dtype=torch.bfloat16, device="cuda")) if with_q else None
    M.moe_paged_kv_append(kv, kn, vn, start, ws, q=q if with_q else None, q_out=out, pos=pos)
    torch.cuda.synchronize()
    assert M.moe_workspace_error(ws) == 0
    at = torch.cat([torch.arange(r, device="cuda") + l for l, r in zip(lens, rows)]) if sum(rows) else ints([]).long()
    b = torch.tensor([i for i, r in enumerate(rows) for _ in range(r)], device="cuda", dtype=torch.long)
    f = ref.rotary_freqs(rd, theta, yarn, 4096)
    live = slice(lead, t - lead)
    want_q = ref.rotate(q0[live].double().unflatten(1, (-1, HD)), at, f)
    want_k = ref.rotate(k0[live].double().unflatten(1, (-1, HD)), at, f)
    page, slot = table[b, at // ps].long(), at % ps
    # half a bf16 step, and the FP32 work before it: cos and sin to 2^-22, three roundings of values up to |x| + |y|
    near = lambda got, want: bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 16).all())
    assert near(k[page, :, slot], want_k)
    assert torch.equal(v[page, :, slot], v0[live].unflatten(1, (-1, HD)))
    if rd == 0:
        assert torch.equal(k[page, :, slot], k0[live].unflatten(1, (-1, HD)))
    if with_q:
        assert near(out[live].unflatten(1, (-1, HD)), want_q)
        for edge in (slice(0, lead), slice(t - lead, t)):
            assert torch.equal(out[edge], q0[edge] if in_place else torch.full_like(out[edge], 7.0))
    # nothing else changed
    k[page, :, slot] = was_k[page, :, slot]
    v[page, :, slot] = was_v[page, :, slot]
    assert torch.equal(k, was_k) and torch.equal(v, was_v)


@pytest.mark.parametrize("rd", [0, 2, 16, 20, 32, 64, 96, 126, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_rotary_widths(M, rd, in_place):
    append_case(M, [0, 15, 100, 16383], [1, 4, 0, 3], 4, 2, 16, rd=rd, in_place=in_place, lead=1)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_append_page_sizes_and_yarn(M, ps):
    append_case(M, [63, 64, 1, 127, 200000], [3, 2, 140, 1, 5], 6, 3, ps, rd=64, theta=500000.0, yarn=4.0)


def test_append_without_queries(M):
    append_case(M, [5, 50], [2, 1], 4, 1, 16, rd=128, with_q=False)


@pytest.mark.parametrize("rows", [[1], [1500, 301], [700] * 4, [1] * 1024])
def test_append_many_rows(M, rows):
    append_case(M, [(i * 37) % 90 for i in range(len(rows))], rows, 2, 1, 32, rd=128)


@pytest.mark.parametrize("rows", [[610], [1500, 301, 3], [2400, 500]])
@pytest.mark.parametrize("nq,nkv", [(8, 1), (4, 2), (2, 2), (16, 2)])
def test_append_rows_side_by_side(M, nq, nkv, rows):
    # few heads and many rows: a CTA works on several rows at once
    append_case(M, [3] * len(rows), rows, nq, nkv, 16, rd=64, in_place=nq == 8)


def test_append_past_the_pages_is_recorded(M):
    lens, rows = [30, 10, 5], [4, 2, 3]
    k, v, table, n, start = ref.make_cache(lens, rows, 1, 16, 0, spare=0)
    table = table[:, :2].contiguous()   # two pages: position 32 and on have none
    table[1, 0] = -3
    n[2] = -1
    was_k = k.clone()
    kv = M.PagedKV(k, v, table, n)
    rows_ = torch.randn(9, HD, device="cuda").bfloat16()
    ws = M.paged_workspace(kv, 1, 1)
    M.moe_paged_kv_append(kv, rows_, rows_, start, ws)
    assert M.moe_workspace_error(ws) in (M.MOE_ERR_CAPACITY, M.MOE_ERR_INVALID_ARG)
    p = table[0, 1].long()
    assert torch.equal(k[p, 0, 14:16], rows_[:2])
    k[p, 0, 14:16] = was_k[p, 0, 14:16]
    assert torch.equal(k, was_k)


WRONG_STARTS = [[-1, 2, 4, 6], [0, 2, 4, 7], [0, 4, 2, 6], [0, 2, -1, 6], [0, 2, 4, 2**31 - 1], [0, 2, -2**31, 6],
                [-2**31, 0, 3, 6], [-2**31, 2**31 - 1, -5, 6], [7, 9, 4, 6], [6, 4, 2, 0], [100, 100, 0, 3]]


@pytest.mark.parametrize("rd", [0, 20, 64])
@pytest.mark.parametrize("start", WRONG_STARTS)
def test_append_skips_wrong_rows_and_records_them(M, start, rd):
    # as in the attention: a sequence whose rows are not the call's is left out, the others are not
    lens, T, nq = [30, 10, 5], 6, 2
    k, v, table, n, good = ref.make_cache([40] * 3, [4] * 3, 1, 16, 0)
    n.copy_(ints(lens))
    good = good // 2  # two rows each
    was_k, was_v = k.clone(), v.clone()
    kv, pos = M.PagedKV(k, v, table, n), M.attn_pos(rotary_dim=rd)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, kn, vn = (torch.randn(T, h * HD, generator=g, device="cuda").bfloat16() for h in (nq, 1, 1))
    out, ws = torch.full_like(q, 7.0), M.paged_workspace(kv, 1, nq)
    M.moe_paged_kv_append(kv, kn, vn, ints(start), ws, q=q, q_out=out, pos=pos)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_INVALID_ARG
    assert M.moe_workspace_error(ws) == 0
    freq = ref.rotary_freqs(rd, 10000.0)
    for t in range(T):
        b = max([b for b in range(3) if 0 <= start[b] <= t < start[b + 1] <= T], default=None)
        if b is None:
            assert bool((out[t] == 7).all())
            continue
        p = lens[b] + t - start[b]
        page, at = table[b, p // 16].long(), ints([p])
        want = [ref.rotate(x[t:t + 1].double().unflatten(1, (-1, HD)), at, freq)[0] for x in (q, kn)]
        for got, w in ((out[t].view(nq, HD), want[0]), (k[page, :, p % 16], want[1])):
            assert bool(((got.double() - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -20 * 16).all())
        assert torch.equal(v[page, 0, p % 16], vn[t])
        k[page, :, p % 16], v[page, :, p % 16] = was_k[page, :, p % 16], was_v[page, :, p % 16]
    assert torch.equal(k, was_k) and torch.equal(v, was_v)
    M.moe_paged_kv_append(kv, kn, vn, good, ws, q=q, q_out=out, pos=pos)  # the workspace stays usable
    assert M.moe_workspace_error(ws) == 0
    assert torch.equal(v[table[2, 0].long(), 0, 5:7], vn[4:])


def test_append_of_many_sequences_with_wrong_rows(M):
    # several rows a CTA; two of 1000 sequences wrong, and sequences without rows
    B, lens = 1000, [(i * 7) % 20 for i in range(1000)]
    rows = [i % 6 for i in range(B)]
    k, v, table, n, start = ref.make_cache(lens, rows, 1, 16, 0)
    s = start.tolist()
    bad = list(s)
    bad[500] = s[500] - 3 - 2**20       # sequence 499 falls, 500 starts before the rows
    T = s[-1] - 2                       # and the last one ends behind them
    vn = torch.randn(T, HD, device="cuda").bfloat16()
    kv, was = M.PagedKV(k, v, table, n), v.clone()
    ws = M.paged_workspace(kv, 1, 1)
    M.moe_paged_kv_append(kv, vn, vn, ints(bad), ws)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_INVALID_ARG
    for b in range(B):
        if b not in (499, 500, B - 1):
            for i in range(rows[b]):
                p = lens[b] + i
                was[table[b, p // 16].long(), 0, p % 16] = vn[s[b] + i]
    assert torch.equal(v, was)


# ---------------------------------------------------------------- together

def test_a_verify_loop_over_pages(M):
    """Rounds of a batch as a server runs them: project, append with rotary
    positions, attend, lm_head logits under rules, accepted prefix, commit."""
    H, nq, nkv, V, K, ps = 256, 4, 2, 1003, 4, 16
    lens = [5, 30, 0]
    B, T = len(lens), len(lens) * K
    k, v, table, n, start = ref.make_cache([l + 60 for l in lens], [K] * B, nkv, ps, 0)
    n.copy_(ints(lens))
    kv = M.PagedKV(k, v, table, n)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w_qkv = (torch.randn(H, (nq + 2 * nkv) * HD, generator=g, device="cuda") / 16).bfloat16()
    w_o = (torch.randn(nq * HD, H, generator=g, device="cuda") / 22).bfloat16()
    w_v = (torch.randn(V, H, generator=g, device="cuda") / 16).bfloat16()
    pos = M.attn_pos(rotary_dim=128)
    ws, lws, hws = M.paged_workspace(kv, K, nq), M.logits_workspace(T, V), M.lm_head_workspace(T)
    freq = ref.rotary_freqs(128, 10000.0)
    tokens = torch.randint(0, V, (B * 200,), generator=g, device="cuda", dtype=torch.int32)
    shadow = [[], [], []]  # committed (rotated) keys and values of every sequence, from the cache itself
    for rnd in range(3):
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        qkv = x @ w_qkv
        q = torch.empty(T, nq * HD, dtype=torch.bfloat16, device="cuda")
        a, b = nq * HD, (nq + nkv) * HD
        before = n.tolist()
        M.moe_paged_kv_append(kv, qkv[:, a:b], qkv[:, b:], start, ws, q=qkv[:, :a], q_out=q, pos=pos)
        o = torch.empty_like(q)
        M.moe_paged_attention(kv, q, start, o, ws, K)
        h = x + o @ w_o
        logits = torch.empty(T, V, device="cuda")
        M.moe_lm_head_logits(h, w_v, logits, hws)
        rules = M.LogitRules(tokens=tokens, begin=ints([i // K * 200 for i in range(T)]),
                             end=ints([i // K * 200 + 50 + i % K for i in range(T)]),
                             repetition=torch.full((T,), 1.2, device="cuda"))
        target = torch.empty(T, dtype=torch.int32, device="cuda")
        M.moe_logits_constrain(logits, rules, lws, out=logits, tok=target)
        draft = target.clone()
        draft[1] = -5         # sequence 0 accepts one draft, sequence 1 all, sequence 2 none
        draft[2 * K] = -5
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        for s in range(B):
            M.verify_accept_prefix(draft[s * K:(s + 1) * K], target[s * K:(s + 1) * K], acc[s:])
            M.moe_kv_commit(n[s:], acc[s:], K, 10**6)
        torch.cuda.synchronize()
        assert acc.tolist() == [1, K, 0]
        assert n.tolist() == [before[0] + 2, before[1] + K, before[2] + 1]
        at = torch.tensor([l + i for l in before for i in range(K)], device="cuda")
        want_q = ref.rotate(qkv[:, :a].double().unflatten(1, (-1, HD)), at, freq)
        assert bool(((q.double().unflatten(1, (-1, HD)) - want_q).abs() <= 2.0 ** -8 * want_q.abs() + 2.0 ** -16).all())
        ref.check_attention(o, None, ref.attention(q, k, v, table, before, [K] * B, nq), f"round {rnd}")
        out, tok, _ = ref.logits((h.double() @ w_v.double().T).float().cpu(), tokens.cpu(),
                                 [i // K * 200 for i in range(T)], [i // K * 200 + 50 + i % K for i in range(T)],
                                 torch.full((T,), 1.2))
        assert bool((logits.cpu() - out).abs().max() <= 1e-4)
        for s in range(B):  # what was committed stays where it is
            for p, (kk, vv) in enumerate(shadow[s]):
                page, slot = table[s, p // ps].long(), p % ps
                assert torch.equal(k[page, :, slot], kk) and torch.equal(v[page, :, slot], vv)
            for p in range(len(shadow[s]), int(n[s])):
                page, slot = table[s, p // ps].long(), p % ps
                shadow[s].append((k[page, :, slot].clone(), v[page, :, slot].clone()))
    for w in (ws, lws, hws):
        assert M.moe_workspace_error(w) == 0


@pytest.mark.parametrize("nq,rows", [(8, [1, 2]), (8, [4, 8])])
def test_wait_limit_is_recorded_and_recovered(M, nq, rows):
    # a zero limit makes every wait give up at once: the call returns, says so, and a zero-filled
    # workspace works again
    lens = [3000, 500]
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 64, 0)
    q = queries(sum(rows), nq, 1)
    ws = M.paged_workspace(M.PagedKV(k, v, table, n), 8, nq)
    torch.cuda.synchronize()
    try:
        M.moe_debug_set_wait_limit_ns(0)
        run(M, k, v, table, n, start, q, nq, 8, ws=ws)
        torch.cuda.synchronize()
    finally:
        M.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_DEVICE_TIMEOUT
    ws.zero_()
    o, lse, _ = run(M, k, v, table, n, start, q, nq, 8, ws=ws)
    assert M.moe_workspace_error(ws) == 0
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, nq))


def test_wait_limit_with_many_rows(M):
    # the same for more than 32 query rows a KV head
    lens, rows, nq = [3000, 500], [9, 12], 8
    k, v, table, n, start = ref.make_cache(lens, rows, 2, 64, 0)
    q = queries(sum(rows), nq, 1)
    ws = M.paged_workspace(M.PagedKV(k, v, table, n), 16, nq)
    torch.cuda.synchronize()
    try:
        M.moe_debug_set_wait_limit_ns(0)
        run(M, k, v, table, n, start, q, nq, 16, ws=ws)
        torch.cuda.synchronize()
    finally:
        M.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_DEVICE_TIMEOUT
    ws.zero_()
    o, lse, _ = run(M, k, v, table, n, start, q, nq, 16, ws=ws)
    assert M.moe_workspace_error(ws) == 0
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, nq))


@pytest.mark.parametrize("rows,nq,nkv", FORMS)
def test_wait_limit_in_every_form(M, rows, nq, nkv):
    lens = [3000, 500]
    k, v, table, n, start = ref.make_cache(lens, rows, nkv, 64, 0)
    q = queries(sum(rows), nq, 1)
    ws = M.paged_workspace(M.PagedKV(k, v, table, n), max(rows), nq)
    torch.cuda.synchronize()
    try:
        M.moe_debug_set_wait_limit_ns(0)
        run(M, k, v, table, n, start, q, nq, max(rows), ws=ws)
        torch.cuda.synchronize()
    finally:
        M.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert M.moe_workspace_error(ws) == M.MOE_ERR_DEVICE_TIMEOUT
    ws.zero_()
    o, lse, _ = run(M, k, v, table, n, start, q, nq, max(rows), ws=ws)
    assert M.moe_workspace_error(ws) == 0
    ref.check_attention(o, lse, ref.attention(q, k, v, table, lens, rows, nq))
