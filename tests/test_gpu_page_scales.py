"""The scorer, the attends and the step on a cache with page scales against
attention written in 64 bits, and appends and steps together as a model runs
them."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import (D, F8, GROUP, PAGE, Append, attend64, check_attend, codes, draw_lists,
                              layout, table)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = D ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def _inputs(seq_lens, q_lens, Hkv, seed, spread=1.0, sides=2, powers=False, nan=True, q8=False,
            q_std=1.0):
    """Scales around 2^-8, log-normal with `spread` binades (powers: powers of
    two); NaN codes in every row past a request's last token and in pages that
    belong to nobody."""
    gen = torch.Generator().manual_seed(seed)
    bt, nb = layout(seq_lens, gen, spare=2)
    kv = codes((nb, Hkv, PAGE, D * sides), gen)
    if nan:
        free = set(range(nb))
        for b, L in enumerate(seq_lens):
            n = -(-L // PAGE)
            free -= set(bt[b, :n].tolist())
            if L % PAGE:
                kv[int(bt[b, n - 1]), :, L % PAGE:] = 0x7F
        kv[sorted(free)] = 0x7F
    e = torch.randn((nb, Hkv, sides), generator=gen) * spread - 8
    sc = torch.exp2(e.round() if powers else e)
    q = (torch.randn((sum(q_lens), GROUP * Hkv, D), generator=gen) * q_std).to(torch.bfloat16)
    qs = 1.0
    if q8:
        qs = 0.011
        q = (q.float() / qs).clamp(-448, 448).to(F8)
    # out-of-use table entries point at a page of NaN
    dead = sorted(set(range(nb)) - set(x for b, L in enumerate(seq_lens)
                                       for x in bt[b, :-(-L // PAGE)].tolist()))[0]
    for b, L in enumerate(seq_lens):
        bt[b, -(-L // PAGE):] = dead
    d = dict(kv=kv, sc=sc, bt=bt, q=q, lens=torch.tensor(seq_lens, dtype=torch.int32))
    d = {k: t.to(DEV) for k, t in d.items()}
    d.update(q_lens=list(q_lens), seq_lens=list(seq_lens), qs=qs, Hkv=Hkv,
             lists=draw_lists(seq_lens, q_lens, Hkv, gen).to(DEV))
    return d


def _ref(c, lists=None, ks=1.0, vs=1.0):
    q = c["q"].double() * c["qs"]
    return attend64(q, c["kv"], c["sc"], c["bt"], c["seq_lens"], c["q_lens"], SM, ks, vs, lists)


SHAPES = [
    # seq_lens, Q, Hkv, q8
    ([2048, 3000], 1, 1, False),
    ([1, 129, 0, 5000], 1, 2, True),
    ([257, 513, 2, 0, 130], 4, 2, False),
    ([257, 2100, 2, 0, 130], 3, 1, True),
    ([700, 9000], 2, 1, False),
    ([2500, 700], 32, 1, False),
    ([2500, 17], 8, 1, True),
    ([1200, 600], 9, 1, False),
    ([1500, 640], 16, 1, True),
]


@pytest.mark.parametrize("seq_lens,Q,Hkv,q8", SHAPES)
def test_score(seq_lens, Q, Hkv, q8):
    """Scores within 2^-18 of the row's largest terms (the query's hi + lo parts)
    plus 32-bit sums of 128 products; -inf exactly where nothing is visible."""
    c = _inputs(seq_lens, [Q] * len(seq_lens), Hkv, 21, spread=2.0, q8=q8)
    _, _, want = _ref(c, ks=0.7)
    got = msa.score(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, 0.7, kv_scales=c["sc"],
                    q_scale=c["qs"])
    fin = torch.isfinite(want)
    assert torch.equal(torch.isneginf(got), ~fin)
    # |q|_max sum|K8| scale bounds each logit's terms; a page's largest is 448 * 128
    size = (c["q"].double().abs().max() * c["qs"] * 448 * 128 * SM * 0.7
            * c["sc"][..., 0].max().double())
    assert ((got.double() - want)[fin].abs() <= (2.0 ** -18 + 2.0 ** -20) * size).all()
    rel = (got.double() - want)[fin].norm() / want[fin].norm()
    assert rel < 2.0 ** -17
    assert msa.get_error() == 0


def test_score_of_unit_scales_has_the_plain_scorers_bits():
    c = _inputs([257, 5000, 0, 1300], [4] * 4, 2, 22)
    c["sc"].fill_(1.0)
    a = msa.score(c["q"], c["kv"], c["bt"], c["lens"], 4, SM, 0.3)
    b = msa.score(c["q"], c["kv"], c["bt"], c["lens"], 4, SM, 0.3, kv_scales=c["sc"])
    assert torch.equal(a, b)


@pytest.mark.parametrize("Q,q8", [(1, False), (4, True), (32, False)])
def test_score_on_a_k_only_cache(Q, q8):
    lens = [900, 40, 3000]
    c = _inputs(lens, [Q] * 3, 2, 23, sides=1, q8=q8)
    both = torch.zeros((*c["kv"].shape[:3], 2 * D), dtype=torch.uint8, device=DEV)
    both[..., :D] = c["kv"]
    sc2 = torch.cat([c["sc"], torch.ones_like(c["sc"])], dim=2)
    kw = dict(q_scale=c["qs"])
    a = msa.score(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"], **kw)
    b = msa.score(c["q"], both, c["bt"], c["lens"], Q, SM, kv_scales=sc2, **kw)
    assert torch.equal(a, b) and torch.isfinite(a).any()


@pytest.mark.parametrize("seq_lens,Q,Hkv,q8", SHAPES)
@pytest.mark.parametrize("splits,union", [(0, False), (1, False), (3, False), (2, True)])
def test_sparse_decode(seq_lens, Q, Hkv, q8, splits, union):
    c = _inputs(seq_lens, [Q] * len(seq_lens), Hkv, 24, spread=2.0, q8=q8)
    out, bound, _ = _ref(c, c["lists"], 0.9, 1.3)
    was = msa.set_union_tile(union)
    try:
        got = msa.sparse_decode(c["q"], c["kv"], c["bt"], c["lens"], c["lists"], Q, SM, 0.9, 1.3,
                                num_splits=splits, kv_scales=c["sc"], q_scale=c["qs"])
    finally:
        msa.set_union_tile(was)
    check_attend(got, out, bound)
    assert (got[(out == 0).all(dim=2)] == 0).all()
    assert msa.get_error() == 0


@pytest.mark.parametrize("seq_lens,Q,Hkv,q8", SHAPES)
def test_dense_decode(seq_lens, Q, Hkv, q8):
    c = _inputs(seq_lens, [Q] * len(seq_lens), Hkv, 25, spread=2.0, q8=q8)
    out, bound, _ = _ref(c, None, 0.9, 1.3)
    got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, 0.9, 1.3,
                           kv_scales=c["sc"], q_scale=c["qs"])
    check_attend(got, out, bound)
    assert (got[(out == 0).all(dim=2)] == 0).all()
    assert msa.get_error() == 0


@pytest.mark.parametrize("Q,L", [(1, 262144), (4, 131000), (1, 200001)])
def test_dense_decode_long(Q, L):
    """Hundreds to 2048 pages in one request: every part of a split row."""
    c = _inputs([L, 300], [Q, Q], 1, 26, spread=1.0)
    out, bound, _ = _ref(c)
    got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
    check_attend(got, out, bound)
    assert msa.get_error() == 0


def test_dense_decode_on_more_units_than_processors():
    """One part a unit: ranges of more than 32 pages read their scales ahead."""
    lens = [5000, 9000, 127, 0] * 10
    c = _inputs(lens, [2] * 40, 4, 27)
    out, bound, _ = _ref(c)
    got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], 2, SM, kv_scales=c["sc"])
    check_attend(got, out, bound)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("seq_lens,q_lens", [([129, 5000, 700, 40], [129, 37, 0, 1]),
                                             ([300, 0, 2500], [5, 0, 61])])
def test_sparse_prefill(seq_lens, q_lens, q8):
    c = _inputs(seq_lens, q_lens, 2, 28, q8=q8)
    cu = torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32, device=DEV)
    out, bound, _ = _ref(c, c["lists"])
    got = msa.sparse_prefill(c["q"], c["kv"], c["bt"], c["lens"], cu, c["lists"], SM,
                             kv_scales=c["sc"], q_scale=c["qs"])
    check_attend(got, out, bound)
    # from scores: the selector's lists, the same attend
    scores = torch.randn((2, sum(q_lens), c["bt"].shape[1]), device=DEV)
    tk, got = msa.sparse_prefill_select(c["q"], c["kv"], c["bt"], c["lens"], cu, scores, SM,
                                        kv_scales=c["sc"], q_scale=c["qs"])
    again = msa.sparse_prefill(c["q"], c["kv"], c["bt"], c["lens"], cu, tk, SM, kv_scales=c["sc"],
                               q_scale=c["qs"])
    assert torch.equal(got, again)
    out, bound, _ = _ref(c, tk)
    check_attend(got, out, bound)
    assert msa.get_error() == 0


@pytest.mark.parametrize("q8", [False, True])
def test_more_rows_than_ctas(q8):
    """Rows for several waves: CTAs that take row after row (330 to 1100 rows), with
    rows of no page, of one page, of an odd number of pages and of 16 between them."""
    gen = torch.Generator().manual_seed(5)
    q_lens = [120, 1, 0, 90, 60, 3]
    lens = [2300, 1, 0, 90, 700, 5000]
    c = _inputs(lens, q_lens, 4, 41, spread=2.0, q8=q8)
    holes = torch.rand(c["lists"].shape, generator=gen).to(DEV)
    c["lists"] = torch.where(holes < 0.3, -1, c["lists"])
    c["lists"][5:9] = -1
    cu = torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32, device=DEV)
    out, bound, _ = _ref(c, c["lists"], 0.9, 1.3)
    args = (c["q"], c["kv"], c["bt"], c["lens"], cu, c["lists"], SM, 0.9, 1.3)
    got = msa.sparse_prefill(*args, kv_scales=c["sc"], q_scale=c["qs"])
    check_attend(got, out, bound)
    assert (got[5:9] == 0).all()
    for _ in range(5):   # whatever the roles' timing: the same bits
        assert torch.equal(got, msa.sparse_prefill(*args, kv_scales=c["sc"], q_scale=c["qs"]))
    assert msa.get_error() == 0
    # tokens past the last request, a bad scale and a bad page in the middle
    cu[-1] = 270
    page = int(c["bt"][0, 3])
    c["sc"][page, 1, 0] = float("nan")
    c["kv"][page, 1] = 0x7F
    got2 = msa.sparse_prefill(*args, kv_scales=c["sc"], q_scale=c["qs"])
    assert msa.get_error() == _native.ERR_SEQ_RANGE | _native.ERR_SCALE
    assert (got2[270:] == 0).all() and torch.isfinite(got2.float()).all()
    same = ~(c["lists"][:120, 1] == 3).any(dim=1)
    assert torch.equal(got2[:120, :16], got[:120, :16]) and torch.equal(got2[120:270], got[120:270])
    assert torch.equal(got2[:120][same], got[:120][same])


def test_a_decode_batch_of_more_rows_than_ctas():
    lens = [(k * 37) % 1500 if k % 10 else 0 for k in range(128)]
    c = _inputs(lens, [1] * 128, 4, 42)
    out, bound, _ = _ref(c, c["lists"])
    got = msa.sparse_decode(c["q"], c["kv"], c["bt"], c["lens"], c["lists"], 1, SM,
                            kv_scales=c["sc"])
    check_attend(got, out, bound)
    assert (got[torch.tensor(lens) == 0] == 0).all()
    assert msa.get_error() == 0


@pytest.mark.parametrize("spread_pages", [[-40, 0, -20, 30], [40, -40, 40, -40], [3, 2, 1, 0]])
@pytest.mark.parametrize("kind", ["sparse", "union", "dense"])
def test_scales_over_their_whole_range(spread_pages, kind):
    """Page V scales from 2^-40 to 2^40 in one list: each element within the
    bound its page's share allows (a small page beside a huge one drowns in the
    output, not in the arithmetic); K scales that make one page's logits 0."""
    Q = 2
    c = _inputs([4 * PAGE], [Q], 1, 29)
    for n, e in enumerate(spread_pages):
        c["sc"][c["bt"][0, n], 0, 1] = 2.0 ** e
        c["sc"][c["bt"][0, n], 0, 0] = 2.0 ** (-40 if n == 2 else -8)
    out, bound, _ = _ref(c)
    if kind == "dense":
        got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
    else:
        lists = torch.full((Q, 1, 16), -1, dtype=torch.int32, device=DEV)
        lists[:, :, :4] = torch.arange(4, dtype=torch.int32)
        was = msa.set_union_tile(kind == "union")
        try:
            got = msa.sparse_decode(c["q"], c["kv"], c["bt"], c["lens"], lists, Q, SM,
                                    kv_scales=c["sc"])
        finally:
            msa.set_union_tile(was)
    check_attend(got, out, bound)
    assert msa.get_error() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 0.0, -1.0, 2.0 ** -41, 2.0 ** 41])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("kind", ["sparse", "union", "dense1", "dense4", "score"])
def test_a_bad_scale_is_flagged_and_its_page_skipped(bad, side, kind):
    Q = 1 if kind == "dense1" else 4
    L = 900
    c = _inputs([L, 600], [Q, Q], 1, 30)
    page = int(c["bt"][0, 3])
    c["kv"][page] = 0x7F                                  # nothing of it may reach the output
    c["sc"][page, 0, side] = bad
    good = c["sc"].clone()
    good[page] = 1.0
    lists = torch.full((2 * Q, 1, 16), -1, dtype=torch.int32, device=DEV)
    lists[:Q, :, :8] = torch.arange(8, dtype=torch.int32)
    lists[Q:, :, :5] = torch.arange(5, dtype=torch.int32)
    less = lists.clone()
    less[:Q, :, 3] = -1
    ref = dict(c, sc=good)
    if kind == "score":
        got = msa.score(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
        if side == 0:
            assert msa.get_error() == _native.ERR_SCALE
            assert torch.isneginf(got[0, :Q, 3]).all() and torch.isfinite(got[0, :Q, :3]).all()
        else:
            assert msa.get_error() == 0                   # the scorer reads no V scale
        return
    out, bound, _ = _ref(ref, less)
    if kind.startswith("dense"):
        got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
    else:
        was = msa.set_union_tile(kind == "union")
        try:
            got = msa.sparse_decode(c["q"], c["kv"], c["bt"], c["lens"], lists, Q, SM,
                                    kv_scales=c["sc"])
        finally:
            msa.set_union_tile(was)
    assert msa.get_error() == _native.ERR_SCALE
    check_attend(got, out, bound)


def test_every_listed_page_bad_gives_zero():
    c = _inputs([400, 300], [1, 1], 1, 31)
    c["sc"][c["bt"][0, :4].long()] = float("nan")
    got = msa.sparse_decode(c["q"], c["kv"], c["bt"], c["lens"], c["lists"], 1, SM,
                            kv_scales=c["sc"])
    assert (got[0] == 0).all() and (got[1] != 0).any()
    for Q in (1, 2):
        q = c["q"].repeat_interleave(Q, dim=0)
        got = msa.dense_decode(q, c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
        assert (got[:Q] == 0).all() and (got[Q:] != 0).any()
    assert msa.get_error() == _native.ERR_SCALE


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kind", ["lists1", "lists4", "parts", "union", "dense1", "dense4", "dense7",
                                  "rows"])
def test_a_nan_reaches_exactly_those_that_see_it(kind, q8):
    """NaN codes of a key (all of its attenders' heads) and of single value dims (that
    dim only), some of them seen by a tile's later tokens alone; a NaN query head."""
    Q = {"lists1": 1, "dense1": 1, "dense7": 7, "rows": 130}.get(kind, 4)
    lens = [900, 514, 386]     # request 1's last four tokens: 510 .. 513, across two pages
    c = _inputs(lens, [Q] * 3, 1, 61, q8=q8)
    bt, kv = c["bt"], c["kv"]
    want_kw = dict(lists=None if kind.startswith("dense") else c["lists"], ks=0.9, vs=1.3)
    clean, bound, _ = _ref(c, **want_kw)
    kv[int(bt[0, 1]), 0, 2, 5] = 0x7F                          # a key of request 0
    if kind != "union":        # (the union's pages are everybody's)
        kv[int(bt[1, 512 // PAGE]), 0, 512 % PAGE, D + 77] = 0xFF
        kv[int(bt[1, 511 // PAGE]), 0, 511 % PAGE, D + 3] = 0x7F
        kv[int(bt[1, 511 // PAGE]), 0, 511 % PAGE, D + 124] = 0x7F
    kv[int(bt[2, 0]), 0, 9, D + 40] = 0x7F
    out, _, _ = _ref(c, **want_kw)
    c["q"].view(torch.uint8 if q8 else torch.int16)[2 * Q, 6, 11] = 0x7F if q8 else 0x7FC0
    out[2 * Q, 6] = float("nan") if (clean[2 * Q, 6] != 0).any() else 0.0
    args = (c["q"], kv, bt, c["lens"])
    kw = dict(kv_scales=c["sc"], q_scale=c["qs"])
    if kind.startswith("dense"):
        got = msa.dense_decode(*args, Q, SM, 0.9, 1.3, **kw)
    elif kind == "rows":
        cu = torch.arange(4, dtype=torch.int32, device=DEV) * Q
        got = msa.sparse_prefill(*args, cu, c["lists"], SM, 0.9, 1.3, **kw)
    else:
        was = msa.set_union_tile(kind == "union")
        try:
            got = msa.sparse_decode(*args, c["lists"], Q, SM, 0.9, 1.3,
                                    num_splits=3 if kind == "parts" else 0, **kw)
        finally:
            msa.set_union_tile(was)
    nan = torch.isnan(out)
    assert nan.any() and not nan.all()
    assert torch.equal(torch.isnan(got), nan)
    check_attend(torch.where(nan, 0.0, got), torch.where(nan, 0.0, out),
                 torch.where(nan, 0.0, bound))
    assert msa.get_error() == 0


@pytest.mark.parametrize("Q", [2, 4])
@pytest.mark.parametrize("S", [0, 600])
def test_step_with_the_union_tile(Q, S):
    """decode_step and the attends with no split count while the union tile is on."""
    lens = [3000, 0, 5000, 1]
    c = _inputs(lens, [Q] * 4, 2, 62)
    bt = torch.zeros((4, max(S, c["bt"].shape[1])), dtype=torch.int32, device=DEV)
    bt[:, :c["bt"].shape[1]] = c["bt"]
    was = msa.set_union_tile(True)
    try:
        s, tk, out = msa.decode_step(c["q"], c["kv"], bt, c["lens"], Q, SM, 1.1, 0.9,
                                     kv_scales=c["sc"])
        out2 = msa.sparse_decode(c["q"], c["kv"], bt, c["lens"], tk, Q, SM, 1.1, 0.9,
                                 kv_scales=c["sc"])
    finally:
        msa.set_union_tile(was)
    o, bound, _ = _ref(dict(c, bt=bt), tk, 1.1, 0.9)
    check_attend(out, o, bound)
    check_attend(out2, o, bound)
    assert msa.get_error() == 0


@pytest.mark.parametrize("Q,q8", [(1, False), (3, True)])
def test_selection_of_long_rows(Q, q8):
    """Selecting attends over rows of 700 to 8200 blocks: the lists of topk and the
    output of the attend on them, decode and prefill."""
    c = _inputs([PAGE * 40, 3], [Q] * 2, 2, 64, q8=q8, nan=False)
    lens = torch.tensor([8200 * PAGE - 5, 700 * PAGE + 1], dtype=torch.int32, device=DEV)
    S = 8200
    gen = torch.Generator().manual_seed(65)
    bt = torch.randint(0, 40, (2, S), generator=gen).to(torch.int32).to(DEV)
    s = torch.randn((2, 2 * Q, S), generator=gen).to(DEV)
    kw = dict(kv_scales=c["sc"], q_scale=c["qs"])
    tk = msa.topk(s, lens, Q)
    out = msa.sparse_decode(c["q"], c["kv"], bt, lens, tk, Q, SM, 1.1, 0.9, **kw)
    cu = torch.arange(3, dtype=torch.int32, device=DEV) * Q
    for splits in (0, 3):
        tk2, out2 = msa.sparse_decode_select(c["q"], c["kv"], bt, lens, s, Q, SM, 1.1, 0.9,
                                             num_splits=splits, **kw)
        tk3, out3 = msa.sparse_prefill_select(c["q"], c["kv"], bt, lens, cu, s, SM, 1.1, 0.9,
                                              num_splits=splits, **kw)
        assert torch.equal(tk, tk2) and torch.equal(tk, tk3) and torch.equal(out2, out3)
        if splits == 0:
            assert torch.equal(out, out2)
    ref = dict(c, bt=bt, seq_lens=lens.tolist())
    o, bound, _ = _ref(ref, tk, 1.1, 0.9)
    check_attend(out, o, bound)
    check_attend(out2, o, bound)
    assert msa.get_error() == 0


@pytest.mark.parametrize("B,Q", [(300, 1), (270, 2), (260, 5)])
def test_dense_decode_of_large_batches(B, Q):
    """More requests than the shared-out assignment takes."""
    lens = [(k * 53) % 260 if k % 7 else 0 for k in range(B)]
    c = _inputs(lens, [Q] * B, 1, 63)
    out, bound, _ = _ref(c)
    got = msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM, kv_scales=c["sc"])
    check_attend(got, out, bound)
    assert (got[(out == 0).all(dim=2)] == 0).all() and msa.get_error() == 0


@pytest.mark.parametrize("Q,S,q8,index", [(1, 1, False, False), (4, 1, True, False),
                                          (4, 600, False, False), (2, 1, False, True),
                                          (4, 600, True, True)])
def test_step_equals_its_stages(Q, S, q8, index):
    """decode_step on page scales: the scores, lists and output of score, topk
    and sparse_decode called in turn (S > 512: the selector's own kernel)."""
    lens = [3000, 0, 5000, 1]
    c = _inputs(lens, [Q] * 4, 2, 32, q8=q8)
    bt = torch.zeros((4, max(S, c["bt"].shape[1])), dtype=torch.int32, device=DEV)
    bt[:, :c["bt"].shape[1]] = c["bt"]
    kw = dict(q_scale=c["qs"])
    ix = {}
    if index:
        ik = c["kv"][..., D:].contiguous()
        isc = c["sc"][..., 1:].contiguous()
        ix = dict(index_k=ik, index_k_scale=0.8, index_scales=isc)
        s = msa.score(c["q"], ik, bt, c["lens"], Q, SM, 0.8, kv_scales=isc, **kw)
    else:
        s = msa.score(c["q"], c["kv"], bt, c["lens"], Q, SM, 1.1, kv_scales=c["sc"], **kw)
    tk = msa.topk(s, c["lens"], Q)
    out = msa.sparse_decode(c["q"], c["kv"], bt, c["lens"], tk, Q, SM, 1.1, 0.9,
                            kv_scales=c["sc"], **kw)
    s2, tk2, out2 = msa.decode_step(c["q"], c["kv"], bt, c["lens"], Q, SM, 1.1, 0.9,
                                    kv_scales=c["sc"], **kw, **ix)
    assert torch.equal(s, s2) and torch.equal(tk, tk2) and torch.equal(out, out2)
    tk3, out3 = msa.sparse_decode_select(c["q"], c["kv"], bt, c["lens"], s, Q, SM, 1.1, 0.9,
                                         kv_scales=c["sc"], **kw)
    assert torch.equal(tk, tk3) and torch.equal(out, out3)
    ref = dict(c, bt=bt)
    o, bound, _ = _ref(ref, tk, 1.1, 0.9)
    check_attend(out, o, bound)
    assert msa.get_error() == 0


def _model_run(scaled, steps, lens, Q, capture=False, overlap=False):
    """A prompt appended, then `steps` decode steps of append and decode_step, on
    one layer; returns what the last step gave and a 64-bit check of it."""
    Hkv, Hq = 2, 32
    gen = torch.Generator().manual_seed(77)
    end = [L + steps * Q for L in lens]
    bt, nb = layout(end, gen)
    bt = bt.to(DEV)
    kv = torch.full((nb, Hkv, PAGE, 2 * D), 0x7F, dtype=torch.uint8, device=DEV)
    sc = torch.full((nb, Hkv, 2), float("nan"), device=DEV) if scaled else None
    ref = Append(kv, sc, bt, lens, 0.02, 0.02) if not scaled else Append(kv, sc, bt, lens)
    per = (1.0, 1.0) if scaled else (0.02, 0.02)
    cs = table(max(end), 64)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)

    def rows(T, k):
        x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen) * (1 + k % 3)
        return x.to(torch.bfloat16).to(DEV).unflatten(1, (-1, D)).split([Hq, Hkv, Hkv], dim=1)

    q, k, v = rows(sum(lens), 0)
    msa.append_kv_prefill(k, v, kv, bt, seq, cu, *per, kv_scales=sc, cos_sin=cs)
    ref.run(k, v, None, lens, cs)
    ref.check(kv, sc)
    ref.settle(kv)
    B = len(lens)
    qb = torch.empty((B * Q, Hq, D), dtype=torch.bfloat16, device=DEV)
    x = torch.empty((B * Q, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device=DEV)
    xs = x.unflatten(1, (-1, D)).split([Hq, Hkv, Hkv], dim=1)
    buffers = msa.DecodeBuffers.allocate(B, Q, Hq, Hkv, bt.shape[1], DEV)

    def step():
        seq.add_(Q)
        msa.append_kv(xs[1], xs[2], kv, bt, seq, Q, *per, kv_scales=sc, cos_sin=cs, q=xs[0],
                      q_out=qb)
        return msa.decode_step(qb, kv, bt, seq, Q, SM, *per, kv_scales=sc, buffers=buffers)

    graph = None
    was = msa.set_input_overlap(overlap)
    try:
        if capture:
            keep = [t.clone() for t in (seq, kv)] + [None if sc is None else sc.clone()]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                x.zero_()
                step()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    step()
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            seq.copy_(keep[0]), kv.copy_(keep[1])
            if sc is not None:
                sc.copy_(keep[2])
            msa.get_error()
        for n in range(steps):
            qn, kn, vn = rows(B * Q, n)
            x.view(B * Q, -1, D).copy_(torch.cat([qn, kn, vn], dim=1))
            graph.replay() if graph else step()
            ref.lens = [L + (n + 1) * Q for L in lens]
            ref.run(kn, vn, None, [Q] * B, cs)
            ref.check(kv, sc)
            ref.settle(kv)
    finally:
        msa.set_input_overlap(was)
    sc64 = sc if scaled else torch.full((nb, Hkv, 2), 1.0, device=DEV)
    out, bound, scores = attend64(qb, kv, sc64, bt, ref.lens, [Q] * B, SM, *per, lists=buffers.topk)
    check_attend(buffers.out, out, bound)
    fin = torch.isfinite(buffers.scores)
    assert fin.any() and msa.get_error() == 0
    return buffers.out.clone(), kv.clone(), None if sc is None else sc.clone()


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("Q", [1, 3])
def test_appends_and_steps_together(scaled, Q):
    """The path as a model runs it, eager, captured and replayed, and with input
    overlap: the same bits each way."""
    runs = [_model_run(scaled, 4, [126, 700, 2500], Q, capture, overlap)
            for capture, overlap in ((False, False), (True, False), (False, True))]
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert a is None or torch.equal(a.nan_to_num() if a.is_floating_point() else a,
                                            b.nan_to_num() if b.is_floating_point() else b)


def test_two_streams_at_once():
    """Two steps with their own buffers on two streams, many times over."""
    cs = [_inputs([3000, 2000], [4, 4], 2, 40 + k) for k in range(2)]
    want, streams, got = [], [torch.cuda.Stream() for _ in cs], [[], []]
    for c in cs:
        want.append(msa.decode_step(c["q"], c["kv"], c["bt"], c["lens"], 4, SM, kv_scales=c["sc"]))
    torch.cuda.synchronize()
    for _ in range(20):
        for k, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[k].append(msa.decode_step(c["q"], c["kv"], c["bt"], c["lens"], 4, SM,
                                              kv_scales=c["sc"])[2])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, want[k][2]) for o in got[k])


def test_a_cache_past_32_bit_offsets():
    """Pages past 2^31 bytes (and past 2^31 elements of scales' rows): the last
    page of a 2.3 GB cache is appended to and attended."""
    NB, Hkv = 70000, 1
    kv = torch.zeros((NB, Hkv, PAGE, 2 * D), dtype=torch.uint8, device=DEV)
    sc = torch.ones((NB, Hkv, 2), device=DEV)
    bt = torch.tensor([[NB - 1, NB - 2]], dtype=torch.int32, device=DEV)
    seq = torch.tensor([129], dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((129, 18, D), generator=gen).to(torch.bfloat16).to(DEV)
    cu = torch.tensor([0, 129], dtype=torch.int32, device=DEV)
    q = msa.append_kv_prefill(x[:, 16:17], x[:, 17:], kv, bt, seq, cu, kv_scales=sc, q=x[:, :16])
    ref = Append(kv[-2:], sc[-2:], torch.tensor([[1, 0]]), [129])
    ref.kv.zero_()
    ref.run(x[:, 16:17], x[:, 17:], None, [129])
    ref.check(kv[-2:], sc[-2:])
    assert (kv[0] == 0).all() and (kv[1] == 0).all()
    last = q[128:].contiguous()
    out = msa.dense_decode(last, kv, bt, seq, 1, SM, kv_scales=sc)
    want, bound, _ = attend64(last, kv[-2:], sc[-2:], torch.tensor([[1, 0]], device=DEV), [129],
                              [1], SM, 1.0, 1.0)
    check_attend(out, want, bound)


def test_python_refusals():
    c = _inputs([300, 20], [1, 1], 2, 33)
    args = (c["q"], c["kv"], c["bt"], c["lens"])
    for sc in (c["sc"][:-1], c["sc"][..., :1].contiguous(), c["sc"].transpose(0, 1), c["sc"].cpu()):
        for f in (lambda s: msa.score(*args, 1, SM, kv_scales=s),
                  lambda s: msa.sparse_decode(*args, c["lists"], 1, SM, kv_scales=s),
                  lambda s: msa.dense_decode(*args, 1, SM, kv_scales=s),
                  lambda s: msa.decode_step(*args, 1, SM, kv_scales=s)):
            with pytest.raises(ValueError):
                f(sc)
    with pytest.raises(TypeError):
        msa.score(*args, 1, SM, kv_scales=c["sc"].double())
    with pytest.raises(ValueError):
        msa.decode_step(*args, 1, SM, kv_scales=c["sc"], index_scales=c["sc"][..., :1].contiguous())
    assert msa.get_error() == 0
