"""The page-scale attends where a page or a row drops out: pages that are not attended
at the end of a tile of tokens, rows without pages between others, split counts that a
caller chose."""
from __future__ import annotations

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import D, PAGE, attend64, check_attend, codes, layout

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = D ** -0.5


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _inputs(lens, Q, Hkv, seed):
    """Page 0 belongs to nobody."""
    gen = torch.Generator().manual_seed(seed)
    bt, nb = layout(lens, gen, spare=0)
    nb += 1
    d = dict(kv=codes((nb, Hkv, PAGE, 2 * D), gen), bt=bt + 1,
             sc=torch.exp2(torch.randn((nb, Hkv, 2), generator=gen) - 8),
             q=torch.randn((len(lens) * Q, 16 * Hkv, D), generator=gen).to(torch.bfloat16),
             lens=torch.tensor(lens, dtype=torch.int32))
    return {k: t.to(DEV) for k, t in d.items()}


# the last tokens' pages: one page whose first rows only the later tokens see; two pages;
# the 33rd page of a CTA, whose scales come with another 32 pages (a batch that fills the
# GPU, so that a CTA takes all of a request)
@pytest.mark.parametrize("L,full", [(900, False), (130, False), (32 * PAGE + 2, True)])
@pytest.mark.parametrize("how", ["k_scale", "v_scale", "entry"])
def test_a_tiles_last_page_that_is_not_attended(L, full, how):
    """NaN values in the rows of a tile's last page that its later tokens see, the page
    skipped for a bad scale or a bad table entry (page 0 is loaded in its place): nothing
    of it reaches an output."""
    Q = 4
    c = _inputs([L] + [5] * (_sms() if full else 1), Q, 1, 3)
    last = (L - 1) // PAGE
    if how == "entry":
        c["bt"][0, last] = c["kv"].shape[0]
        spoilt, flag = 0, _native.ERR_PAGE_RANGE
    else:
        spoilt, flag = int(c["bt"][0, last]), _native.ERR_SCALE
        c["sc"][spoilt, 0, int(how == "v_scale")] = float("nan")
    outs = []
    for code in (0, 0x7F):
        c["kv"][spoilt, 0, :6, D:] = code
        outs.append(msa.dense_decode(c["q"], c["kv"], c["bt"], c["lens"], Q, SM,
                                     kv_scales=c["sc"]))
    assert msa.get_error() == flag
    assert torch.isfinite(outs[0].float()).all() and torch.equal(outs[0], outs[1])
    # and it is the attention over the other pages
    n = min(last, 16)
    if n == last:
        lists = torch.full((Q, 1, 16), -1, dtype=torch.int32, device=DEV)
        lists[..., :n] = torch.arange(n, dtype=torch.int32)
        out, bound, _ = attend64(c["q"][:Q].double(), c["kv"], c["sc"], c["bt"][:1], [L], [Q], SM,
                                 1.0, 1.0, lists)
        check_attend(outs[1][:Q], out, bound)


@pytest.mark.parametrize("varlen", [False, True])
def test_long_runs_of_rows_without_pages(varlen):
    """Two dozen rows for every CTA that takes row after row, most of them of padding
    requests or of lists without a block: in runs of one to nine, next to rows of one page
    and of several."""
    wave = 2 * _sms()
    # (visible tokens, listed) of a wave's rows; a CTA gets one row of each
    waves = [(0, 1), (0, 1), (0, 1), (700, 1), (0, 1), (400, 0), (400, 0), (1, 1), (1, 1)]
    waves += [(0, 1)] * 4 + [(300, 0)] * 5 + [(129, 1), (0, 1), (2000, 1), (0, 1), (0, 1)]
    kinds = [w for w in waves for _ in range(wave)] + [(260, 1)] * 7
    lens = [max(n, int(varlen)) for n, _ in kinds]
    B = len(lens)
    gen = torch.Generator().manual_seed(9)
    bt, nb = layout([2100, 700], gen)           # the requests share their pages
    c = dict(kv=codes((nb, 1, PAGE, 2 * D), gen).to(DEV), bt=bt[:1].repeat(B, 1).contiguous().to(DEV),
             sc=torch.exp2(torch.randn((nb, 1, 2), generator=gen) - 8).to(DEV),
             q=torch.randn((B, 16, D), generator=gen).to(torch.bfloat16).to(DEV),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    lists = torch.full((B, 1, 16), -1, dtype=torch.int32)
    for b, (n, listed) in enumerate(kinds):
        if n and listed:
            lists[b, 0, :(n - 1) // PAGE + 1] = torch.arange((n - 1) // PAGE + 1, dtype=torch.int32)
    lists = lists.to(DEV)
    a = (c["q"], c["kv"], c["bt"], c["lens"])
    if varlen:
        cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
        call = lambda: msa.sparse_prefill(*a, cu, lists, SM, kv_scales=c["sc"])
    else:
        call = lambda: msa.sparse_decode(*a, lists, 1, SM, kv_scales=c["sc"])
    got = call()
    for _ in range(20):   # whatever the roles' timing: the same bits
        assert torch.equal(got, call())
    assert msa.get_error() == 0
    some = [b for b in range(B) if (lists[b] >= 0).any()]
    rest = torch.ones(B, dtype=torch.bool)
    rest[some] = False
    assert (got[rest.to(DEV)] == 0).all()
    some = some[::7]
    out, bound, _ = attend64(c["q"][some].double(), c["kv"], c["sc"], c["bt"][some],
                             [lens[b] for b in some], [1] * len(some), SM, 1.0, 1.0, lists[some])
    check_attend(got[some], out, bound)


@pytest.mark.parametrize("lens,Q", [([900, 3000, 0, 5], 4), ([2500], 32), ([700, 40], 2)])
def test_the_union_tile_has_no_say_over_lists_on_page_scales(lens, Q):
    """The same bits with the switch on and off, in every form, also where the caller
    takes its split count from the switch."""
    Hkv, B = 2, len(lens)
    c = _inputs(lens, Q, Hkv, 11)
    gen = torch.Generator().manual_seed(12)
    S = c["bt"].shape[1]
    scores = torch.randn((Hkv, B * Q, S), generator=gen).to(DEV)
    a = (c["q"], c["kv"], c["bt"], c["lens"])
    kw = dict(kv_scales=c["sc"])
    lists = msa.topk(scores, c["lens"], Q)
    outs = []
    for on in (False, True):
        was = msa.set_union_tile(on)
        try:
            buffers = msa.DecodeBuffers.allocate(B, Q, 16 * Hkv, Hkv, S, torch.device(DEV))
            outs.append((msa.sparse_decode(*a, lists, Q, SM, **kw),
                         msa.sparse_decode(*a, lists, Q, SM, num_splits=3, **kw),
                         *msa.sparse_decode_select(*a, scores, Q, SM, **kw),
                         *msa.decode_step(*a, Q, SM, buffers=buffers, **kw)))
        finally:
            msa.set_union_tile(was)
    for off, on in zip(*outs):
        assert torch.equal(off, on)
    assert msa.get_error() == 0


@pytest.mark.parametrize("S", [0, 600])      # selection inside the attend kernel, and before it
@pytest.mark.parametrize("scaled", [True, False])
def test_a_step_takes_the_split_count_of_its_buffers(scaled, S):
    """A count that the caller chose holds, with page scales as without; the one that
    allocate chooses is for the cache with one scale per tensor."""
    lens, Q, Hkv = [2600, 900], 2, 1
    c = _inputs(lens, Q, Hkv, 13)
    bt = torch.zeros((2, max(S, c["bt"].shape[1])), dtype=torch.int32, device=DEV)
    bt[:, :c["bt"].shape[1]] = c["bt"]
    a = (c["q"], c["kv"], bt, c["lens"])
    kw = dict(kv_scales=c["sc"] if scaled else None)
    for chosen in (3, 0):
        bufs = msa.DecodeBuffers.allocate(2, Q, 16 * Hkv, Hkv, bt.shape[1], torch.device(DEV),
                                          num_splits=chosen)
        assert bufs.num_splits == 3 or chosen == 0
        bufs.workspace.fill_(0xA5)
        scores, lists, out = msa.decode_step(*a, Q, SM, buffers=bufs, **kw)
        parts = chosen or (0 if scaled else bufs.num_splits)
        assert bool((bufs.workspace != 0xA5).any()) == (parts > 1)
        assert torch.equal(out, msa.sparse_decode(*a, lists, Q, SM, num_splits=parts, **kw))
    assert msa.get_error() == 0
