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
