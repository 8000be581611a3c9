"""Orders between threads that no run can be made to show, read from the kernels' source:
what has to stand in front of an access to memory that another thread or CTA uses."""
from __future__ import annotations

import os
import re

import pytest

from block_sparse_gqa_score_gb300 import build


def source(name: str) -> str:
    """The file's code without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def function(text: str, name: str) -> str:
    """The body of the function `name` (its definition)."""
    at = re.search(rf"\b{name}\([^;{{]*\)\s*{{", text)
    assert at, name
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at.end():i]


@pytest.mark.parametrize("kernel", ["fork_kernel", "compact_kernel"])
def test_remote_stores_wait_for_the_cluster(kernel):
    """Another CTA's shared memory may be touched only when the whole cluster has started,
    which a cluster barrier ahead of the first remote store makes sure of."""
    body = function(source("msa_pages.cu"), kernel)
    first = body.index("store_remote(")
    waits = [m.start() for m in re.finditer(r"cluster_started_wait\(\)|cluster_sync\(\)", body)]
    assert waits and waits[0] < first
    assert body.count("cluster_started_arrive()") == body.count("cluster_started_wait()") == 1
    # nobody leaves while others may still store to it
    assert body.rindex("cluster_sync()") > body.rindex("store_remote(")


def test_scratch_of_a_given_up_row_is_ordered():
    """select_by_maxima leaves a row to select_row, which writes the same shared words from
    other lanes: what it wrote itself is ordered before."""
    body = function(source("msa_topk.cu"), "select_by_maxima")
    left = body.index("return false")
    wrote = body.rindex("block[k] =", 0, left)
    assert body.count("return false") == 1
    assert "__syncwarp()" in body[wrote:left]


def test_scorer_waits_for_the_half_that_a_unit_leaves_out():
    """A unit of at most eight tokens uses one half of the tile; its pages' factors take the
    places of those that the other half's warps may still be reading, unless the products
    wait until these have handed back their last pair."""
    body = function(source("msa_score_prefill.cu"), "score_prefill_kernel")
    unit = body[body.index("tail->q_full[i & 1], (i >> 1) & 1"):]
    before = unit[:unit.index("x < pages")]
    assert re.search(r"ntok <= kHalfTokens[^;]*n_1 > 0[^;]*wait\(&tail->s_empty\[1\], \(n_1 - 1\) & 1\)",
                     before)
