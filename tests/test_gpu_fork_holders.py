"""fork_pages where somebody besides the parent row holds its begun page: another row, or a
prefix cache that is counted in refs alone.  The new rows append into begun pages, so none
of them may be handed one that others still read."""
from __future__ import annotations

import random

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import D, F8, PAGE
from tests.test_gpu_pages import Pool, full, i32, pages_of, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


class Held(Pool):
    """alike: (a, b): row b is made the same as row a, page for page; extra: pages (row,
    entry) that a holder of no row keeps too."""

    def __init__(self, lens, S, NB, seed, alike=(), extra=(), **kw):
        super().__init__(lens, S, NB, seed, **kw)
        for a, b in alike:
            for p in self.rows[b]:
                self.refs[p] -= 1
            self.rows[b], self.lens[b] = list(self.rows[a]), self.lens[a]
            for p in self.rows[b]:
                self.refs[p] += 1
        for b, e in extra:
            self.refs[self.rows[b][e]] += 1
        self.table = full(self.rows, S).cuda()

    def fork(self, parents, grow):
        free = [p for p in range(self.NB) if self.refs[p] == 0]
        refs, rows, lens, copies, taken = list(self.refs), [], [], [], set()
        for p, g in zip(parents, grow):
            n = self.lens[p] if p >= 0 else 0
            row = list(self.rows[p]) if p >= 0 else []
            copy = (-1, -1, 0)
            if n % PAGE and (p in taken or self.refs[row[-1]] > 1):
                copy = (row[-1], free[0], n % PAGE)
                row[-1] = free.pop(0)
            taken.add(p)
            while len(row) < pages_of(n + g):
                row.append(free.pop(0))
            rows.append(row)
            lens.append(n + g)
            copies.append(copy)
        for step, every in ((-1, self.rows), (1, rows)):
            for row in every:
                for p in row:
                    refs[p] += step
        return rows, lens, refs, copies


CASES = [
    # lens, alike, extra, parents, grow
    ([5], [], [(0, 0)], [0], [1]),                           # a cache keeps the one begun page
    ([300], [], [(0, 2)], [0, 0, 0], [1, 1, 0]),
    ([300], [], [(0, 0), (0, 1)], [0, 0], [1, 1]),           # only full pages: the first child goes on
    ([300, 300], [(0, 1)], [], [0, 1], [1, 1]),              # two rows alike, both go on
    ([300, 300], [(0, 1)], [], [1], [1]),                    # one of them leaves
    ([300, 300], [(0, 1)], [], [1, 1, 0], [0, 90, 300]),
    ([300, 300], [(0, 1)], [(0, 2)], [-1, 0], [7, 1]),
    ([256, 256], [(0, 1)], [(1, 1)], [0, 1, 1], [1, 0, 5]),  # no page is begun
    ([200, 130, 200], [(0, 2)], [(1, 1)], [], []),           # all leave
    ([1 + 13 * k for k in range(64)], [(k, k + 1) for k in range(0, 64, 4)],
     [(k, -1) for k in range(2, 64, 5)], [(k * k + 1) % 64 for k in range(90)],
     [k % 140 for k in range(90)]),
]


@pytest.mark.parametrize("lens,alike,extra,parents,grow", CASES)
def test_begun_pages_of_other_holders(lens, alike, extra, parents, grow):
    x = Held(lens, 9, 900, 21, alike, extra, kept=2)
    rows, want_lens, refs, copies = x.fork(parents, grow)
    want = x.copied(copies)
    t, n, r, c = msa.fork_pages(*x.gpu()[:2], i32(parents), x.gpu()[2], x.caches, grow=i32(grow))
    same(t, full(rows, 9))
    same(n, want_lens)
    same(r, refs)
    same(c, copies)
    for a, b in zip(x.caches, want):
        assert torch.equal(a, b)
    # no begun page of a new row has another holder
    for row, m in zip(rows, want_lens):
        assert m % PAGE == 0 or int(r[row[-1]]) == 1
    assert msa.get_error() == 0


def test_rows_at_random():
    r = random.Random(5)
    for seed in range(6):
        n = r.choice([3, 40, 1500])
        lens = [r.choice([0, 1, 127, 128, 200, 256, 300]) for _ in range(n)]
        heads = [b for b in range(n) if lens[b]]
        x = Held(lens, 4, 8 * n + 40, 30 + seed,
                 [(a, b) for a, b in zip(heads[::3], heads[1::3])],
                 [(b, -1) for b in heads if r.random() < 0.2], Hkv=1)
        m = r.choice([1, n, 2 * n])
        parents = [r.randrange(-1, n) for _ in range(m)]
        grow = [r.choice([0, 1, 60, 128]) for _ in range(m)]
        rows, want_n, want_r, want_c = x.fork(parents, grow)
        t, lens_out, refs, copies = msa.fork_pages(*x.gpu()[:2], i32(parents), x.gpu()[2],
                                                   grow=i32(grow))
        same(t, full(rows, 4))
        same(lens_out, want_n)
        same(refs, want_r)
        same(copies, [list(c) for c in want_c])
    assert msa.get_error() == 0


def test_the_copies_need_pages():
    """Room for the growth but not for the copy that the other holder asks for."""
    x = Held([100], 2, 2, 22, extra=[(0, 0)])
    t, n, r, c = msa.fork_pages(*x.gpu()[:2], i32([0, 0]), x.gpu()[2], x.caches, grow=i32([1, 1]))
    assert msa.get_error() == _native.ERR_NO_PAGES
    same(t, [[-1, -1]] * 2)
    same(n, [0, 0])
    same(r, x.refs)
    same(c, [(-1, -1, 0)] * 2)


def test_appends_leave_a_kept_page_alone():
    """A prefix cache keeps a begun page on page scales; the row goes on with keys so large
    that the append requantises what its page holds."""
    x = Held([40], 2, 6, 23, extra=[(0, 0)], Hkv=1)
    page = x.rows[0][0]
    kv = (torch.randn(x.caches[0].shape, device="cuda") * 50).to(F8).view(torch.uint8)
    sc = torch.full((6, 1, 2), 2.0 ** -9, device="cuda")
    kept, kept_sc = kv[page].clone(), sc[page].clone()
    t, n, _, c = msa.fork_pages(*x.gpu()[:2], i32([0]), x.gpu()[2], [kv, sc], grow=i32([1]))
    own = int(t[0, 0])
    assert c.tolist() == [[page, own, 40]] and own != page
    assert torch.equal(kv[own, :, :40], kept[:, :40]) and torch.equal(sc[own], kept_sc)
    k = torch.full((1, 1, D), 500.0, device="cuda", dtype=torch.bfloat16)
    msa.append_kv(k, k, kv, t, n, 1, kv_scales=sc)
    assert float(sc[own].min()) > 2.0 ** -9            # the scale grew
    assert torch.equal(kv[page], kept) and torch.equal(sc[page], kept_sc)
    assert msa.get_error() == 0
