"""The cache's pages (fork_pages, compact_pages, copy_pages) against their meaning, page
by page on the host."""
from __future__ import annotations

import random

import pytest
import torch

import block_sparse_gqa_score_gb300 as msa
from block_sparse_gqa_score_gb300 import _native
from tests.page_cache import D, F8, GROUP, PAGE
from tests.prefill_ref import cu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    msa.get_error(clear=True)
    yield


def pages_of(n):
    return -(-n // PAGE)


def i32(x, shape=None):
    t = torch.tensor(x, dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


class Pool:
    """Rows on the host, and the pool's tensors on the GPU.  `shared`: rows of a request
    (neighbours) share that many leading pages."""

    def __init__(self, lens, S, NB, seed, shared=None, Hkv=2, kept=0):
        r = random.Random(seed)
        free = list(range(NB))
        r.shuffle(free)
        self.S, self.NB, self.lens = S, NB, list(lens)
        self.rows, self.refs = [], [0] * NB
        for b, n in enumerate(lens):
            sh = shared[b] if shared else 0
            row = list(self.rows[b - 1][:sh]) if sh else []
            while len(row) < pages_of(n):
                row.append(free.pop())
            self.rows.append(row)
            for p in row:
                self.refs[p] += 1
        for _ in range(kept):
            self.refs[free.pop()] += 1
        gen = torch.Generator(device="cuda").manual_seed(seed)
        junk = [[r.randrange(-9, 1 << 30) for _ in range(S)] for _ in lens]   # behind the rows
        self.table = i32([row + j[len(row):] for row, j in zip(self.rows, junk)], (len(lens), S))
        self.caches = [
            torch.randint(0, 256, (NB, Hkv, PAGE, 2 * D), dtype=torch.uint8, device="cuda", generator=gen),
            torch.rand((NB, Hkv, 2), device="cuda", generator=gen),
            torch.randint(0, 256, (NB, Hkv, PAGE, D), dtype=torch.uint8, device="cuda", generator=gen),
            torch.rand((NB, Hkv, 1), device="cuda", generator=gen)]

    def gpu(self):
        return self.table, i32(self.lens), i32(self.refs)

    def fork(self, parents, grow):
        """(rows, lens, refs, copies) of the next step."""
        free = [p for p in range(self.NB) if self.refs[p] == 0]
        refs, rows, lens, copies, taken = list(self.refs), [], [], [], set()
        for p, g in zip(parents, grow):
            n = self.lens[p] if p >= 0 else 0
            row = list(self.rows[p]) if p >= 0 else []
            copy = (-1, -1, 0)
            if n % PAGE and p in taken:
                copy = (row[-1], free[0], n % PAGE)
                row[-1] = free.pop(0)
            taken.add(p)
            while len(row) < pages_of(n + g):
                row.append(free.pop(0))
            rows.append(row)
            lens.append(n + g)
            copies.append(copy)
        for row in self.rows:
            for p in row:
                refs[p] -= 1
        for row in rows:
            for p in row:
                refs[p] += 1
        return rows, lens, refs, copies

    def copied(self, copies):
        out = [c.clone() for c in self.caches]
        for a, b, r in copies:
            if a < 0 or r == 0:
                continue
            for c in out:
                if c.dtype == torch.uint8:
                    c[b, :, :r] = c[a, :, :r]
                else:
                    c[b] = c[a]
        return out


def full(rows, S):
    return torch.tensor([r + [-1] * (S - len(r)) for r in rows], dtype=torch.int32).reshape(-1, S)


def same(got, want):
    assert torch.equal(got.cpu(), want if isinstance(want, torch.Tensor) else
                       torch.tensor(want, dtype=torch.int32).reshape(got.shape))


FORKS = [
    # lens, S, NB, shared, parents, grow
    ([1], 1, 2, None, [0], [0]),
    ([1], 2, 9, None, [0, 0, 0], [1, 127, 128]),
    ([128, 127, 129], 4, 30, None, [2, 1, 0, 1, 2, 2, -1, -1], [1, 1, 1, 2, 0, 300, 0, 200]),
    ([300, 300, 310], 4, 20, [0, 2, 2], [1, 1, 0], [1, 1, 1]),      # row 2 is freed
    ([500, 0, 256], 6, 40, None, [], []),                           # every row is freed
    ([500, 0, 256], 6, 40, None, [1, 1, -1], [0, 128, 0]),
    ([], 3, 10, None, [-1, -1], [5, 384]),
    ([900] * 8, 9, 200, [0] + [7] * 7, [7, 7, 7, 7, 0, 0, 3, 3], [4] * 8),
    ([1500 + 31 * k for k in range(200)], 70, 40000, None, [(k * k) % 200 for k in range(333)],
     [k % 300 for k in range(333)]),
]


@pytest.mark.parametrize("lens,S,NB,shared,parents,grow", FORKS)
def test_fork(lens, S, NB, shared, parents, grow):
    x = Pool(lens, S, NB, 5, shared, kept=1)
    rows, want_lens, refs, copies = x.fork(parents, grow)
    want = x.copied(copies)
    t, n, r, c = msa.fork_pages(*x.gpu()[:2], i32(parents), x.gpu()[2], x.caches,
                                grow=i32(grow))
    same(t, full(rows, S))
    same(n, want_lens)
    same(r, refs)
    same(c, copies)
    for a, b in zip(x.caches, want):
        assert torch.equal(a, b)
    assert msa.get_error() == 0


def test_fork_by_itself_and_copies_later():
    """Without caches nothing is moved; copy_pages moves it, for other layers, in any
    number of tensors."""
    x = Pool([200, 130], 4, 30, 6)
    parents, grow = [0, 0, 1, 1], [0] * 4
    _, _, _, copies = x.fork(parents, grow)
    before = [c.clone() for c in x.caches]
    layers = [c.clone() for _ in range(20) for c in x.caches]        # 80 tensors, two launches
    want = x.copied(copies)
    *_, c = msa.fork_pages(*x.gpu()[:2], i32(parents), x.gpu()[2])
    assert all(torch.equal(a, b) for a, b in zip(x.caches, before))
    msa.copy_pages(c, layers)
    for k, a in enumerate(layers):
        assert torch.equal(a, want[k % 4])
    assert msa.get_error() == 0


def test_fork_without_room_changes_nothing():
    x = Pool([200, 130], 4, 8, 7, kept=1)           # three pages are free
    before = [c.clone() for c in x.caches]
    parents, grow = i32([0, 0, 1, 1]), i32([60, 60, 0, 0])
    t, n, r, c = msa.fork_pages(*x.gpu()[:2], parents, x.gpu()[2], x.caches, grow=grow)
    assert msa.get_error() == _native.ERR_NO_PAGES
    same(t, torch.full((4, 4), -1, dtype=torch.int32))
    same(n, [0] * 4)
    same(r, x.refs)
    same(c, [(-1, -1, 0)] * 4)
    assert all(torch.equal(a, b) for a, b in zip(x.caches, before))
    # three pages are enough for this one
    rows, lens, refs, _ = x.fork([0, 0, 1, 1], [0, 0, 0, 127])
    t, n, r, _ = msa.fork_pages(*x.gpu()[:2], parents, x.gpu()[2], grow=i32([0, 0, 0, 127]))
    same(t, full(rows, 4))
    same(r, refs)
    assert msa.get_error() == 0


def test_fork_bad_inputs():
    x = Pool([200, 130, 300], 4, 40, 8)
    t0, n0, r0 = x.gpu()
    # a parent that is no row: an empty row, the others as if it were not there
    t, n, r, _ = msa.fork_pages(t0, n0, i32([0, 3, -2, 1, 2]), r0, grow=i32([0, 5, 5, 0, 0]))
    rows, lens, refs, _ = x.fork([0, -1, -1, 1, 2], [0, 0, 0, 0, 0])
    same(t, full(rows, 4))
    same(n, lens)
    same(r, refs)
    assert msa.get_error() == _native.ERR_ROW_RANGE
    # lengths and growth out of range
    n1 = n0.clone()
    n1[1] = 4 * PAGE + 1
    t, n, r, _ = msa.fork_pages(t0, n1, i32([0, 1, 2]), r0, grow=i32([-1, 3, 213]))
    same(n, [200, 3, 300])
    assert t[1, 1:].tolist() == [-1, -1, -1]
    assert msa.get_error() == _native.ERR_SEQ_RANGE
    # entries out of the pool, and a held page that is counted as free
    t1, r1 = t0.clone(), r0.clone()
    t1[0, 0] = 40
    t1[2, 2] = -5
    t, n, r, c = msa.fork_pages(t1, n0, i32([0, 0, 2, 2]), r0, x.caches)
    assert t[:, 0].tolist()[:2] == [-1, -1] and t[2].tolist()[2] == -1
    assert c.tolist()[3] == [-1, -1, 0]
    assert msa.get_error() == _native.ERR_PAGE_RANGE
    r1[x.rows[0][0]] = 0
    msa.fork_pages(t0, n0, i32([0, 0]), r1)
    assert msa.get_error() == _native.ERR_REFS


COMPACT = [
    # lens, S, NB, shared, kept
    ([1], 1, 1, None, 0),
    ([1], 1, 2, None, 0),
    ([300, 5, 0], 4, 9, None, 1),
    ([300, 310, 320], 4, 64, [0, 2, 2], 3),
    ([128 * 9], 9, 9, None, 0),                       # nothing to move
    ([], 2, 50, None, 7),
    ([700] * 40, 6, 700, None, 20),
    ([1500 + 31 * k for k in range(200)], 70, 40001, None, 1000),
]


@pytest.mark.parametrize("lens,S,NB,shared,kept", COMPACT)
def test_compact(lens, S, NB, shared, kept):
    x = Pool(lens, S, NB, 9, shared, kept=kept)
    used = [p for p in range(NB) if x.refs[p]]
    L = len(used)
    holes = [p for p in range(L) if not x.refs[p]]
    move = dict(zip([p for p in used if p >= L], holes))
    copies = [(a, b, PAGE) for a, b in move.items()]
    refs = list(x.refs)
    for a, b in move.items():
        refs[b], refs[a] = refs[a], 0
    want = x.copied(copies)
    t, r, c = msa.compact_pages(*x.gpu(), x.caches)
    same(t, full([[move.get(p, p) for p in row] for row in x.rows], S))
    same(r, refs)
    same(c, copies + [(-1, -1, 0)] * (NB // 2 - len(copies)))
    for a, b in zip(x.caches, want):
        assert torch.equal(a, b)
    assert msa.get_error() == 0


def test_compact_bad_entries():
    x = Pool([300, 400], 5, 40, 10)
    t0, n0, r0 = x.gpu()
    t0[0, 1] = 40
    r0[x.rows[1][2]] = 0
    t, r, _ = msa.compact_pages(t0, n0, r0)
    assert t[0, 1] == -1 and t[1, 2] == -1 and t[0, 0] >= 0 and t[1, 3] >= 0
    assert msa.get_error() == _native.ERR_PAGE_RANGE | _native.ERR_REFS
    n0[1] = -4
    t, _, _ = msa.compact_pages(x.table, n0, i32(x.refs))
    assert t[1].tolist() == [-1] * 5
    assert msa.get_error() & _native.ERR_SEQ_RANGE


def test_copy_bad_entries_are_skipped():
    x = Pool([300, 400], 5, 40, 11)
    c = [(1, 2, 128), (40, 3, 5), (3, -1, 5), (4, 40, 1), (5, 6, 129), (7, 8, -1), (9, 10, 0),
         (11, 12, 1), (-1, -1, 77), (13, 14, 127)]
    want = x.copied([c[0], c[7], c[9]])
    msa.copy_pages(i32(c), x.caches)
    for a, b in zip(x.caches, want):
        assert torch.equal(a, b)
    assert msa.get_error() == _native.ERR_PAGE_RANGE


def test_past_four_gigabytes():
    kv = torch.zeros((140000, 1, PAGE, 2 * D), dtype=torch.uint8, device="cuda")
    kv[139990] = 77
    kv[5, 0, 100:] = 3
    msa.copy_pages(i32([(139990, 5, 100), (139990, 139999, 128)]), [kv])
    assert bool((kv[5, 0, :100] == 77).all()) and bool((kv[5, 0, 100:] == 3).all())
    assert bool((kv[139999] == 77).all()) and int(kv.count_nonzero()) == (100 + 28 + 256) * 256


def test_captured_fork_then_step():
    """A step of beams captured as one graph: fork, append, dense decode; the same as the
    calls one by one on the host's plan."""
    Hkv, B = 1, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = Pool([200, 200, 255, 256], 4, 40, 12, Hkv=Hkv)
    kv = torch.randn(x.caches[0].shape, device="cuda", generator=gen).mul(50).to(F8).view(torch.uint8)
    t0, n0, r0 = x.gpu()
    parents = i32([0, 0, 1, 1])
    q = torch.randn((B, GROUP, D), device="cuda", generator=gen).to(torch.bfloat16)
    k, v = (torch.randn((B, Hkv, D), device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    grow = i32([1] * B)
    t, n, r, c = (torch.zeros_like(t0), torch.zeros_like(n0), torch.zeros_like(r0),
                  torch.zeros((B, 3), dtype=torch.int32, device="cuda"))
    out = torch.zeros_like(q)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def step(cache):
        msa.fork_pages(t0, n0, parents, r0, [cache], grow=grow, block_table_out=t, seq_lens_out=n,
                       refs_out=r, copies=c)
        msa.append_kv(k, v, cache, t, n, 1, 0.01, 0.01)
        msa.dense_decode(q, cache, t, n, 1, D ** -0.5, 0.01, 0.01, out=out, workspace=ws)

    warm = kv.clone()
    step(warm)
    g = torch.cuda.CUDAGraph()
    live = kv.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(live)
    live.copy_(kv)
    for p in ([0, 0, 1, 1], [3, 3, 3, 2], [2, 1, 0, 3]):
        parents.copy_(i32(p))
        live.copy_(kv)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        rows, lens, refs, copies = x.fork(p, [1] * B)
        same(t, full(rows, 4))
        same(r, refs)
        host = kv.clone()
        for a, b, m in copies:
            if a >= 0:
                host[b, :, :m] = host[a, :, :m]
        msa.append_kv(k, v, host, full(rows, 4).cuda(), i32(lens), 1, 0.01, 0.01)
        assert torch.equal(host, live)
        want = msa.dense_decode(q, host, full(rows, 4).cuda(), i32(lens), 1, D ** -0.5, 0.01, 0.01)
        assert torch.equal(out, want)
    assert msa.get_error() == 0


def test_prefill_of_new_rows_together():
    """What a serving step does: two requests leave, a prompt of a chunk comes and another
    goes on, the pages are moved together; then append, scores, lists, sparse and dense
    attention of the chunks, the same as in a cache of its own."""
    Hkv, sm = 2, D ** -0.5
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = Pool([700, 2300, 90], 40, 120, 13, Hkv=Hkv)
    kv = torch.randn(x.caches[0].shape, device="cuda", generator=gen).mul(50).to(F8).view(torch.uint8)
    sc = torch.exp2(torch.randint(-9, -6, (x.NB, Hkv, 2), device="cuda", generator=gen).float())
    plain_kv, plain_sc = kv.clone(), sc.clone()
    t0, n0, r0 = x.gpu()
    chunks = [300, 150]
    t, n, r, _ = msa.fork_pages(t0, n0, i32([1, -1]), r0, [kv, sc], grow=i32(chunks))
    t, r, _ = msa.compact_pages(t, n, r, [kv, sc])
    assert int((r != 0).sum()) == pages_of(2600) + 2 and bool((r[:pages_of(2600) + 2] > 0).all())
    T = sum(chunks)
    q, k, v = (torch.randn((T, h, D), device="cuda", generator=gen).to(torch.bfloat16)
               for h in (GROUP * Hkv, Hkv, Hkv))

    def run(cache, scales, table, lens):
        at = cu(chunks)
        msa.append_kv_prefill(k, v, cache, table, lens, at, kv_scales=scales)
        s = msa.score_prefill(q, cache, table, lens, at, sm, kv_scales=scales)
        lists = msa.topk_prefill(s, lens, at)
        sparse = msa.sparse_prefill(q, cache, table, lens, at, lists, sm, kv_scales=scales)
        also, fused = msa.sparse_prefill_select(q, cache, table, lens, at, s, sm, kv_scales=scales)
        assert torch.equal(also, lists) and torch.equal(fused, sparse)
        return s, lists, sparse, msa.dense_prefill(q, cache, table, lens, at, sm, kv_scales=scales)

    # a cache of its own: the row's pages as they were, then the spare ones
    spare = [p for p in range(x.NB) if x.refs[p] == 0]
    row = x.rows[1] + spare[:pages_of(2600) - len(x.rows[1])]
    own = full([row, spare[10:12]], 40).clamp(min=0).cuda()
    want = run(plain_kv, plain_sc, own, n)
    got = run(kv, sc, t, n)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert msa.get_error() == 0


def test_most_rows():
    """As many rows as a fork takes, on both sides."""
    n = 8192
    r = random.Random(16)
    x = Pool([r.choice([0, 1, 127, 128, 129, 200, 256]) for _ in range(n)], 3, 4 * n, 16, Hkv=1)
    parents = [r.randrange(-1, n) for _ in range(n)]
    grow = [r.choice([0, 1, 128]) for _ in range(n)]
    free = [p for p in range(x.NB) if x.refs[p] == 0]
    assert len(free) > 2 * n
    t0, n0, r0 = x.gpu()
    t, lens, refs, copies = msa.fork_pages(t0, n0, i32(parents), r0, grow=i32(grow))
    rows, want_n, want_r, want_c = x.fork(parents, grow)
    same(t, full(rows, 3))
    same(lens, want_n)
    same(refs, want_r)
    same(copies, [list(c) for c in want_c])
    with pytest.raises(msa.MSAError):
        msa.fork_pages(t0, n0, i32(parents + [0]), r0)
    assert msa.get_error() == 0


def test_overlapped_calls_keep_their_order():
    """With input overlap on, calls that read tables, lengths and caches right behind the
    calls on pages find what these wrote: tables and caches that are rewritten in turn."""
    B, S, Hkv, sm = 32, 40, 2, D ** -0.5
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = Pool([4700 + 3 * b for b in range(B)], S, 2 * B * S, 15, Hkv=Hkv)
    t0, n0, r0 = x.gpu()
    kv0 = torch.randn(x.caches[0].shape, device="cuda", generator=gen).mul(50).to(F8).view(torch.uint8)
    q = torch.randn((B, GROUP * Hkv, D), device="cuda", generator=gen).to(torch.bfloat16)
    orders = [i32([(a * b + 1) % B // k * k for b in range(B)]) for a, k in ((5, 1), (7, 4), (11, 2))]
    one = i32([1] * B)
    t = t0.clamp(0, x.NB - 1)
    n, r, co = n0.clone(), r0.clone(), torch.full((B, 3), -1, dtype=torch.int32, device="cuda")
    t2, r2 = t.clone(), r0.clone()
    moves = torch.full((x.NB // 2, 3), -1, dtype=torch.int32, device="cuda")
    moves[:, 2] = 0

    def run(sync):
        kv = kv0.clone()
        torch.cuda.synchronize()
        out = []
        for p in orders:
            for f in (lambda: msa.fork_pages(t0, n0, p, r0, [kv], grow=one, block_table_out=t,
                                             seq_lens_out=n, refs_out=r, copies=co),
                      lambda: out.append(msa.score(q, kv, t, n, 1, sm)),
                      lambda: msa.compact_pages(t, n, r, [kv], block_table_out=t2, refs_out=r2, copies=moves),
                      lambda: out.append(msa.dense_decode(q, kv, t2, n, 1, sm, 0.01, 0.01)),
                      lambda: out.append(msa.decode_step(q, kv, t2, n, 1, sm, 0.01, 0.01)[2])):
                f()
                if sync:
                    torch.cuda.synchronize()
            kv.copy_(kv0)
        torch.cuda.synchronize()
        return out

    want = run(True)
    was = msa.set_input_overlap(True)
    try:
        for _ in range(5):
            for a, b in zip(run(False), want):
                assert torch.equal(a, b)
    finally:
        msa.set_input_overlap(was)
    assert msa.get_error() == 0


def test_refusals():
    x = Pool([300, 5], 4, 20, 14)
    t0, n0, r0 = x.gpu()
    p = i32([0, 1])
    for kw in (dict(block_table=t0[0]), dict(seq_lens=n0[:1]), dict(refs=r0.long()),
               dict(parents=p.cpu()), dict(grow=i32([1])), dict(block_table_out=t0),
               dict(refs_out=r0), dict(seq_lens_out=n0), dict(copies=torch.zeros((2, 2), dtype=torch.int32, device="cuda")),
               dict(caches=[x.caches[0][:10]]), dict(caches=[x.caches[0].half()]),
               dict(caches=[x.caches[0][:, :, :64].contiguous()]), dict(caches=[x.caches[1].flatten(1)]),
               dict(caches=[x.caches[0].cpu()])):
        a = dict(block_table=t0, seq_lens=n0, parents=p, refs=r0)
        a.update(kw)
        with pytest.raises((ValueError, TypeError, msa.MSAError)):
            msa.fork_pages(**a)
        if "parents" not in kw and "grow" not in kw and "seq_lens_out" not in kw:
            a.pop("parents")
            with pytest.raises((ValueError, TypeError, msa.MSAError)):
                msa.compact_pages(**a)
    with pytest.raises(ValueError):
        msa.copy_pages(i32([1, 2, 3]), x.caches)
    with pytest.raises(TypeError):
        msa.copy_pages(torch.zeros((1, 3), device="cuda"), x.caches)
    assert msa.get_error() == 0
