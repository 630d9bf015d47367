"""GPU tests of the page pool (tv_pages_*) against its plain statement: every table, count,
list and copied byte has to be equal."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


class Both:
    """The pool on the GPU and its model, changed side by side."""

    def __init__(self, rows, max_pages, num_pages, page_size):
        self.m = sm.Pool(rows, max_pages, num_pages, page_size)
        self.upload()
        self.copies = torch.full((rows, 3), -9, dtype=torch.int32, device="cuda")
        self.moves = torch.full((num_pages, 3), -9, dtype=torch.int32, device="cuda")
        self.n_moves = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def upload(self):
        m = self.m
        self.table, self.n, self.ref = (torch.from_numpy(t.copy()).cuda()
                                        for t in (m.table, m.n, m.ref))
        self.pool = tv.make_page_pool(self.ref, self.table, self.n, m.ps)

    @staticmethod
    def dev(v):
        return torch.from_numpy(np.asarray(v, np.int32)).cuda()

    def same(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        self.status.zero_()
        assert np.array_equal(self.table.cpu().numpy(), self.m.table)
        assert np.array_equal(self.n.cpu().numpy(), self.m.n)
        assert np.array_equal(self.ref.cpu().numpy(), self.m.ref)

    def reserve(self, length, new_length, status=0):
        tv.pages_reserve(self.pool, self.dev(length), self.dev(new_length), self.copies,
                         status=self.status)
        none = np.tile(np.array([-1, -1, 0], np.int32), (len(self.m.n), 1))
        c = none if status == tv.TV_ERR_BOUNDS else self.m.reserve(length, new_length)
        assert (c is None) == (status == tv.TV_ERR_NO_PAGES)
        self.same(status)
        assert np.array_equal(self.copies.cpu().numpy(), none if c is None else c)
        return c

    def fork(self, src, length):
        tv.pages_fork(self.pool, self.dev(src), self.dev(length), status=self.status)
        self.m.fork(src, length)
        self.same()

    def release(self, keep):
        tv.pages_release(self.pool, self.dev(keep), status=self.status)
        self.m.release(keep)
        self.same()

    def compact(self):
        tv.pages_compact(self.pool, self.moves, self.n_moves, status=self.status)
        c = self.m.compact()
        self.same()
        assert int(self.n_moves.item()) == len(c)
        assert np.array_equal(self.moves.cpu().numpy()[:len(c)], c)
        return c


@pytest.mark.parametrize("rows,num,ps,seed", [(1, 3, 4, 0), (7, 90, 1, 1), (40, 700, 16, 2),
                                              (300, 9001, 64, 3)])
def test_random_life_of_a_pool(rows, num, ps, seed):
    r = np.random.default_rng(seed)
    most = max(2, 3 * num // (4 * rows))
    b = Both(rows, most, num, ps)
    length = np.zeros(rows, np.int64)
    for _ in range(12):
        new = np.minimum(length + r.integers(0, 3 * ps + 1, rows), most * ps)
        new[r.random(rows) < 0.2] = -1
        if b.m.ref.astype(bool).sum() + ((new - length).clip(0) // ps + 2).sum() < num:
            b.reserve(length, new)
            length = np.maximum(length, new)
        gone = r.random(rows) < 0.3
        cut = np.where(gone, np.where(r.random(rows) < 0.5, 0, length // 2), -1)
        b.release(cut)
        length = np.where(gone, cut, length)
        empty = np.flatnonzero(b.m.n == 0)
        full = np.flatnonzero(b.m.n > 0)
        src = np.full(rows, -1)
        if len(full):
            for e in empty:
                if r.random() < 0.7:
                    src[e] = r.choice(full)
                    length[e] = r.integers(0, length[src[e]] + 1)
        b.fork(src, length)
        if r.random() < 0.4:
            b.compact()
        b.m.check()


def test_every_holder_writes_and_one_keeps():
    b = Both(5, 8, 40, 16)
    b.reserve([0] * 5, [40, 0, 0, 0, 0])
    b.fork([-1, 0, 0, -1, 0], [0, 40, 33, 0, 40])
    c = b.reserve([40, 40, 33, 0, 40], [41, 48, 50, 0, 60])
    assert c[0, 0] == -1 and (c[[1, 2, 4], 0] >= 0).all() and c[:, 2].tolist() == [0, 8, 1, 0, 8]
    # not every holder writes: each writer moves off
    b.release([-1, 0, 0, -1, 0])
    b.fork([-1, 0, 0, -1, -1], [0, 41, 41, 0, 0])
    c = b.reserve([41, 41, 41, 0, 0], [42, 42, -1, 0, 0])
    assert (c[:2, 0] >= 0).all()
    # whole pages: fresh ones, nothing to copy
    b.release([0] * 5)
    b.reserve([0] * 5, [32, 0, 0, 0, 0])
    b.fork([-1, 0, -1, -1, -1], [0, 32, 0, 0, 0])
    assert (b.reserve([32, 32, 0, 0, 0], [33, 33, 0, 0, 0])[:, 2] == 0).all()
    # back inside a shared whole page
    c = b.reserve([32, 17, 0, 0, 0], [-1, 18, 0, 0, 0])
    assert c[1, 2] == 1


def test_pages_run_out_and_nothing_changes():
    b = Both(3, 10, 7, 4)
    b.reserve([0, 0, 0], [8, 8, 0])
    b.reserve([8, 8, 0], [16, 16, 0], status=tv.TV_ERR_NO_PAGES)
    b.reserve([8, 8, 0], [16, 12, 0])
    b.reserve([16, 12, 0], [17, 12, 0], status=tv.TV_ERR_NO_PAGES)
    b.release([0, -1, -1])
    b.reserve([0, 12, 0], [1, 28, 0], status=tv.TV_ERR_NO_PAGES)
    b.reserve([0, 12, 0], [0, 28, 0])


def test_more_pages_asked_for_than_32_bits_count():
    rows, most = 40, 1 << 26
    table = torch.empty((rows, most), dtype=torch.int32, device="cuda")
    n, ref = Both.dev([0] * rows), Both.dev([0] * 100)
    pool = tv.make_page_pool(ref, table, n, 16)
    copies = torch.zeros((rows, 3), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.pages_reserve(pool, Both.dev([0] * rows), Both.dev([1 << 30] * rows), copies, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == tv.TV_ERR_NO_PAGES
    assert int(n.sum()) == 0 and int(ref.sum()) == 0


@pytest.mark.parametrize("what", ["too_many", "length", "negative", "page", "low_page", "free",
                                  "n_pages"])
def test_reserve_refuses_bad_rows_whole(what):
    b = Both(4, 4, 30, 8)
    b.reserve([0] * 4, [8, 16, 9, 1])
    length, new = [8, 16, 9, 1], [9, 17, 12, 3]
    if what == "too_many":
        new[1] = 33
    elif what == "length":
        length[2], new[2] = 17, 18
    elif what == "negative":
        length[2], new[2] = -1, 2
    elif what == "n_pages":
        b.m.n[3] = 5
    else:
        b.m.table[2, 1] = {"page": 30, "low_page": -1, "free": 25}[what]
    b.upload()
    b.reserve(length, new, status=tv.TV_ERR_BOUNDS)


def test_fork_and_release_refuse_bad_rows():
    b = Both(6, 4, 30, 8)
    b.reserve([0] * 6, [24, 8, 0, 0, 0, 0])
    before = [t.clone() for t in (b.table, b.n, b.ref)]

    def refused(src, length):
        tv.pages_fork(b.pool, b.dev(src), b.dev(length), status=b.status)
        torch.cuda.synchronize()
        assert int(b.status.item()) == tv.TV_ERR_BOUNDS
        b.status.zero_()
        for t, e in zip((b.table, b.n, b.ref), before):
            assert torch.equal(t, e)

    refused([-1, 0, -1, -1, -1, -1], [0, 8, 0, 0, 0, 0])      # row 1 holds pages
    refused([-1, -1, 6, -1, -1, -1], [0, 0, 8, 0, 0, 0])      # no such source
    refused([-1, -1, 0, -1, -1, -1], [0, 0, 25, 0, 0, 0])     # more than the source holds
    refused([-1, -1, 0, -1, -1, -1], [0, 0, -1, 0, 0, 0])
    refused([-1, -1, 0, -1, -1, -1], [0, 0, 2 ** 31 - 1, 0, 0, 0])
    refused([-1, -1, 2, -1, -1, -1], [0, 0, 0, 0, 0, 0])      # its own source
    # a source that is forked into itself: that row fails, the other one works
    tv.pages_fork(b.pool, b.dev([-1, -1, 0, 2, -1, -1]), b.dev([0, 0, 8, 8, 0, 0]),
                  status=b.status)
    b.m.fork([-1, -1, 0, -1, -1, -1], [0, 0, 8, 0, 0, 0])
    b.same(tv.TV_ERR_BOUNDS)
    # a released entry that names nothing, or a free page
    b.m.table[0, 1], b.m.table[0, 2] = 77, 29
    b.upload()
    tv.pages_release(b.pool, b.dev([8, -1, -1, -1, -1, -1]), status=b.status)
    b.m.table[0, 1:3], b.m.n[0] = -1, 1
    b.same(tv.TV_ERR_BOUNDS)
    # a table that names no page: compaction leaves the entry
    b.m.table[1, 0], b.m.ref[:] = 99, 0
    b.m.ref[b.m.table[0, 0]] = 2
    b.upload()
    tv.pages_compact(b.pool, b.moves, b.n_moves, status=b.status)
    torch.cuda.synchronize()
    assert int(b.status.item()) == tv.TV_ERR_BOUNDS and int(b.table[1, 0]) == 99


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layers,DL,DR,ps", [(1, 8, 8, 1), (3, 64, 16, 16), (2, 512, 64, 64),
                                             (1, 24, 8, 37)])
def test_copies(dt, layers, DL, DR, ps):
    """Whole pages, first rows, skipped entries, strided rows with guard bands, a count."""
    r = np.random.default_rng(DL + ps)
    num = 41
    wide = [torch.randn((layers, num * ps, d + 16), device="cuda").to(dt) for d in (DL, DR)]
    c, k = wide[0][:, :, 8:8 + DL], wide[1][:, :, 8:8 + DR]
    perm = r.permutation(num)
    n = 20
    lst = np.stack([perm[:n], perm[n:2 * n], r.integers(0, ps + 1, n)], 1).astype(np.int32)
    lst[3, 0] = -1
    lst[5] = (-1, -1, 0)
    lst[6, 2] = ps
    for count in (None, 0, 11, 99):
        want = [t.float().cpu().numpy() for t in wide]
        for t, d in zip(want, (DL, DR)):
            sm.copy_pages(t[:, :, 8:8 + d], ps, lst if count is None else lst[:count])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tv.pages_copy(c, k, ps, torch.from_numpy(lst).cuda(), status=status,
                      count=None if count is None else Both.dev([count]))
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for t, e in zip(wide, want):
            assert np.array_equal(t.float().cpu().numpy(), e)


@pytest.mark.parametrize("entry", [(41, 0, 1), (0, 41, 1), (0, -1, 1), (0, 1, 17), (0, 1, -1),
                                   (2 ** 31 - 1, 0, 1)])
def test_copy_skips_entries_outside_the_cache(entry):
    x = torch.randn((41 * 16, 32), device="cuda")
    y = torch.randn((41 * 16, 8), device="cuda")
    want = (x.clone(), y.clone())
    want[0][7 * 16:7 * 16 + 3] = want[0][5 * 16:5 * 16 + 3]
    want[1][7 * 16:7 * 16 + 3] = want[1][5 * 16:5 * 16 + 3]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.pages_copy(x, y, 16, Both.dev([entry, (5, 7, 3)]), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == tv.TV_ERR_BOUNDS
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_cache_past_32_bit_offsets():
    """Rows behind element 2^31 of the array."""
    ps, DL = 64, 512
    num = (1 << 31) // (ps * DL) + 40
    x = torch.zeros((num * ps, DL), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((num * ps, 8), dtype=torch.bfloat16, device="cuda")
    x[(num - 1) * ps:] = torch.randn((ps, DL), device="cuda").bfloat16()
    tv.pages_copy(x, y, ps, Both.dev([(num - 1, num - 3, ps), (num - 2, 0, ps)]))
    torch.cuda.synchronize()
    assert torch.equal(x[(num - 3) * ps:(num - 2) * ps], x[(num - 1) * ps:])


def test_captured_step_replays():
    """Release, fork, reserve and copy in a graph: every replay gives the same tables."""
    b = Both(4, 6, 40, 16)
    b.reserve([0] * 4, [45, 0, 0, 0])
    x = torch.randn((2, 40 * 16, 16), device="cuda")
    y = torch.randn((2, 40 * 16, 8), device="cuda")
    keep, src = b.dev([-1, 0, 0, 0]), b.dev([-1, 0, 0, 0])
    length, new = b.dev([45] * 4), b.dev([53] * 4)

    def go():
        tv.pages_release(b.pool, keep, status=b.status)
        tv.pages_fork(b.pool, src, length, status=b.status)
        tv.pages_reserve(b.pool, length, new, b.copies, status=b.status)
        tv.pages_copy(x, y, 16, b.copies, status=b.status)

    go()
    torch.cuda.synchronize()
    first = [t.clone() for t in (b.table, b.n, b.ref, b.copies, x, y)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    for t, e in zip((b.table, b.n, b.ref, b.copies, x, y), first):
        assert torch.equal(t, e)
    b.m.fork([-1, 0, 0, 0], [0, 45, 45, 45])
    assert np.array_equal(b.m.reserve([45] * 4, [53] * 4), b.copies.cpu().numpy())
    b.same()


def test_capture_on_a_stream_given_explicitly_keeps_its_own_workspace():
    b = Both(3, 4, 20, 16)
    length, new = b.dev([0] * 3), b.dev([20, 0, 5])
    side = torch.cuda.Stream()
    tv.pages_reserve(b.pool, length, length, b.copies, stream=side)
    torch.cuda.synchronize()
    kept = dict(tv._ws_cache)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tv.pages_reserve(b.pool, length, new, b.copies, status=b.status,
                         stream=torch.cuda.current_stream())
    assert tv._ws_cache.keys() == kept.keys()
    g.replay()
    b.m.reserve([0] * 3, [20, 0, 5])
    b.same()
