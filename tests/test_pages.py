"""Copying, forking, freeing and compacting cache pages: against a plain model, and their refusals."""
import ctypes
import random

import pytest
import torch

from memory_bound_decode_qk_gb300 import _build, edge_ops

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, UNSUP, CUDA, VALUE = range(9)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return edge_ops.lib()


# ---------------------------------------------------------------- refusals (no GPU)

C0, C1, TAB, TAB2, LENS, REFS, REFS2, A, B, ST, PAIRS, WS = (0x10000000 * i for i in range(1, 13))


def ptrs(v):
    return None if v is None else (ctypes.c_void_p * max(1, len(v)))(*v)


def copy(L, caches=(C0, C1), bytes=4096, pages=64, src=A, dst=B, n=4):
    return L.edge_pages_copy(ptrs(caches), 2 if caches is None else len(caches), bytes, pages, src, dst, n, None)


def free(L, tab=TAB, rows=8, width=4, lens=LENS, refs=REFS, pages=64, seqs=A, n=4):
    return L.edge_pages_free(tab, rows, width, lens, refs, pages, seqs, n, None)


def fork(L, caches=(C0, C1), bytes=4096, pages=64, ps=16, tab=TAB, rows=8, width=4, lens=LENS, refs=REFS, par=A, chi=B,
         n=4, st=ST, pairs=PAIRS):
    return L.edge_pages_fork(ptrs(caches), 2 if caches is None else len(caches), bytes, pages, ps, tab, rows, width, lens,
                             refs, par, chi, n, st, pairs, None)


def compact(L, caches=(C0, C1), bytes=4096, pages=64, out=TAB2, tab=TAB, rows=8, width=4, ro=REFS2, refs=REFS, ws=WS,
            wb=1 << 20):
    return L.edge_pages_compact(ptrs(caches), 2 if caches is None else len(caches), bytes, pages, out, tab, rows, width,
                                ro, refs, ws, wb, None)


@pytest.mark.parametrize("call,status", [
    (lambda L: copy(L, caches=None), NULL), (lambda L: copy(L, caches=(C0, None)), NULL),
    (lambda L: copy(L, src=None), NULL), (lambda L: copy(L, dst=None), NULL),
    (lambda L: copy(L, n=-1), SHAPE), (lambda L: copy(L, bytes=0), SHAPE), (lambda L: copy(L, pages=-1), SHAPE),
    (lambda L: copy(L, src=A + 2), ALIGN), (lambda L: copy(L, dst=B + 1), ALIGN),
    (lambda L: copy(L, caches=(C0, C0)), ALIAS), (lambda L: copy(L, caches=(C0, C0 + 4096)), ALIAS),
    (lambda L: copy(L, src=C0 + 64), ALIAS), (lambda L: copy(L, dst=C1), ALIAS),
    (lambda L: copy(L, n=65537), UNSUP), (lambda L: copy(L, bytes=2 ** 31), UNSUP), (lambda L: copy(L, bytes=2 ** 30, n=2 ** 16), UNSUP),
    (lambda L: free(L, tab=None), NULL), (lambda L: free(L, lens=None), NULL), (lambda L: free(L, refs=None), NULL),
    (lambda L: free(L, seqs=None), NULL), (lambda L: free(L, rows=-1), SHAPE), (lambda L: free(L, n=-1), SHAPE),
    (lambda L: free(L, width=-1), SHAPE), (lambda L: free(L, pages=-1), SHAPE),
    (lambda L: free(L, tab=TAB + 2), ALIGN), (lambda L: free(L, refs=REFS + 1), ALIGN), (lambda L: free(L, seqs=A + 2), ALIGN),
    (lambda L: free(L, lens=TAB + 16), ALIAS), (lambda L: free(L, refs=LENS), ALIAS), (lambda L: free(L, seqs=LENS + 4), ALIAS),
    (lambda L: fork(L, caches=None), NULL), (lambda L: fork(L, par=None), NULL), (lambda L: fork(L, chi=None), NULL),
    (lambda L: fork(L, st=None), NULL), (lambda L: fork(L, pairs=None), NULL), (lambda L: fork(L, tab=None), NULL),
    (lambda L: fork(L, lens=None), NULL), (lambda L: fork(L, refs=None), NULL), (lambda L: fork(L, ps=0), SHAPE),
    (lambda L: fork(L, n=-1), SHAPE), (lambda L: fork(L, n=8193), UNSUP), (lambda L: fork(L, ps=2 ** 29), UNSUP),
    (lambda L: fork(L, st=ST + 2), ALIGN), (lambda L: fork(L, st=A), ALIAS), (lambda L: fork(L, pairs=B - 16), ALIAS),
    (lambda L: fork(L, refs=C1 + 8), ALIAS), (lambda L: fork(L, chi=LENS), ALIAS),
    (lambda L: compact(L, caches=None), NULL), (lambda L: compact(L, refs=None), NULL), (lambda L: compact(L, ro=None), NULL),
    (lambda L: compact(L, tab=None), NULL), (lambda L: compact(L, out=None), NULL), (lambda L: compact(L, ws=None), NULL),
    (lambda L: compact(L, rows=-1), SHAPE), (lambda L: compact(L, wb=100), SHAPE), (lambda L: compact(L, wb=-1), SHAPE),
    (lambda L: compact(L, ws=WS + 4), ALIGN), (lambda L: compact(L, out=TAB + 4), ALIAS), (lambda L: compact(L, ro=REFS + 8), ALIAS),
    (lambda L: compact(L, out=REFS), ALIAS), (lambda L: compact(L, ws=C0), ALIAS), (lambda L: compact(L, ro=C1), ALIAS),
])
def test_refusals(L, call, status):
    assert call(L) == status


def test_nothing_to_do_launches_nothing(L):
    assert copy(L, n=0) == OK and copy(L, caches=()) == OK and copy(L, pages=0) == OK
    assert free(L, n=0) == OK and free(L, rows=0) == OK
    assert fork(L, n=0) == OK
    assert compact(L, pages=0) == OK
    assert L.edge_pages_compact_workspace(-1) == -1 and L.edge_pages_compact_workspace(64) >= 64 * 4
    assert L.edge_last_cuda_error() == 0


def test_page_caches_checks():
    with pytest.raises(ValueError, match="CUDA"):
        edge_ops.PageCaches([torch.zeros(32, 2, 8)], 16)
    with pytest.raises(ValueError, match="whole pages"):
        edge_ops.PageCaches([torch.zeros(33, 2, 8)], 16)
    with pytest.raises(ValueError):
        edge_ops.PageCaches([], 16)


# ---------------------------------------------------------------- a plain model

class Model:
    """Block table, lengths, counts and the pages' contents as plain lists; the operations one after the other."""

    def __init__(self, table, lens, refs, data, page):
        self.table, self.lens, self.refs = [list(r) for r in table], list(lens), list(refs)
        self.data, self.page = list(data), page  # data[p]: any value that stands for page p's bytes
        self.pages = len(self.refs)

    def held(self, row):
        return [p for p in self.table[row] if 0 <= p < self.pages]

    def copy(self, src, dst):
        pairs = [(s, d) for s, d in zip(src, dst) if 0 <= s < self.pages and 0 <= d < self.pages and s != d]
        old = list(self.data)
        targets = {d for _, d in pairs}
        for i, (s, d) in enumerate(pairs):
            if s not in targets and all(e != d for _, e in pairs[i + 1:]):
                self.data[d] = old[s]

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for p in self.held(r):
                    self.refs[p] -= 1
                self.table[r] = [-1] * len(self.table[r])
                self.lens[r] = 0

    def fork(self, parents, children):
        status, pairs, taken = [], [], set()
        rows, width = len(self.table), len(self.table[0])
        empty = [not self.held(r) and self.lens[r] == 0 for r in range(rows)]
        for i, (a, c) in enumerate(zip(parents, children)):
            if not (0 <= a < rows and 0 <= c < rows) or c in parents or c in children[:i] or not empty[c]:
                status.append(2)
                pairs.append((-1, -1))
                continue
            n = max(0, min(self.lens[a], width * self.page))
            full, part = divmod(n, self.page)
            last = self.table[a][full] if part else -1
            pair = (-1, -1)
            if 0 <= last < self.pages:
                new = next((p for p in range(self.pages) if self.refs[p] <= 0 and p not in taken), None)
                if new is None:
                    status.append(1)
                    pairs.append(pair)
                    continue
                taken.add(new)
                pair = (last, new)
            row = self.table[a][:full] + [pair[1]] + [-1] * width
            self.table[c] = row[:width]
            for p in self.table[a][:full]:
                if 0 <= p < self.pages:
                    self.refs[p] += 1
            self.lens[c] = n
            status.append(0)
            pairs.append(pair)
        for s, d in pairs:
            if s >= 0:
                self.refs[d] = 1
                self.data[d] = self.data[s]
        return status, pairs

    def compact(self):
        live = [p for p in range(self.pages) if self.refs[p] > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        new = {p: p for p in live}
        new.update(zip([p for p in live if p >= n], holes))
        refs = [0] * self.pages
        for p, q in new.items():
            refs[q] = self.refs[p]
            self.data[q] = self.data[p]
        self.refs = refs
        self.table = [[new.get(p, -1) if 0 <= p < self.pages else p for p in r] for r in self.table]
        return [new.get(p, -1) for p in range(self.pages)]


gpu = pytest.mark.gpu


class World:
    """A pool with its model: page p of cache c is filled with values that name both."""

    def __init__(self, pages, page, slot, rows, width, caches=3, dtype=torch.bfloat16, shift=0, seed=0):
        r = random.Random(seed)
        order = list(range(pages))
        r.shuffle(order)
        table, lens = [], []
        for _ in range(rows):
            n = r.randrange(0, width * page + 1) if r.random() < 0.8 else 0
            need = -(-n // page)
            if need > len(order):
                n = need = 0
            lens.append(n)
            table.append([order.pop() for _ in range(need)] + [-1] * (width - need))
        refs = [0] * pages
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        self.m = Model(table, lens, refs, range(pages), page)
        g = torch.Generator().manual_seed(seed)
        size = torch.empty((), dtype=dtype).element_size()
        self.start = [torch.randint(0, 256, (pages, page * slot * size), generator=g, dtype=torch.uint8) for _ in range(caches)]
        self.raw, views = [], []
        for s in self.start:
            flat = torch.empty(s.numel() + 64 + shift * size, dtype=torch.uint8, device="cuda").fill_(0xA5)
            self.raw.append(flat)
            v = flat[32 + shift * size:32 + shift * size + s.numel()]
            v.copy_(s.flatten())
            views.append(v.view(dtype).view(pages * page, slot))
        self.shift = shift * size
        self.caches = edge_ops.PageCaches(views, page)
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda").view(rows, width)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.refs = torch.tensor(refs, dtype=torch.int32, device="cuda")

    def check(self):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.m.table and self.lens.tolist() == self.m.lens
        assert self.refs.tolist() == self.m.refs
        for s, raw in zip(self.start, self.raw):
            want = torch.full_like(raw.cpu(), 0xA5)
            want[32 + self.shift:32 + self.shift + s.numel()] = s[torch.tensor(self.m.data, dtype=torch.long)].flatten()
            assert torch.equal(raw.cpu(), want)


def dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


SHAPES = [dict(pages=40, page=16, slot=64, rows=6, width=5), dict(pages=23, page=13, slot=5, rows=4, width=4),
          dict(pages=500, page=1, slot=256, rows=30, width=20), dict(pages=64, page=16, slot=2048, rows=8, width=6, caches=1),
          dict(pages=30, page=4, slot=33, rows=5, width=5, dtype=torch.float32, caches=2),
          dict(pages=40, page=16, slot=64, rows=6, width=5, shift=1), dict(pages=40, page=8, slot=64, rows=6, width=5, caches=131),
          dict(pages=9000, page=2, slot=8, rows=200, width=30)]


@gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_copy(i):
    w = World(**SHAPES[i], seed=i)
    r = random.Random(i)
    order = list(range(w.m.pages))
    r.shuffle(order)
    n = len(order) // 3
    src, dst = order[:n], order[n:2 * n]
    edge_ops.pages_copy(w.caches, dev(src), dev(dst))
    w.m.copy(src, dst)
    w.check()
    # one source for several, pages outside the pool, a page onto itself, pairs that meet
    src = [order[0], order[0], -1, order[1], w.m.pages, order[2], order[3], order[4], order[5], order[0]]
    dst = [order[6], order[7], order[8], 2 ** 31 - 1, order[9], order[2], order[10], order[10], order[3], order[1]]
    edge_ops.pages_copy(w.caches, dev(src), dev(dst))
    w.m.copy(src, dst)
    w.check()


@gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_free(i):
    w = World(**SHAPES[i], seed=10 + i)
    rows = [0, 2, 2, -1, len(w.m.table), 1]
    edge_ops.pages_free(w.table, w.lens, w.refs, dev(rows))
    w.m.free(rows)
    w.check()


@gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_fork(i):
    w = World(**SHAPES[i], seed=20 + i)
    rows = len(w.m.table)
    drop = list(range(1, rows, 2))
    edge_ops.pages_free(w.table, w.lens, w.refs, dev(drop))
    w.m.free(drop)
    r = random.Random(i)
    keep = list(range(0, rows, 2))
    parents = [r.choice(keep) for _ in drop] + [0, rows, -1, 0, 0]
    children = drop + [0, drop[0], drop[0], keep[-1], drop[0]]   # itself, strangers, one that is in use, one that is named
    pairs = torch.full((len(parents), 2), 7, dtype=torch.int32, device="cuda")
    status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev(parents), dev(children), pairs=pairs)
    want, moved = w.m.fork(parents, children)
    w.check()
    assert status.tolist() == want and [tuple(p) for p in pairs.tolist()] == moved
    # and again: the forks' children hold pages now
    status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev(parents), dev(children))
    assert status.tolist() == w.m.fork(parents, children)[0]
    w.check()


@gpu
def test_fork_without_free_pages():
    w = World(pages=8, page=4, slot=16, rows=1, width=6, seed=1)
    # one sequence of 3 full pages and a part, every page but one taken
    w.m.table = [[5, 2, 7, 1, -1, -1]] + [[-1] * 6 for _ in range(4)]
    w.m.lens, w.m.refs = [14, 0, 0, 0, 0], [9, 1, 1, 9, 0, 1, 9, 1]
    w.table, w.lens, w.refs = dev(w.m.table), dev(w.m.lens), dev(w.m.refs)
    for _ in range(2):
        status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev([0, 0, 0, 0]), dev([1, 2, 3, 4]))
        assert status.tolist() == w.m.fork([0] * 4, [1, 2, 3, 4])[0]
        w.check()
    # a parent that ends on a page's border needs none
    w.lens[0] = w.m.lens[0] = 12
    status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev([0, 0]), dev([2, 3]))
    assert status.tolist() == w.m.fork([0, 0], [2, 3])[0] == [0, 0]
    w.check()


@gpu
def test_fork_of_odd_rows():
    # lengths beyond the row or negative, entries outside the pool
    w = World(pages=12, page=4, slot=16, rows=1, width=3, seed=2)
    w.m.table = [[0, 5, 3], [99, -7, 4], [-1, -1, -1], [-1, 12, -3], [-1, -1, -1], [-1, -1, -1]]
    w.m.lens, w.m.refs = [10 ** 9, 6, 0, 0, 0, -3], [1, 0, 0, 1, 1, 1, 0, 0, 0, 0, 0, 0]
    w.table, w.lens, w.refs = dev(w.m.table), dev(w.m.lens), dev(w.m.refs)
    status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev([0, 1, 5]), dev([2, 3, 4]))
    assert status.tolist() == w.m.fork([0, 1, 5], [2, 3, 4])[0]
    w.check()


@gpu
def test_many_forks_at_once():
    w = World(pages=6000, page=4, slot=8, rows=2, width=4, caches=2, seed=3)
    rows = 3001
    w.m.table = [[3, 17, 8, -1]] + [[-1] * 4 for _ in range(rows - 1)]
    w.m.lens, w.m.refs = [11] + [0] * (rows - 1), [0] * 6000
    for p in (3, 17, 8):
        w.m.refs[p] = 1
    w.table, w.lens, w.refs = dev(w.m.table), dev(w.m.lens), dev(w.m.refs)
    parents, children = [0] * (rows - 1), list(range(rows - 1, 0, -1))
    status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev(parents), dev(children))
    assert status.tolist() == [0] * (rows - 1)
    w.m.fork(parents, children)
    w.check()


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_compact(i, in_place):
    w = World(**SHAPES[i], seed=30 + i)
    drop = list(range(0, len(w.m.table), 3))
    edge_ops.pages_free(w.table, w.lens, w.refs, dev(drop))
    w.m.free(drop)
    w.table[0, -1] = w.m.table[0][-1] = w.m.pages + 3          # no page: stays
    free = next(p for p in range(w.m.pages) if w.m.refs[p] == 0)
    w.table[0, 0] = w.m.table[0][0] = free                     # a free page: becomes -1
    if in_place:
        new = edge_ops.pages_compact(w.caches, w.table, w.refs)
        want = w.m.compact()
    else:
        before = w.table.clone(), w.refs.clone()
        out = torch.full_like(w.table, 77), torch.full_like(w.refs, 77)
        new = edge_ops.pages_compact(w.caches, w.table, w.refs, table_out=out[0], refs_out=out[1],
                                     workspace=edge_ops.pages_compact_workspace(w.refs).fill_(0x5A))
        want = w.m.compact()
        assert torch.equal(w.table, before[0]) and torch.equal(w.refs, before[1])
        w.table, w.refs = out
    w.check()
    assert new.tolist() == want
    # a compact pool stays as it is
    edge_ops.pages_compact(w.caches, w.table, w.refs)
    assert w.m.compact() == [p if p < sum(x > 0 for x in w.m.refs) else -1 for p in range(w.m.pages)]
    w.check()


@gpu
def test_full_and_empty_pools():
    for refs in ([0] * 20, [1] * 20):
        w = World(pages=20, page=4, slot=16, rows=2, width=2, seed=4)
        w.m.table, w.m.refs = [[-1, -1], [-1, -1]], list(refs)
        w.table, w.refs = dev(w.m.table), dev(refs)
        w.m.lens = [0, 0]
        w.lens = dev([0, 0])
        assert edge_ops.pages_compact(w.caches, w.table, w.refs).tolist() == w.m.compact()
        w.check()


@gpu
def test_random_histories():
    r = random.Random(5)
    w = World(pages=120, page=8, slot=24, rows=14, width=8, caches=2, seed=6)
    for _ in range(40):
        what = r.randrange(3)
        if what == 0:
            rows = [r.randrange(14) for _ in range(r.randrange(1, 5))]
            edge_ops.pages_free(w.table, w.lens, w.refs, dev(rows))
            w.m.free(rows)
        elif what == 1:
            par, chi = ([r.randrange(14) for _ in range(6)] for _ in range(2))
            status = edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, dev(par), dev(chi))
            assert status.tolist() == w.m.fork(par, chi)[0]
        else:
            edge_ops.pages_compact(w.caches, w.table, w.refs)
            w.m.compact()
        w.check()


@gpu
def test_on_another_stream_and_in_a_graph():
    w = World(pages=60, page=8, slot=64, rows=8, width=4, seed=8)
    drop, keep = [1, 3, 5, 7], [0, 2, 4, 6]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    edge_ops.pages_free(w.table, w.lens, w.refs, dev(drop), stream=side)
    side.synchronize()
    w.m.free(drop)
    w.check()
    a, b = dev(keep), dev(drop)
    pairs, status = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    ws = edge_ops.pages_compact_workspace(w.refs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, a, b, status=status, pairs=pairs)
        edge_ops.pages_compact(w.caches, w.table, w.refs, workspace=ws)
        edge_ops.pages_free(w.table, w.lens, w.refs, b)
    for _ in range(3):
        graph.replay()
        assert status.tolist() == w.m.fork(keep, drop)[0]
        w.m.compact()
        w.m.free(drop)
        w.check()


@gpu
def test_binding_checks_its_tensors():
    w = World(pages=20, page=4, slot=16, rows=3, width=2, seed=9)
    i32 = dev([0, 1])
    with pytest.raises(TypeError):
        edge_ops.pages_copy(w.caches, i32.long(), i32)
    with pytest.raises(ValueError):
        edge_ops.pages_copy(w.caches, i32, i32[:1])
    with pytest.raises(ValueError):
        edge_ops.pages_copy(w.caches, i32.cpu(), i32)
    with pytest.raises(ValueError):
        edge_ops.pages_free(w.table, w.lens[:-1], w.refs, i32)
    with pytest.raises(ValueError):
        edge_ops.pages_free(w.table.t(), w.lens, w.refs, i32)
    with pytest.raises(ValueError):
        edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs[:-1], i32, i32)
    with pytest.raises(edge_ops.EdgeError):
        edge_ops.pages_fork(w.caches, w.table, w.lens, w.refs, i32, i32, status=i32)
    with pytest.raises(edge_ops.EdgeError):
        edge_ops.pages_compact(w.caches, w.table, w.refs, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        edge_ops.pages_compact(w.caches, w.table, w.refs, table_out=w.table[:1])
    w.check()
