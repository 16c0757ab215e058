"""The paged-cache operators together, as a decoding program runs them.

Two layers, a pool of pages common to both: prompts are written to the cache with rotary positions of three axes and
attended to, sequences are forked, grow apart by single tokens, are freed, and the pool is compacted.  Every step's
attention is held to the formula over the cache's own contents, gathered through the block table by plain indexing.
"""
import pytest
import torch

import paged_ref
from memory_bound_decode_qk_gb300 import edge_ops, synth

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, PAGES, ROWS, WIDTH, LAYERS = 8, 2, 128, 8, 96, 6, 12, 2
SECTIONS = (24, 20, 20)


class Program:
    def __init__(self, dtype, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        self.k = [torch.zeros(PAGES * PAGE, HK, D, dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.zeros_like(k) for k in self.k]
        self.caches = edge_ops.PageCaches(self.k + self.v, PAGE)
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        cos, sin = synth.rope_cache(1e6, D, 512)
        self.cos, self.sin = cos.cuda(), sin.cuda()
        w = 1.0 + 0.1 * torch.randn(2, LAYERS, D, generator=self.g)
        self.wq, self.wk = (x.to(dtype).cuda() for x in w)

    def grow(self, news):
        """Room for news[row] further tokens: the caller's own allocation, in plain indexing."""
        slots = []
        for row, n in news:
            a = int(self.lens[row])
            for j in range(a, a + n):
                if j % PAGE == 0:
                    page = int((self.refs <= 0).nonzero()[0])
                    self.refs[page] = 1
                    self.table[row, j // PAGE] = page
                slots.append(int(self.table[row, j // PAGE]) * PAGE + j % PAGE)
            self.lens[row] = a + n
        return torch.tensor(slots, device="cuda")

    def step(self, news):
        """New tokens of some rows through both layers; returns the layers' attention outputs."""
        slots = self.grow(news)
        rows = [r for r, _ in news]
        starts = [0]
        pos = []
        for r, n in news:
            starts.append(starts[-1] + n)
            end = int(self.lens[r])
            pos += range(end - n, end)
        p = torch.tensor(pos)
        positions = torch.stack([p, p // 3, p % 7]).cuda()
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        table, lens = self.table[rows].contiguous(), self.lens[rows].contiguous()
        outs = []
        for i in range(LAYERS):
            qkv = torch.randn(len(pos), (HQ + 2 * HK) * D, generator=self.g).to(self.dtype).cuda()
            q = edge_ops.qkv_rope_cache(qkv, HQ, HK, self.wq[i], self.wk[i], positions, self.cos, self.sin, slots,
                                        self.k[i], self.v[i], sections=SECTIONS, axis_order="cycled")
            one = all(n == 1 for _, n in news)
            out = edge_ops.paged_attention(q, self.k[i], self.v[i], table, lens, page_size=PAGE,
                                           q_starts=None if one else starts)
            ref, tol, _, _ = paged_ref.attention(q, self.k[i], self.v[i], table.cpu(), lens.cpu(), starts.cpu(), PAGE,
                                                 D ** -0.5)
            paged_ref.check_rows(out, ref, tol, self.dtype)
            outs.append(out)
        return outs

    def look(self, rows, seed):
        """Attention of fixed queries over some rows, which writes nothing."""
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(len(rows), HQ, D, generator=g).to(self.dtype).cuda()
        table, lens = self.table[rows].contiguous(), self.lens[rows].contiguous()
        return [edge_ops.paged_attention(q, k, v, table, lens, page_size=PAGE) for k, v in zip(self.k, self.v)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts_forks_steps_and_compaction(dtype):
    p = Program(dtype, 1)
    p.step([(0, 37), (1, 80), (2, 5)])          # prompts
    p.step([(0, 1), (1, 1), (2, 1)])            # a decode step
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = edge_ops.pages_fork(p.caches, p.table, p.lens, p.refs, i32(0, 0, 1), i32(3, 4, 5))
    assert status.tolist() == [0, 0, 0]
    # a fork sees what its parent sees, bit for bit
    a, b = p.look([0, 1], 3), p.look([3, 5], 3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # the forks grow apart: a token of one leaves the others as they were
    before = p.look([0, 3, 5], 4)
    p.step([(4, 1)])
    p.step([(4, 20), (1, 3)])
    assert all(torch.equal(x, y) for x, y in zip(before, p.look([0, 3, 5], 4)))
    # parents go, their shared pages stay with the forks
    edge_ops.pages_free(p.table, p.lens, p.refs, i32(0, 1))
    assert all(torch.equal(x[1:], y[1:]) for x, y in zip(before, p.look([2, 3, 5], 4)))
    want = p.look([2, 3, 4, 5], 5)
    used = int((p.refs > 0).sum())
    edge_ops.pages_compact(p.caches, p.table, p.refs)
    assert int(p.table.max()) < used and bool((p.refs[:used] > 0).all()) and bool((p.refs[used:] == 0).all())
    assert all(torch.equal(x, y) for x, y in zip(want, p.look([2, 3, 4, 5], 5)))
    # the pool serves on
    p.step([(0, 30), (3, 1), (5, 2)])
    edge_ops.pages_free(p.table, p.lens, p.refs, i32(0, 2, 3, 4, 5))
    assert bool((p.refs == 0).all()) and bool((p.table == -1).all())


def test_a_captured_step_serves_growing_sequences():
    # one decode step of both layers in a graph; between replays the host only moves positions, slots and lengths
    p = Program(torch.bfloat16, 7)
    p.step([(0, 20), (1, 33)])
    qkv = torch.randn(LAYERS, 2, (HQ + 2 * HK) * D, generator=p.g).to(p.dtype).cuda()
    positions, slots = torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    table, lens = torch.zeros(2, WIDTH, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    qs = [torch.empty(2, HQ, D, dtype=p.dtype, device="cuda") for _ in range(LAYERS)]
    outs = [torch.empty_like(q) for q in qs]
    ws = edge_ops.paged_attention_workspace(qs[0], p.k[0])

    def step():
        for i in range(LAYERS):
            edge_ops.qkv_rope_cache(qkv[i], HQ, HK, p.wq[i], p.wk[i], positions, p.cos, p.sin, slots, p.k[i], p.v[i],
                                    q_out=qs[i], sections=SECTIONS)
            edge_ops.paged_attention(qs[i], p.k[i], p.v[i], table, lens, page_size=PAGE, out=outs[i], workspace=ws)

    side = torch.cuda.Stream()
    slots.fill_(-1)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(10):
        slots.copy_(p.grow([(0, 1), (1, 1)]))
        positions.copy_((p.lens[:2].long() - 1).expand(3, 2))
        table.copy_(p.table[:2])
        lens.copy_(p.lens[:2])
        graph.replay()
        torch.cuda.synchronize()
        for i in range(LAYERS):
            ref, tol, _, _ = paged_ref.attention(qs[i], p.k[i], p.v[i], table.cpu(), lens.cpu(), None, PAGE, D ** -0.5)
            paged_ref.check_rows(outs[i], ref, tol, p.dtype)
