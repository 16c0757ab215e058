"""The paged-cache calls on caches whose element and byte offsets pass 32 bits."""
import pytest
import torch

import paged_ref
from memory_bound_decode_qk_gb300 import edge_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,new,page", [(torch.float32, 3, 16), (torch.bfloat16, 1, 16), (torch.bfloat16, 9, 16),
                                         (torch.bfloat16, 90, 13), (torch.bfloat16, 90, 16)])
def test_attention_of_pages_behind_32_bits(dt, new, page):
    hq, hk, D, L = 8, 2, 128, 300
    slots = (2 ** 32 + 2 ** 20) // (hk * D) // page * page  # over 2^32 elements of 2 or 4 bytes
    count = -(-L // page)
    pages = slots // page
    table = torch.randperm(count, generator=torch.Generator().manual_seed(1)).int() + (pages - count)
    table[::3] -= pages - count  # some at the start of the pool
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.empty(slots, hk, D, dtype=dt, device="cuda") for _ in range(2))
    for p in table.tolist():
        for x in (k, v):
            x[p * page:(p + 1) * page] = torch.randn(page, hk, D, generator=g, device="cuda")
    q = torch.randn(new, hq, D, generator=g, device="cuda").to(dt)
    lens = torch.tensor([L], dtype=torch.int32)
    starts = torch.tensor([0, new], dtype=torch.int32)
    out = edge_ops.paged_attention(q, k, v, table.view(1, -1).cuda(), lens.cuda(), page_size=page, q_starts=starts.cuda())
    # the same keys in a small pool
    at = torch.cat([torch.arange(p * page, (p + 1) * page) for p in table.tolist()]).cuda()
    ref, tol, _, _ = paged_ref.attention(q, k[at], v[at], torch.arange(count, dtype=torch.int32).view(1, -1), lens, starts,
                                         page, D ** -0.5)
    paged_ref.check_rows(out, ref, tol, dt)


def test_page_moves_behind_32_bits():
    # 6 GB a cache: a copy from its end to its start, a fork into its last free page, and a compaction from there
    page_bytes, page = 64 * 8 * 128 * 2, 64
    pages = 6 * 2 ** 30 // page_bytes
    k = torch.zeros(pages * page, 8, 128, dtype=torch.bfloat16, device="cuda")
    caches = edge_ops.PageCaches([k], page)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    k[-page:] = torch.randn(page, 8, 128, device="cuda")
    last = k[-page:].clone()
    edge_ops.pages_copy(caches, i32([pages - 1]), i32([3]))
    assert torch.equal(k[3 * page:4 * page], last)
    # every page but the one before the last is taken: the fork's copy goes there
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 2] = 0
    table, lens = i32([[pages - 1], [-1]]), i32([5, 0])
    assert edge_ops.pages_fork(caches, table, lens, refs, i32([0]), i32([1])).tolist() == [0]
    assert table.tolist() == [[pages - 1], [pages - 2]] and torch.equal(k[-2 * page:-page], last)
    refs[:pages - 2] = 0
    edge_ops.pages_compact(caches, table, refs)
    assert table.tolist() == [[1], [0]] and int(refs.sum()) == 2
    assert torch.equal(k[:page], last) and torch.equal(k[page:2 * page], last)


def test_millions_of_empty_sequences():
    # one wide chunk between millions of sequences without tokens, which every CTA has to pass over
    B, G, D, n = 2 ** 22 + 5, 16, 64, 4_300_000
    at = B // 2
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(16, 1, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, G, D, generator=g, device="cuda", dtype=torch.float16).to(torch.bfloat16)
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    starts[at + 1:] = n
    lens = torch.full((B,), 11, dtype=torch.int32, device="cuda")
    out = edge_ops.paged_attention(q, k, v, torch.zeros(B, 1, dtype=torch.int32, device="cuda"), lens, page_size=16,
                                   q_starts=starts, causal=False)
    rows = torch.randperm(n, generator=torch.Generator().manual_seed(4))[:50].cuda()
    ref, tol, _, _ = paged_ref.attention(q[rows], k, v, torch.zeros(1, 1, dtype=torch.int32),
                                         torch.tensor([11], dtype=torch.int32), torch.tensor([0, 50]), 16, D ** -0.5,
                                         causal=False)
    paged_ref.check_rows(out[rows], ref, tol, torch.bfloat16)
    assert torch.isfinite(out.view(-1, D).sum(1, dtype=torch.float32)).all()
