"""Attention over a paged cache: against the formula in 64 bits, and its refusals.

The bounds are derived in paged_ref.py from the number formats alone.
"""
import math
import random

import pytest
import torch

import paged_ref
from memory_bound_decode_qk_gb300 import _build, edge_ops

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, UNSUP, CUDA, VALUE = range(9)
F32, F16, BF16, FP8 = 0, 1, 2, 3
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def L():
    _build.build()
    return edge_ops.lib()


# ---------------------------------------------------------------- refusals (no GPU)

OUT, LSE, Q, K, V, TAB, LENS, ST, WS = (0x10000000 * i for i in range(1, 10))


def call(L, out=OUT, out_dt=BF16, lse=LSE, q=Q, k=K, v=V, dt=BF16, T=4, hq=8, hk=2, D=128, slots=1024,
         page=16, tab=TAB, B=4, pages=8, lens=LENS, st=None, scale=0.1, causal=1, window=0, inv=1.0,
         ws=WS, n=1 << 30):
    return L.edge_paged_attention(out, out_dt, lse, q, k, v, dt, T, hq, hk, D, slots, page, tab, B, pages,
                                  lens, st, scale, causal, window, inv, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(tab=None), NULL), (dict(lens=None), NULL), (dict(ws=None), NULL),
    (dict(dt=FP8, out_dt=FP8), DTYPE), (dict(out_dt=F16), DTYPE), (dict(dt=9), DTYPE),
    (dict(T=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(hk=3), SHAPE), (dict(D=0), SHAPE),
    (dict(slots=-1), SHAPE), (dict(page=0), SHAPE), (dict(B=-1), SHAPE), (dict(pages=-1), SHAPE),
    (dict(T=5), SHAPE),                       # no q_starts: one token per sequence
    (dict(n=0), SHAPE), (dict(n=1000), SHAPE), (dict(n=-5), SHAPE),
    (dict(T=2 ** 62, hq=8, st=ST), SHAPE),
    (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=math.nan), VALUE),
    (dict(scale=math.inf), VALUE), (dict(causal=2), VALUE), (dict(window=-1), VALUE),
    (dict(causal=0, window=4), VALUE), (dict(out_dt=FP8, inv=0.0), VALUE),
    (dict(D=257), UNSUP), (dict(T=2 ** 28, st=ST), UNSUP), (dict(pages=2 ** 27), UNSUP),
    (dict(q=Q + 1), ALIGN), (dict(k=K + 1), ALIGN), (dict(out=OUT + 1), ALIGN), (dict(lse=LSE + 2), ALIGN),
    (dict(tab=TAB + 2), ALIGN), (dict(lens=LENS + 1), ALIGN), (dict(st=ST + 2), ALIGN), (dict(ws=WS + 8), ALIGN),
    (dict(out=Q), ALIAS), (dict(out=K + 2048), ALIAS), (dict(lse=OUT + 16), ALIAS), (dict(ws=OUT, n=1 << 24), ALIAS),
    (dict(ws=V, n=1 << 24), ALIAS), (dict(lse=LENS), ALIAS), (dict(out=TAB), ALIAS),
])
def test_refusals(L, kw, status):
    assert call(L, **kw) == status


def test_nothing_to_do_launches_nothing(L):
    assert call(L, T=0, B=0) == OK
    assert call(L, T=0, st=ST) == OK
    assert call(L, T=3, B=0, st=ST) == OK
    assert L.edge_last_cuda_error() == 0


def test_workspace_query(L):
    assert L.edge_paged_attention_workspace(BF16, 8, 2, 128) > 0
    for bad in ((FP8, 8, 2, 128), (BF16, 8, 3, 128), (BF16, 0, 1, 128), (BF16, 8, 2, 257), (BF16, 8, 2, 0)):
        assert L.edge_paged_attention_workspace(*bad) == -1


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    good = dict(q=z(2, 4, 64), k_cache=z(32, 2, 64), v_cache=z(32, 2, 64), block_table=z(2, 4, dtype=torch.int32),
                lens=z(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        edge_ops.paged_attention(**good, page_size=8)


# ---------------------------------------------------------------- GPU

gpu = pytest.mark.gpu


def make(dt, hq, hk, D, page, shape, seed=0, spare=3, sharp=1.0):
    """shape: [(keys, new tokens)].  Pages are scattered; everything that is no key of a sequence holds NaN."""
    g = torch.Generator().manual_seed(seed)
    t = TORCH[dt]
    need = [-(-max(L, 0) // page) for L, _ in shape]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = max(1, max(need)) + 1
    table = torch.full((len(shape), width), -1, dtype=torch.int32)
    k = torch.full((pages * page, hk, D), math.nan)
    v = k.clone()
    for b, (L, _) in enumerate(shape):
        for i in range(need[b]):
            p = order.pop()
            table[b, i] = p
            m = min(page, L - i * page)
            k[p * page:p * page + m] = torch.randn(m, hk, D, generator=g)
            v[p * page:p * page + m] = torch.randn(m, hk, D, generator=g)
    starts = [0]
    for _, n in shape:
        starts.append(starts[-1] + n)
    q = sharp * torch.randn(starts[-1], hq, D, generator=g)
    return dict(q=q.to(t), k=k.to(t), v=v.to(t), table=table, lens=torch.tensor([s[0] for s in shape], dtype=torch.int32),
                starts=torch.tensor(starts, dtype=torch.int32), page=page)


def run(c, *, starts=True, lse=True, fp8=False, inv=None, causal=True, window=0, scale=None, tail=0, **kw):
    """The call, with `tail` rows behind the last sequence, its outputs filled with a pattern first."""
    d = {n: x.cuda() for n, x in c.items() if n != "page"}
    q = torch.cat([d["q"], torch.full_like(d["q"][:1], math.nan).expand(tail, -1, -1)]) if tail else d["q"]
    out = torch.full(q.shape, 0xA5 if fp8 else 7.0, dtype=torch.uint8 if fp8 else q.dtype, device="cuda")
    stats = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    got = edge_ops.paged_attention(q, d["k"], d["v"], d["table"], d["lens"], page_size=c["page"],
                                   q_starts=d["starts"] if starts else None, scale=scale, causal=causal,
                                   window=window, out=out, lse=stats, fp8=fp8, inv_scale=inv or 1.0, **kw)
    assert got is out
    return out, stats


def verify(c, *, starts=True, fp8=False, inv=None, causal=True, window=0, scale=None, **kw):
    out, stats = run(c, starts=starts, fp8=fp8, inv=inv, causal=causal, window=window, scale=scale, **kw)
    torch.cuda.synchronize()
    s = c["q"].shape[2] ** -0.5 if scale is None else scale
    ref, tol, lse, ltol = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"],
                                              c["starts"] if starts else None, c["page"], s, causal, window)
    n = c["q"].shape[0]
    paged_ref.check_rows(out[:n], ref, tol, c["q"].dtype, inv if fp8 else None)
    assert (out[n:] == (0xA5 if fp8 else 7.0)).all(), "rows of no sequence were written"
    if stats is not None:
        got = stats.cpu().double()[:n]
        same = got == lse
        assert (same | ((got - lse).abs() <= ltol)).all()
        assert (stats[n:] == 7.0).all()
    return out, stats


HEADS = [(4, 2, 64), (8, 2, 128), (16, 2, 256), (6, 1, 128), (3, 3, 128), (24, 4, 256), (5, 1, 80), (4, 2, 96),
         (2, 1, 33), (40, 2, 64), (6, 2, 192), (2, 2, 1)]


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", HEADS)
def test_decode(dt, hq, hk, D):
    lens = [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 300]
    verify(make(dt, hq, hk, D, 16, [(n, 1) for n in lens], seed=D), starts=False)


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", HEADS)
@pytest.mark.parametrize("page", [16, 13])
def test_chunks(dt, hq, hk, D, page):
    shape = [(1, 1), (7, 7), (40, 3), (0, 0), (65, 17), (130, 64), (5, 0), (161, 2)]
    verify(make(dt, hq, hk, D, page, shape, seed=D + page), tail=2)


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [1, 8, 16, 64, 128, 256, 48])
def test_page_sizes(dt, page):
    verify(make(dt, 8, 2, 128, page, [(257, 5), (64, 33), (100, 100), (1, 1)], seed=page))


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 2, 256)])
def test_window(dt, window, hq, hk, D):
    verify(make(dt, hq, hk, D, 16, [(300, 1), (200, 70), (140, 140), (64, 1), (65, 2)], seed=window), window=window)


@gpu
@pytest.mark.parametrize("dt,new", [("f32", 9), ("bf16", 1), ("bf16", 9), ("bf16", 90)])
def test_the_widest_window_is_none(dt, new):
    # fewer keys than new tokens in one sequence: its first positions are negative
    c = make(dt, 8, 2, 128, 16, [(300, new), (5, new), (90, new)], seed=27)
    want, _ = run(c)
    for window in (300, 2 ** 30 - 1, 2 ** 31 - 1):
        got, _ = verify(c, window=window)
        assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", [(8, 8, 64), (8, 2, 128), (4, 1, 256)])
def test_cross_attention(dt, hq, hk, D):
    # every key of the sequence is seen; more queries than keys, and none at all
    verify(make(dt, hq, hk, D, 16, [(100, 7), (3, 40), (129, 1), (0, 5)], seed=3), causal=False)


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing(dt):
    # no keys at all; fewer keys than new tokens (the first queries sit before the sequence)
    c = make(dt, 8, 2, 128, 16, [(0, 1), (3, 9), (0, 4), (20, 1), (1, 100)], seed=5)
    out, lse = verify(c, tail=1)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (out[1:7] == 0).all() and (lse[1:7] == -math.inf).all()


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 30])
def test_bad_pages_are_not_read(dt, new):
    c = make(dt, 8, 2, 128, 16, [(100, new), (50, min(new, 50)), (33, 1)], seed=6)
    pages = c["k"].shape[0] // 16
    c["table"][0, 2] = -1
    c["table"][0, 4] = pages           # the page past the pool
    c["table"][1, :] = -2 ** 31        # a sequence with no page in the pool
    c["table"][2, 0] = 2 ** 31 - 1
    verify(c)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_lengths_past_the_table_are_clamped(dt):
    c = make(dt, 8, 2, 128, 16, [(64, 1), (64, 3)], seed=7, spare=4)
    c["table"] = c["table"][:, :4].contiguous()
    c["lens"] = torch.tensor([10 ** 9, 64], dtype=torch.int32)
    verify(c)
    c["lens"] = torch.tensor([-5, 64], dtype=torch.int32)
    verify(c)


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_values_behind_the_mask_do_not_matter(dt):
    # keys that only later queries see hold NaN and infinity: earlier rows stay as the formula has them
    c = make(dt, 8, 2, 128, 16, [(200, 150)], seed=8)
    for j, bad in ((120, math.nan), (150, math.inf), (199, math.nan)):
        slot = int(c["table"][0, j // 16]) * 16 + j % 16
        c["v"][slot] = bad
        c["k"][slot] = math.nan
    out, lse = run(c, lse=True)
    torch.cuda.synchronize()
    ref, tol, _, _ = paged_ref.attention(c["q"], c["k"].nan_to_num(0, 0, 0), c["v"].nan_to_num(0, 0, 0), c["table"],
                                         c["lens"], c["starts"], 16, 128 ** -0.5)
    clean = 120 - 50  # queries before position 120
    paged_ref.check_rows(out[:clean], ref[:clean], tol[:clean], c["q"].dtype)
    assert torch.isnan(out[clean:]).all()


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_fp8_output(dt, new):
    verify(make(dt, 8, 2, 128, 16, [(200, new), (77, new), (41, new)], seed=9), fp8=True, inv=100.0, tail=1)


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_sharp_scores(dt):
    # scores of +-100s: one key carries a row, and the maximum moves late
    verify(make(dt, 8, 2, 128, 16, [(300, 1), (300, 50)], seed=10, sharp=30.0), scale=0.2)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_growing_scores(dt):
    # each key scores higher than the last, so every tile moves the maximum
    c = make(dt, 4, 1, 64, 16, [(400, 1), (400, 70)], seed=11)
    for b in range(2):
        for j in range(400):
            c["k"][int(c["table"][b, j // 16]) * 16 + j % 16] = j / 16
    c["q"] = torch.full_like(c["q"], 0.5)
    verify(c)


@gpu
@pytest.mark.parametrize("dt,hq,hk,D", [("bf16", 8, 2, 128), ("f16", 16, 2, 256), ("f32", 4, 1, 64)])
def test_long_sequences_split_over_the_gpu(dt, hq, hk, D):
    verify(make(dt, hq, hk, D, 64, [(20011, 1), (5, 1), (9000, 1)], seed=12), starts=False)
    verify(make(dt, hq, hk, D, 16, [(6007, 9), (1, 1), (3000, 2)], seed=13))


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_sequences(dt):
    r = random.Random(14)
    verify(make(dt, 4, 2, 64, 16, [(r.randrange(1, 60), 1) for _ in range(1500)], seed=14), starts=False)
    verify(make(dt, 4, 2, 64, 16, [(r.randrange(4, 40), r.randrange(0, 4)) for _ in range(700)], seed=15))


@gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_unaligned_caches(dt):
    c = make(dt, 8, 2, 128, 16, [(100, 20), (37, 1)], seed=16)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}

    def shift(x):
        raw = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        y = raw[1:].view(x.shape)
        y.copy_(x)
        return y

    out = edge_ops.paged_attention(shift(d["q"]), shift(d["k"]), shift(d["v"]), d["table"], d["lens"], page_size=16,
                                   q_starts=d["starts"], out=shift(torch.zeros_like(d["q"])))
    ref, tol, _, _ = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], 16, 128 ** -0.5)
    paged_ref.check_rows(out, ref, tol, c["q"].dtype)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [1, 20, 200])
def test_an_output_aligned_to_its_elements(new, fp8):
    # every tensor but the output (and the statistics) on 16 bytes
    c = make("bf16", 8, 2, 128, 16, [(300, new), (257, new)], seed=26)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}
    odt = torch.uint8 if fp8 else torch.bfloat16
    raw = torch.full((d["q"].numel() + 2,), 7, dtype=odt, device="cuda")
    stats = torch.full((2 * new * 8 + 2,), 7.0, device="cuda")
    edge_ops.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], page_size=16, q_starts=d["starts"],
                             out=raw[1:-1].view(d["q"].shape), lse=stats[1:-1].view(-1, 8), fp8=fp8, inv_scale=50.0)
    ref, tol, lse, lt = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], 16, 128 ** -0.5)
    paged_ref.check_rows(raw[1:-1].view(d["q"].shape), ref, tol, torch.bfloat16, 50.0 if fp8 else None)
    assert ((stats[1:-1].view(-1, 8).cpu().double() - lse).abs() <= lt).all()
    assert raw[0] == 7 and raw[-1] == 7 and stats[0] == 7 and stats[-1] == 7


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 60])
def test_same_bits_again_and_with_a_dirty_workspace(dt, new):
    c = make(dt, 8, 2, 128, 16, [(2000, new), (77, new), (900, new)], seed=17)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}
    ws = edge_ops.paged_attention_workspace(d["q"], d["k"])
    first, lse = run(c)
    for fill in (0, 255):
        ws.fill_(fill)
        again, lse2 = run(c, workspace=ws)
        assert torch.equal(first, again) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("new", [1, 60])
def test_other_stream_and_graph(new):
    c = make("bf16", 8, 2, 128, 16, [(500, new), (77, new)], seed=18)
    want, _ = run(c)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = (d["q"], d["k"], d["v"], d["table"], d["lens"])
    for stream in (side, side.cuda_stream):
        got = edge_ops.paged_attention(*args, page_size=16, q_starts=d["starts"], stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
    ws = edge_ops.paged_attention_workspace(d["q"], d["k"])
    out = torch.zeros_like(d["q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        edge_ops.paged_attention(*args, page_size=16, q_starts=d["starts"], out=out, workspace=ws)
    # replays read what the buffers hold then: shorter sequences
    for cut in (0, 3):
        d["lens"].copy_(c["lens"] - cut)
        graph.replay()
        torch.cuda.synchronize()
        ref, tol, _, _ = paged_ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"] - cut, c["starts"], 16,
                                             128 ** -0.5)
        paged_ref.check_rows(out, ref, tol, torch.bfloat16)


@gpu
def test_empty_calls():
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 64, device="cuda")
    k = torch.zeros(32, 2, 64, device="cuda")
    # no tokens, with and without sequences; a cache without pages; a table without columns
    for b in (0, 2):
        starts = torch.zeros(b + 1, **i32)
        assert edge_ops.paged_attention(q, k, k, torch.zeros(b, 3, **i32), torch.ones(b, **i32), page_size=8,
                                        q_starts=starts).shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, device="cuda")
    for cache, width in ((k[:0], 3), (k, 0)):
        out = edge_ops.paged_attention(q, cache, cache, torch.zeros(2, width, **i32), torch.full((2,), 9, **i32),
                                       page_size=8)
        assert (out == 0).all()


@gpu
def test_binding_checks_its_tensors():
    c = make("bf16", 4, 2, 64, 16, [(40, 2)], seed=19)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}

    def go(**kw):
        a = dict(q=d["q"], k_cache=d["k"], v_cache=d["v"], block_table=d["table"], lens=d["lens"], page_size=16,
                 q_starts=d["starts"])
        edge_ops.paged_attention(**{**a, **kw})

    go()
    for bad, error in [(dict(k_cache=d["k"].half()), TypeError), (dict(v_cache=d["v"][:-1]), ValueError),
                       (dict(block_table=d["table"].long()), TypeError), (dict(lens=d["lens"].long()), TypeError),
                       (dict(lens=d["lens"].cpu()), ValueError), (dict(q_starts=d["starts"][:-1]), ValueError),
                       (dict(q=d["q"].transpose(0, 1)), ValueError), (dict(lse=torch.zeros(2, 4)), ValueError),
                       (dict(out=torch.zeros_like(d["q"])[:1]), ValueError), (dict(page_size=0), edge_ops.EdgeError),
                       (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), edge_ops.EdgeError),
                       (dict(scale=0.0), edge_ops.EdgeError), (dict(window=-1), edge_ops.EdgeError)]:
        with pytest.raises(error):
            go(**bad)


# chunks of many rows per key head

WIDE = [(8, 2, 128), (3, 3, 128), (6, 1, 64), (12, 2, 80), (24, 2, 104), (40, 1, 128), (4, 2, 256), (16, 1, 192)]


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", WIDE)
@pytest.mark.parametrize("page", [8, 32, 128, 384])
def test_wide_chunks(dt, hq, hk, D, page):
    # units that end inside, at and behind a tile of 128 rows or keys; whole prompts and late chunks
    verify(make(dt, hq, hk, D, page, [(300, 300), (1100, 130), (129, 1), (128, 128), (70, 0), (0, 3), (513, 257)], seed=page + D),
           tail=3)


@gpu
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 4, 64), (4, 2, 256)])
@pytest.mark.parametrize("window", [1, 64, 127, 128, 129, 300])
def test_wide_chunks_window(hq, hk, D, window):
    verify(make("bf16", hq, hk, D, 16, [(600, 400), (260, 260), (900, 100)], seed=window), window=window)


@gpu
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 4, 64), (4, 2, 256)])
def test_wide_chunks_cross_and_bad_pages(hq, hk, D):
    c = make("f16", hq, hk, D, 16, [(333, 200), (40, 300), (0, 200), (1000, 90)], seed=21)
    verify(c, causal=False, fp8=True, inv=50.0)
    pages = c["k"].shape[0] // 16
    c["table"][0, 3] = -1
    c["table"][0, 20] = pages
    c["table"][1, :] = pages + 7
    c["table"][3, 8:40] = -5
    verify(c, causal=False)
    verify(c)


@gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 4, 64), (4, 2, 256)])
def test_wide_values_behind_the_mask(dt, hq, hk, D):
    # NaN and infinite values that only later queries see, in several units and tiles
    c = make(dt, hq, hk, D, 16, [(700, 600), (400, 300)], seed=22)
    for b, j, bad in ((0, 350, math.nan), (0, 690, math.inf), (1, 399, -math.inf)):
        slot = int(c["table"][b, j // 16]) * 16 + j % 16
        c["v"][slot] = bad
    out, lse = run(c)
    torch.cuda.synchronize()
    ref, tol, rl, lt = paged_ref.attention(c["q"], c["k"], c["v"].nan_to_num(0, 0, 0), c["table"], c["lens"],
                                           c["starts"], 16, D ** -0.5)
    clean = torch.ones(900, dtype=torch.bool)
    clean[250:600] = False
    clean[899] = False
    ref[~clean], tol[~clean] = math.nan, math.nan
    paged_ref.check_rows(out, ref, tol, c["q"].dtype)
    assert torch.isnan(out[250:600]).any(-1).all() and not torch.isfinite(out[899]).any()
    assert ((lse.cpu().double() - rl).abs() <= lt).all()


@gpu
def test_wide_chunk_splits_and_repeats():
    # one sequence over the whole GPU: units in several pieces; the same bits each time
    c = make("bf16", 8, 2, 128, 16, [(9000, 300), (33, 33)], seed=23, sharp=3.0)
    first, lse = verify(c)
    again, lse2 = run(c)
    assert torch.equal(first, again) and torch.equal(lse, lse2)


@gpu
def test_wide_growing_scores():
    c = make("bf16", 4, 1, 128, 16, [(900, 300)], seed=24)
    for j in range(900):
        c["k"][int(c["table"][0, j // 16]) * 16 + j % 16] = j / 16
    c["q"] = torch.full_like(c["q"], 0.5)
    verify(c)


@gpu
def test_wide_chunk_on_another_stream_and_in_a_graph():
    c = make("bf16", 8, 2, 128, 16, [(700, 200), (300, 300)], seed=25)
    want, _ = verify(c)
    d = {n: x.cuda() for n, x in c.items() if n != "page"}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = (d["q"], d["k"], d["v"], d["table"], d["lens"])
    got = edge_ops.paged_attention(*args, page_size=16, q_starts=d["starts"], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs with a workspace each, replayed together
    outs, graphs = [torch.zeros_like(d["q"]) for _ in range(2)], []
    works = [edge_ops.paged_attention_workspace(d["q"], d["k"]) for _ in range(2)]
    for out, ws in zip(outs, works):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            edge_ops.paged_attention(*args, page_size=16, q_starts=d["starts"], out=out, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
