"""Rotary positions with several axes: against the oracle, the form with one axis, and its refusals.

The oracle takes one position per token, so a case's angles are gathered first: row t of its cache holds, for every
pair, the cos and sin of that pair's axis.  Token t then has position t, or one past the cache where an axis is out.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from helpers import TORCH_FMT, storage
from memory_bound_decode_qk_gb300 import _build, edge_ops, synth
from test_gpu_parity import Guarded, check_out, dev
from tolerances import ETA_NORM

OK, NULL, DTYPE, SHAPE, ALIGN, ALIAS, UNSUP, CUDA, VALUE = range(9)
F32, F16, BF16, FP8 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return edge_ops.lib()


# ---------------------------------------------------------------- refusals (no GPU)

QO, KO, Q, K, WQ, WK, POS, COS, SIN, KC, VC, SL = (0x10000000 * i for i in range(1, 13))


def ints(v):
    return None if v is None else (ctypes.c_int32 * max(1, len(v)))(*v)


def qk(L, rot=64, pos=POS, axes=3, sections=(8, 12, 12), order=0, P=4096, flags=0, T=4, qo=QO, D=128):
    return L.edge_qk_norm_rope_axes(qo, KO, BF16, Q, K, WQ, WK, BF16, T, 8, 2, D, rot, 0, pos, axes, ints(sections),
                                    order, COS, SIN, P, 1e-6, 1, 1.0, flags, None)


def rope(L, rot=64, pos=POS, axes=3, sections=(8, 12, 12), order=0, P=4096, flags=0, T=4, qo=QO, D=128):
    return L.edge_rope_axes(qo, KO, BF16, Q, K, BF16, T, 8, 2, D, rot, 0, pos, axes, ints(sections), order, COS, SIN, P,
                            1.0, None)


def qkv(L, rot=64, pos=POS, axes=3, sections=(8, 12, 12), order=0, P=4096, flags=0, T=4, qo=QO, D=128):
    return L.edge_qkv_rope_cache_axes(qo, KC, VC, Q, WQ, WK, BF16, T, 8, 2, D, rot, 0, pos, axes, ints(sections), order,
                                      COS, SIN, P, SL, 64, 1e-6, 1, 1, None)


@pytest.mark.parametrize("entry", [qk, rope, qkv])
@pytest.mark.parametrize("kw,status", [
    (dict(sections=None), NULL), (dict(pos=None), NULL),
    (dict(axes=0, sections=()), SHAPE), (dict(axes=5, sections=(8, 8, 8, 4, 4)), SHAPE),
    (dict(sections=(8, 12, 11)), SHAPE), (dict(sections=(8, 12, 13)), SHAPE), (dict(sections=(-8, 20, 20)), SHAPE),
    (dict(sections=(2 ** 31 - 1, 2 ** 31 - 1, 34)), SHAPE),
    (dict(order=1, sections=(0, 20, 12)), SHAPE),          # axis 1 has no 20th pair: 3 * 19 + 1 > 31
    (dict(order=2), VALUE), (dict(order=-1), VALUE),
    (dict(qo=POS + 64), ALIAS),                            # inside the positions of the last axis
    (dict(rot=65, sections=(8, 12, 12)), SHAPE), (dict(D=2050), UNSUP),
])
def test_refusals(L, entry, kw, status):
    assert entry(L, **kw) == status


def test_flags_and_empty_calls(L):
    assert qk(L, flags=2) == VALUE
    for entry in (qk, rope, qkv):
        assert entry(L, T=0) == OK
        assert entry(L, T=0, order=1, sections=(12, 10, 10)) == OK
    assert L.edge_last_cuda_error() == 0


def axis_of(j, sections, order):
    n = len(sections)
    if order == "cycled":
        return j % n if j // n < sections[j % n] else 0
    return next(a for a in range(n) if j < sum(sections[:a + 1]))


@pytest.mark.parametrize("sections,half", [((11, 11, 10), 32), ((12, 10, 10), 32), ((24, 20, 20), 64), ((5, 3), 8),
                                           ((8,), 8), ((7, 3, 3, 3), 16)])
def test_dealt_sections_have_their_pairs(sections, half):
    # every pair has an axis, and each axis its number of pairs
    axes = [axis_of(j, sections, "cycled") for j in range(half)]
    assert [axes.count(a) for a in range(len(sections))] == list(sections)


# ---------------------------------------------------------------- GPU

gpu = pytest.mark.gpu

CASES = {
    # lane-group paths: the axis border inside a 16-byte vector, dealt pairs, both layouts, every type
    "text256_blocks": dict(dtype=torch.bfloat16, T=70, Hq=16, Hk=2, D=256, rot=64, layout=0, sections=(8, 12, 12), order="blocks"),
    "text256_cycled": dict(dtype=torch.bfloat16, T=70, Hq=24, Hk=4, D=256, rot=64, layout=0, sections=(12, 10, 10), order="cycled"),
    "d128_blocks_odd": dict(dtype=torch.bfloat16, T=33, Hq=32, Hk=8, D=128, rot=128, layout=0, sections=(17, 24, 23), order="blocks"),
    "d128_cycled": dict(dtype=torch.float16, T=33, Hq=32, Hk=8, D=128, rot=128, layout=0, sections=(24, 20, 20), order="cycled"),
    "d256_interleaved": dict(dtype=torch.bfloat16, T=19, Hq=16, Hk=8, D=256, rot=256, layout=1, sections=(30, 50, 48), order="blocks"),
    "d64_f16_interleaved_cycled": dict(dtype=torch.float16, T=40, Hq=4, Hk=4, D=64, rot=32, layout=1, sections=(6, 5, 5), order="cycled"),
    "f32_d128": dict(dtype=torch.float32, T=21, Hq=8, Hk=2, D=128, rot=128, layout=0, sections=(22, 21, 21), order="cycled"),
    "f32_interleaved": dict(dtype=torch.float32, T=21, Hq=8, Hk=2, D=128, rot=64, layout=1, sections=(10, 11, 11), order="blocks"),
    "four_axes": dict(dtype=torch.bfloat16, T=12, Hq=4, Hk=2, D=128, rot=64, layout=0, sections=(5, 9, 9, 9), order="blocks"),
    "four_axes_cycled": dict(dtype=torch.bfloat16, T=12, Hq=4, Hk=2, D=128, rot=64, layout=0, sections=(11, 7, 7, 7), order="cycled"),
    "two_axes_empty": dict(dtype=torch.bfloat16, T=12, Hq=4, Hk=2, D=128, rot=64, layout=0, sections=(0, 32), order="blocks"),
    "one_axis": dict(dtype=torch.bfloat16, T=12, Hq=4, Hk=2, D=128, rot=64, layout=0, sections=(32,), order="cycled"),
    # many heads
    "many_d128": dict(dtype=torch.bfloat16, T=1300, Hq=32, Hk=8, D=128, rot=128, layout=0, sections=(16, 24, 24), order="blocks"),
    "many_d256": dict(dtype=torch.bfloat16, T=1100, Hq=16, Hk=8, D=256, rot=128, layout=0, sections=(24, 20, 20), order="cycled"),
    "many_d256_unweighted": dict(dtype=torch.float16, T=900, Hq=24, Hk=4, D=256, rot=64, layout=0, sections=(8, 12, 12), order="blocks"),
    # any size or alignment
    "generic_d96": dict(dtype=torch.bfloat16, T=9, Hq=3, Hk=1, D=96, rot=96, layout=0, sections=(16, 16, 16), order="cycled"),
    "generic_odd": dict(dtype=torch.float16, T=6, Hq=2, Hk=3, D=37, rot=20, layout=1, sections=(4, 3, 3), order="blocks"),
    "generic_rot24": dict(dtype=torch.bfloat16, T=5, Hq=4, Hk=2, D=256, rot=24, layout=0, sections=(4, 4, 4), order="cycled"),
    "misaligned": dict(dtype=torch.bfloat16, T=11, Hq=16, Hk=2, D=256, rot=64, layout=0, sections=(8, 12, 12), order="blocks", misalign=1),
}
P = 512


def inputs(c, seed=0):
    T, n = c["T"], len(c["sections"])
    inp = synth.qk_inputs(seed, c["dtype"], T, c["Hq"], c["Hk"], c["D"], c["rot"], theta=1e4, cache_len=P,
                          positions="arange", w_mean=0.0, w_std=0.1)
    r = np.random.RandomState(7 + T)
    pos = r.randint(0, P, (n, T)).astype(np.int64)
    pos[:, 0], pos[:, 1] = 0, P - 1
    # out of the cache on one axis, the first or the last, or on all
    for t, (a, bad) in enumerate([(0, -1), (n - 1, P), (0, 1 << 40), (n - 1, -(1 << 62))]):
        if t + 2 < T:
            pos[a, t + 2] = bad
    inp["positions"] = torch.from_numpy(pos)
    cos, sin = inp["cos"].numpy(), inp["sin"].numpy()
    half = c["rot"] // 2
    axis = np.array([axis_of(j, c["sections"], c["order"]) for j in range(half)])
    good = ((pos >= 0) & (pos < P)).all(0)
    at = np.where(good, pos, 0)[axis].T                       # [T, half]
    inp["row_cos"] = np.ascontiguousarray(cos[at, np.arange(half)])
    inp["row_sin"] = np.ascontiguousarray(sin[at, np.arange(half)])
    inp["row_pos"] = np.where(good, np.arange(T), T).astype(np.int64)
    return inp


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_prologue(name, fp8):
    c = CASES[name]
    inp, fmt = inputs(c), TORCH_FMT[c["dtype"]]
    out_fmt, inv = (oracle.E4M3, 40.0) if fp8 else (fmt, 1.0)
    ref = oracle.qk_norm_rope(storage(inp["q"]), storage(inp["k"]), storage(inp["wq"]), storage(inp["wk"]), fmt, c["rot"],
                              c["layout"], inp["row_pos"], inp["row_cos"], inp["row_sin"], 1e-6, 1, out_fmt=out_fmt,
                              inv_scale=inv, eta=ETA_NORM)
    mis, odt = c.get("misalign", 0), torch.uint8 if fp8 else c["dtype"]
    q, k, wq, wk = (dev(inp[n], mis) for n in ("q", "k", "wq", "wk"))
    gq, gk = Guarded(q.shape, odt, mis), Guarded(k.shape, odt, mis)
    edge_ops.qk_norm_rope(q, k, wq, wk, dev(inp["positions"]), dev(inp["cos"]), dev(inp["sin"]), rotary_dim=c["rot"],
                          layout=c["layout"], weight_offset=1, q_out=gq.t, k_out=gk.t, fp8=fp8, inv_scale=inv,
                          sections=c["sections"], axis_order=c["order"])
    torch.cuda.synchronize()
    gq.check()
    gk.check()
    check_out(name + " q", storage(gq.t.cpu()), ref.q_out, ref.q_pre, ref.q_mag, fmt, out_fmt, ETA_NORM, inv, ref.q_lo, ref.q_hi)
    check_out(name + " k", storage(gk.t.cpu()), ref.k_out, ref.k_pre, ref.k_mag, fmt, out_fmt, ETA_NORM, inv, ref.k_lo, ref.k_hi)


@gpu
@pytest.mark.parametrize("name", [n for n in CASES if "misaligned" not in n])
def test_rope_alone(name):
    c = CASES[name]
    inp, fmt = inputs(c), TORCH_FMT[c["dtype"]]
    q, k = dev(inp["q"]), dev(inp["k"])
    edge_ops.rope(q, k, dev(inp["positions"]), dev(inp["cos"]), dev(inp["sin"]), rotary_dim=c["rot"], layout=c["layout"],
                  q_out=q, k_out=k, sections=c["sections"], axis_order=c["order"])
    torch.cuda.synchronize()
    for got, x in ((q, inp["q"]), (k, inp["k"])):
        r = oracle.rope(storage(x), fmt, c["rot"], c["layout"], inp["row_pos"], inp["row_cos"], inp["row_sin"],
                        diagnostics=True)
        check_out(name, storage(got.cpu()), r[0], r[1], r[2], fmt, fmt, ETA_NORM)


@gpu
@pytest.mark.parametrize("name", [n for n in CASES if "misaligned" not in n])
def test_qkv_write(name):
    c = CASES[name]
    inp, fmt, T, S = inputs(c), TORCH_FMT[c["dtype"]], c["T"], c["T"] + 3
    qkv = torch.cat([inp["q"].reshape(T, -1), inp["k"].reshape(T, -1), inp["k"].flip(0).reshape(T, -1)], 1).contiguous()
    slots = np.random.RandomState(3).permutation(S)[:T].astype(np.int64)
    slots[-1] = -1
    fill = np.full((S, c["Hk"], c["D"]), 3.0)
    old = synth.to_dtype(fill, c["dtype"])
    ref = oracle.qkv_rope_cache(storage(qkv), storage(inp["wq"]), storage(inp["wk"]), fmt, c["Hq"], c["Hk"], c["rot"],
                                c["layout"], inp["row_pos"], inp["row_cos"], inp["row_sin"], slots, storage(old),
                                storage(old), 1e-6, 1, eta=ETA_NORM)
    kc, vc = Guarded(old.shape, c["dtype"]), Guarded(old.shape, c["dtype"])
    kc.t.copy_(old)
    vc.t.copy_(old)
    q = edge_ops.qkv_rope_cache(dev(qkv), c["Hq"], c["Hk"], dev(inp["wq"]), dev(inp["wk"]), dev(inp["positions"]),
                                dev(inp["cos"]), dev(inp["sin"]), dev(torch.from_numpy(slots)), kc.t, vc.t,
                                rotary_dim=c["rot"], layout=c["layout"], weight_offset=1, sections=c["sections"],
                                axis_order=c["order"])
    torch.cuda.synchronize()
    kc.check()
    vc.check()
    check_out(name + " q", storage(q.cpu()), ref.q_out, ref.q_pre, ref.q_mag, fmt, fmt, ETA_NORM, 1.0, ref.q_lo, ref.q_hi)
    gk, w = storage(kc.t.cpu()), slots[:-1]
    check_out(name + " k", gk[w], ref.k_cache[w], ref.k_pre[w], ref.k_mag[w], fmt, fmt, ETA_NORM, 1.0, ref.k_lo[w],
              ref.k_hi[w])
    untouched = np.setdiff1d(np.arange(S), w)
    assert np.array_equal(gk[untouched], storage(old)[untouched])
    assert np.array_equal(storage(vc.t.cpu()), ref.v_cache)


@gpu
@pytest.mark.parametrize("name", ["d128_cycled", "d256_interleaved", "f32_d128", "generic_d96"])
@pytest.mark.parametrize("unrounded", [False, True])
def test_equal_positions_are_one_position(name, unrounded):
    c = CASES[name]
    inp = inputs(c)
    one = inp["positions"][0].contiguous()
    args = [dev(inp[n]) for n in ("q", "k", "wq", "wk")]
    kw = dict(rotary_dim=c["rot"], layout=c["layout"], weight_offset=1, unrounded=unrounded)
    a = edge_ops.qk_norm_rope(*args, dev(one), dev(inp["cos"]), dev(inp["sin"]), **kw)
    b = edge_ops.qk_norm_rope(*args, dev(one.expand(3, -1).contiguous()), dev(inp["cos"]), dev(inp["sin"]), **kw,
                              sections=c["sections"], axis_order=c["order"])
    # at these widths both take the same form of the head's arithmetic
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_in_a_graph_with_changing_positions():
    c = CASES["d128_blocks_odd"]
    inp = inputs(c)
    args = [dev(inp[n]) for n in ("q", "k", "wq", "wk")]
    pos, cs, sn = dev(inp["positions"]), dev(inp["cos"]), dev(inp["sin"])
    kw = dict(rotary_dim=c["rot"], weight_offset=1, sections=c["sections"], axis_order=c["order"])
    out = [torch.empty_like(args[0]), torch.empty_like(args[1])]
    edge_ops.qk_norm_rope(*args, pos, cs, sn, q_out=out[0], k_out=out[1], **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        edge_ops.qk_norm_rope(*args, pos, cs, sn, q_out=out[0], k_out=out[1], **kw)
    pos.copy_(pos.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    want = edge_ops.qk_norm_rope(*args, pos, cs, sn, **kw)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@gpu
def test_binding_checks_positions():
    c = CASES["text256_blocks"]
    inp = inputs(c)
    args = [dev(inp[n]) for n in ("q", "k", "wq", "wk")]
    cs, sn = dev(inp["cos"]), dev(inp["sin"])
    for pos in (inp["positions"][:2], inp["positions"][:, :-1].contiguous(), inp["positions"].int(), inp["positions"][0]):
        with pytest.raises(ValueError, match="positions"):
            edge_ops.qk_norm_rope(*args, dev(pos), cs, sn, rotary_dim=64, sections=(8, 12, 12))
