"""Measured cases of the paged-cache operators: attention of a chunk of new tokens over a paged KV cache, rotary
positions with several axes, and the moves of cache pages.  Each has a plain form in elementary torch operations and
the call a user's program makes of this package (`own`)."""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    def attend(name, **k):
        base = {"name": name, "op": "attend", "causal": True, "window": 0, "fp8": False, "lse": False}
        return {**base, **k}

    return [
        # one user, a short conversation, one new token: latency
        attend("decode one 16/2x256", dt="bf16", hq=16, hk=2, d=256, ps=16, b=1, lmin=517, lmax=517, nmin=1, nmax=1),
        # a serving batch: one new token for each of 64 sequences of mixed lengths
        attend("decode batch 32/8x128", dt="bf16", hq=32, hk=8, d=128, ps=16, b=64, lmin=64, lmax=8192, nmin=1, nmax=1),
        # a few users with long documents, one new token each
        attend("decode long 24/4x256", dt="fp16", hq=24, hk=4, d=256, ps=64, b=3, lmin=30011, lmax=131072, nmin=1,
               nmax=1),
        # blocks of 16 drafted tokens to verify, heads of a draft model (no shared key heads); FP8 for the next product
        attend("verify block 32/32x128", dt="bf16", hq=32, hk=32, d=128, ps=16, b=8, lmin=300, lmax=4096, nmin=16,
               nmax=16, fp8=True),
        # chunked prefill: 1024 new tokens late in two long prompts
        attend("chunk over 16k 32/8x128", dt="bf16", hq=32, hk=8, d=128, ps=16, b=2, lmin=16384, lmax=16384,
               nmin=1024, nmax=1024),
        # whole prompts of odd lengths through a layer with a sliding window
        attend("prompts windowed 16/8x256", dt="fp16", hq=16, hk=8, d=256, ps=32, b=4, lmin=1201, lmax=5003, nmin=6000,
               nmax=6000, window=1024),
        # fp32 chunks of odd sizes over pages of 13 tokens, with the softmax statistics for a later merge
        attend("odd chunks fp32 8/2x128", dt="fp32", hq=8, hk=2, d=128, ps=13, b=5, lmin=45, lmax=999, nmin=1, nmax=37,
               lse=True),
        # new tokens of a video prompt through the prologue: time, height and width positions, blocks of channels
        {"name": "prologue axes 16/8x256", "op": "prologue", "dt": "bf16", "t": 1156, "hq": 16, "hk": 8, "d": 256,
         "rot": 128, "order": "blocks", "offset": 1},
        # the decode step's fused QKV split and cache write, axes dealt in turn over the channels
        {"name": "qkv write axes 32/8x128", "op": "qkv", "dt": "bf16", "t": 64, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "order": "cycled", "offset": 0, "slots": 16384},
        # a block of pages copied in every layer's caches (a prompt's pages for a second holder)
        {"name": "copy 1000 pages", "op": "copy", "dt": "bf16", "caches": 16, "hk": 8, "d": 128, "ps": 16,
         "pages": 4096, "n": 1000},
        # one step of a beam search over 16 rows: half the rows are dropped and become copies of the others
        {"name": "beam step 8 of 16", "op": "beam", "dt": "bf16", "caches": 48, "hk": 8, "d": 128, "ps": 16,
         "pages": 1024, "rows": 16, "lmin": 200, "lmax": 700},
        # a cache in which finished sequences left holes, moved together
        {"name": "compact 4096 pages", "op": "compact", "dt": "bf16", "caches": 16, "hk": 8, "d": 128, "ps": 16,
         "pages": 4096, "rows": 64, "lmin": 16, "lmax": 1024},
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend"] * 6 + ["prologue", "qkv", "copy", "beam", "compact"])
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "attend":
        hq, hk, d = rng.choice([(16, 2, 256), (24, 4, 256), (32, 8, 128), (16, 8, 256), (32, 32, 128), (8, 2, 128),
                                (8, 8, 64), (5, 1, 64), (6, 2, 80), (12, 4, 96)])
        b = span(1, 64)
        chunk = rng.choice([1, 1, 2])
        nmax = 1 if chunk == 1 else span(2, 1500)
        top = 60000 // b if chunk == 1 else min(16384, max(64, 40_000_000 // (b * nmax)))
        if dt == "fp32":
            top = max(64, top // 4)
        lmax = span(1, max(2, top))
        return {"op": "attend", "dt": dt, "hq": hq, "hk": hk, "d": d, "ps": rng.choice([1, 8, 13, 16, 32, 64, 128]),
                "b": b, "lmin": span(1, lmax), "lmax": lmax, "nmin": 1, "nmax": nmax,
                "causal": rng.random() < 0.8, "window": rng.choice([0, 0, span(1, 2000)]),
                "fp8": rng.random() < 0.2, "lse": rng.random() < 0.3}
    if op in ("prologue", "qkv"):
        hq, hk, d, rot = rng.choice([(16, 2, 256, 64), (24, 4, 256, 64), (32, 8, 128, 128), (16, 8, 256, 256),
                                     (8, 2, 128, 96), (6, 2, 80, 80), (16, 8, 256, 128)])
        case = {"op": op, "dt": dt, "t": span(1, 4096), "hq": hq, "hk": hk, "d": d, "rot": rot,
                "order": rng.choice(["blocks", "cycled"]), "offset": rng.choice([0, 1])}
        if op == "qkv":
            case["slots"] = case["t"] + span(1, 16384)
        return case
    case = {"op": op, "dt": dt, "caches": rng.choice([2, 8, 16, 24]), "hk": rng.choice([1, 2, 4, 8]),
            "d": rng.choice([80, 128, 256]) // (2 if dt == "fp32" else 1), "ps": rng.choice([1, 13, 16, 32])}
    if op == "copy":
        pages = span(4, 3000)
        return {**case, "pages": pages, "n": span(1, pages // 2)}
    rows = span(2, 32)
    lmax = span(1, 1500)
    return {**case, "rows": rows, "lmin": span(1, lmax), "lmax": lmax,
            "pages": 2 * rows * -(-lmax // case["ps"]) + rows + span(1, 500)}


def _lengths(case, what):
    """Lengths of the case's sequences, fixed by the case alone: spread over their logarithm, the largest among them."""
    count = case["b"] if "b" in case else case["rows"]
    lo, hi = case["lmin"], case["lmax"]
    r = random.Random("%s %d %d %d" % (what, count, lo, hi))
    out = [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(count)]
    out[r.randrange(count)] = hi
    return out


def _chunks(case):
    """(keys, new tokens) of each sequence; the new tokens are the last of the keys."""
    r = random.Random("chunks %d %d" % (case["nmin"], case["nmax"]))
    lens = _lengths(case, "keys")
    return [(n, min(n, int(round(math.exp(r.uniform(math.log(case["nmin"]), math.log(case["nmax"]))))))) for n in lens]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    return {"attend": _prepare_attend, "prologue": _prepare_rotary, "qkv": _prepare_rotary, "copy": _prepare_copy,
            "beam": _prepare_rows, "compact": _prepare_rows}[case["op"]](case, _gen(seed))


def _tables(g, counts, pages, first=0):
    """A page table whose rows take counts[i] pages each, scattered over the pool from page `first` on; -1 behind."""
    width = max(1, max(counts))
    order = (torch.randperm(pages - first, generator=g, device="cuda") + first).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    return table


def _prepare_attend(case, g):
    dt, ps = TYPES[case["dt"]], case["ps"]
    chunks = _chunks(case)
    lens, news = [c[0] for c in chunks], [c[1] for c in chunks]
    counts = [-(-n // ps) for n in lens]
    pages = sum(counts) + 5
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s = {"op": "attend", "case": case, "table": _tables(g, counts, pages), "lens": _ints(lens), "starts": _ints(starts),
         "ps": ps, "scale": case["d"] ** -0.5, "causal": case["causal"], "window": case["window"] if case["causal"] else 0,
         "lmax": max(lens), "nmax": max(news), "fp8": case["fp8"], "inv": 64.0}
    # heads as the QK-norm prologue leaves them; queries sharp enough that a few keys carry most of a row
    s["q"] = (2.0 * _normal(g, starts[-1], case["hq"], case["d"])).to(dt)
    s["k"] = _normal(g, pages * ps, case["hk"], case["d"]).to(dt)
    s["v"] = _normal(g, pages * ps, case["hk"], case["d"]).to(dt)
    s["one"] = case["nmax"] == 1
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        s["out"] = torch.empty(s["q"].shape, dtype=torch.uint8 if case["fp8"] else dt, device="cuda")
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if case["lse"] else None
        s["work"] = edge_ops.paged_attention_workspace(s["q"], s["k"])
    return s


def _sections(rot):
    """A split of rot/2 pairs into time, height and width like 1 : 1.5 : 1.5, that can also be dealt in turn."""
    half = rot // 2
    h = half * 5 // 16
    return (half - 2 * h, h, h)


def _prepare_rotary(case, g):
    dt, t, hq, hk, d, rot = TYPES[case["dt"]], case["t"], case["hq"], case["hk"], case["d"], case["rot"]
    s = {"op": case["op"], "case": case, "sections": _sections(rot), "order": case["order"], "rot": rot,
         "offset": case["offset"], "eps": 1e-6, "hq": hq, "hk": hk}
    cache = 32768
    angle = torch.arange(cache, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
        -2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    # frames of 8 x 8 patches one after the other, somewhere in the cache; one token in 97 is padding (-1 on every axis)
    i = torch.arange(t, device="cuda")
    start = int(torch.randint(0, cache - 8192, (1,), generator=g, device="cuda"))
    grid = torch.stack([i // 64, i // 8 % 8, i % 8]) + start
    s["positions"] = torch.where(i % 97 == 96, torch.full_like(grid, -1), grid).contiguous()
    w = 0.02 * _normal(g, 2, d) + (0.0 if case["offset"] else 1.0)
    s["wq"], s["wk"] = w[0].to(dt), w[1].to(dt)
    if case["op"] == "prologue":
        s["q"], s["k"] = _normal(g, t, hq, d).to(dt), _normal(g, t, hk, d).to(dt)
        if own:
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        n = case["slots"]
        s["qkv"] = _normal(g, t, (hq + 2 * hk) * d).to(dt)
        s["k_cache"], s["v_cache"] = _normal(g, n, hk, d).to(dt), _normal(g, n, hk, d).to(dt)
        # slot 0 is nobody's: padding tokens (-1) write nothing
        slots = torch.randperm(n - 1, generator=g, device="cuda")[:t] + 1
        s["slots"] = torch.where(i % 97 == 96, torch.full_like(slots, -1), slots)
        if own:
            s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
    return s


def _pool(case, g):
    """All caches of a model as one allocation, [caches, slots, heads, head size]."""
    shape = (case["caches"], case["pages"] * case["ps"], case["hk"], case["d"])
    return _normal(g, *shape).to(TYPES[case["dt"]])


def _hold(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        s["caches"] = edge_ops.PageCaches(list(s["pool"]), s["ps"])
    return s


def _prepare_copy(case, g):
    order = torch.randperm(case["pages"], generator=g, device="cuda").to(torch.int32)
    n = case["n"]
    return _hold({"op": "copy", "case": case, "pool": _pool(case, g), "ps": case["ps"],
                  "src": order[:n].contiguous(), "dst": order[n:2 * n].contiguous()})


def _prepare_rows(case, g):
    ps, lens = case["ps"], _lengths(case, "rows")
    counts = [-(-n // ps) for n in lens]
    s = {"op": case["op"], "case": case, "pool": _pool(case, g), "ps": ps}
    s["table"] = _tables(g, counts + [max(counts)], case["pages"])[:-1].contiguous()
    s["lens"] = _ints(lens)
    s["refs"] = torch.zeros(case["pages"], dtype=torch.int32, device="cuda")
    held = s["table"].flatten()
    s["refs"].index_add_(0, held.clamp(min=0).long(), (held >= 0).int())
    if case["op"] == "beam":
        half = max(1, case["rows"] // 2)
        order = torch.randperm(case["rows"], generator=g, device="cuda").to(torch.int32)
        s["children"] = order[:half].contiguous()
        pick = torch.randint(0, case["rows"] - half, (half,), generator=g, device="cuda") + half
        s["parents"] = order[pick].contiguous()
    else:
        # the second half of the rows shares the first page of the first row (a common prefix)
        s["table"][case["rows"] // 2:, 0] = s["table"][0, 0]
        s["refs"].zero_()
        held = s["table"].flatten()
        s["refs"].index_add_(0, held.clamp(min=0).long(), (held >= 0).int())
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        if own:
            from memory_bound_decode_qk_gb300 import edge_ops

            s["work"] = edge_ops.pages_compact_workspace(s["refs"])
    return _hold(s)


# ---------------------------------------------------------------- one pass

def run(state):
    return _RUN[state["op"]](state)


def _attend(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        out = edge_ops.paged_attention(
            s["q"], s["k"], s["v"], s["table"], s["lens"], page_size=s["ps"], q_starts=None if s["one"] else s["starts"],
            scale=s["scale"], causal=s["causal"], window=s["window"], out=s["out"], lse=s["lse"], fp8=s["fp8"],
            inv_scale=s["inv"], workspace=s["work"])
        if s["fp8"]:
            out = out.view(torch.float8_e4m3fn)
        return out if s["lse"] is None else (out, s["lse"])
    b, n, m, ps = s["lens"].numel(), s["nmax"], s["lmax"], s["ps"]
    q, hk, d = s["q"], s["k"].shape[1], s["q"].shape[2]
    g = q.shape[1] // hk
    j = torch.arange(m, device=q.device)
    page = s["table"].long()[:, j // ps]
    slot = page.clamp(min=0) * ps + j % ps
    inside = (j < s["lens"][:, None]) & (page >= 0)
    k, v = s["k"][slot].float(), s["v"][slot].float()  # [b, m, hk, d]
    starts = s["starts"].long()
    row = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    take = (starts[:-1, None] + torch.arange(n, device=q.device)).clamp(max=q.shape[0] - 1)
    qs = q[take].float().view(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)
    score = (qs @ k.permute(0, 2, 3, 1)).view(b, hk, g, n, m)
    score *= s["scale"]
    at = (s["lens"].long() - starts.diff())[:, None] + torch.arange(n, device=q.device)  # [b, n]
    seen = inside[:, None, :].expand(b, n, m)
    if s["causal"]:
        seen = seen & (j <= at[:, :, None])
        if s["window"] > 0:
            seen = seen & (j > at[:, :, None] - s["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(b, hk, g * n, m) @ v.permute(0, 2, 1, 3)).view(b, hk, g, n, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    out = out.permute(0, 3, 1, 2, 4)[seq, row - starts[seq]].reshape(q.shape)
    if s["fp8"]:
        out = (out * s["inv"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    else:
        out = out.to(q.dtype)
    if not s["case"]["lse"]:
        return out
    lse = (top + total.log()).view(b, hk * g, n).permute(0, 2, 1)
    return out, lse[seq, row - starts[seq]].contiguous()


def _pair_axis(sections, order, half):
    """The axis of each pair, as a list."""
    if order == "blocks":
        return [a for a, c in enumerate(sections) for _ in range(c)]
    return [j % len(sections) if j // len(sections) < sections[j % len(sections)] else 0 for j in range(half)]


def _angles(s):
    axis = torch.tensor(_pair_axis(s["sections"], s["order"], s["rot"] // 2), device=s["cos"].device)
    pos = s["positions"]
    ok = ((pos >= 0) & (pos < s["cos"].shape[0])).all(0)
    at = pos.clamp(0, s["cos"].shape[0] - 1)[axis].T  # [t, half]
    j = torch.arange(s["rot"] // 2, device=at.device)
    return s["cos"][at, j], s["sin"][at, j], ok


def _heads(x, w, s, cos, sin, ok):
    """RMS norm of each head rounded to its type, then the rotation of its first channels."""
    f = x.float()
    f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * (w.float() + s["offset"])
    f = f.to(x.dtype).float()
    half = s["rot"] // 2
    a, b = f[..., :half], f[..., half:2 * half]
    c, n = cos[:, None], sin[:, None]
    turned = torch.cat([a * c - b * n, b * c + a * n, f[..., 2 * half:]], -1)
    return torch.where(ok[:, None, None], turned, f).to(x.dtype)


def _prologue(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        return edge_ops.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["cos"], s["sin"],
                                     rotary_dim=s["rot"], weight_offset=s["offset"], eps=s["eps"], q_out=s["q_out"],
                                     k_out=s["k_out"], sections=s["sections"], axis_order=s["order"])
    turn = _angles(s)
    return _heads(s["q"], s["wq"], s, *turn), _heads(s["k"], s["wk"], s, *turn)


def _qkv(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        q = edge_ops.qkv_rope_cache(s["qkv"], s["hq"], s["hk"], s["wq"], s["wk"], s["positions"], s["cos"], s["sin"],
                                    s["slots"], s["k_cache"], s["v_cache"], rotary_dim=s["rot"],
                                    weight_offset=s["offset"], eps=s["eps"], q_out=s["q_out"], sections=s["sections"],
                                    axis_order=s["order"])
        return q, s["k_cache"], s["v_cache"]
    t, hq, hk = s["qkv"].shape[0], s["hq"], s["hk"]
    x = s["qkv"].view(t, hq + 2 * hk, -1)
    turn = _angles(s)
    q = _heads(x[:, :hq], s["wq"], s, *turn)
    k = _heads(x[:, hq:hq + hk], s["wk"], s, *turn)
    valid, at = (s["slots"] >= 0)[:, None, None], s["slots"].clamp(min=0)
    s["k_cache"][at] = torch.where(valid, k, s["k_cache"][at])
    s["v_cache"][at] = torch.where(valid, x[:, hq + hk:], s["v_cache"][at])
    return q, s["k_cache"], s["v_cache"]


def _by_page(s):
    pool = s["pool"]
    return pool.view(pool.shape[0], -1, s["ps"], *pool.shape[2:])


def _copy(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        edge_ops.pages_copy(s["caches"], s["src"], s["dst"])
        return s["pool"]
    pool = _by_page(s)
    pool[:, s["dst"].long()] = pool[:, s["src"].long()]
    return s["pool"]


def _beam(s):
    table, lens, refs, ps = s["table"], s["lens"], s["refs"], s["ps"]
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        edge_ops.pages_free(table, lens, refs, s["children"])
        status = edge_ops.pages_fork(s["caches"], table, lens, refs, s["parents"], s["children"])
        return table, lens, refs, status, s["pool"]
    children, parents = s["children"].long(), s["parents"].long()
    old = table[children]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().int())
    table[children] = -1
    lens[children] = 0
    held = lens[parents].long()
    full, part = held // ps, held % ps != 0
    free = torch.sort((refs != 0).int(), stable=True).indices
    fresh = free[(part.long().cumsum(0) - 1).clamp(min=0)].int()
    rows = table[parents]
    column = torch.arange(table.shape[1], device=table.device)
    row = torch.where(column < full[:, None], rows, torch.where(
        (column == full[:, None]) & part[:, None], fresh[:, None], torch.full_like(rows, -1)))
    table[children] = row
    lens[children] = held.int()
    refs.index_add_(0, row.clamp(min=0).flatten().long(), (row >= 0).flatten().int())
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    src, dst = torch.where(part, last, rows[:, 0].long()), torch.where(part, fresh.long(), rows[:, 0].long())
    pool = _by_page(s)
    pool[:, dst] = pool[:, src]
    return table, lens, refs, torch.zeros_like(s["children"]), s["pool"]


def _compact(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        edge_ops.pages_compact(s["caches"], s["table"], s["refs"], table_out=s["table_out"], refs_out=s["refs_out"],
                               workspace=s["work"])
        return s["table_out"], s["refs_out"], s["pool"]
    refs, table = s["refs"], s["table"]
    page = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    count = live.sum()
    # the k-th free page below `count` takes the k-th page in use from `count` on
    hole, stray = ~live & (page < count), live & (page >= count)
    holes = torch.sort((~hole).int(), stable=True).indices
    strays = torch.sort((~stray).int(), stable=True).indices
    new = torch.where(stray, holes[(stray.long().cumsum(0) - 1).clamp(min=0)], page)
    origin = torch.where(hole, strays[(hole.long().cumsum(0) - 1).clamp(min=0)], page)
    s["table_out"].copy_(torch.where(table >= 0, new[table.clamp(min=0).long()].int(), table))
    s["refs_out"].copy_(torch.where(page < count, refs[origin], torch.zeros_like(refs)))
    pool = _by_page(s)
    pool.copy_(pool[:, origin])
    return s["table_out"], s["refs_out"], s["pool"]


_RUN = {"attend": _attend, "prologue": _prologue, "qkv": _qkv, "copy": _copy, "beam": _beam, "compact": _compact}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = SIZE[case["dt"]]
    op = case["op"]
    if op == "attend":
        keys = pairs = rows = 0
        window = case["window"] if case["causal"] else 0
        for length, new in _chunks(case):
            rows += new
            first = max(0, length - new + 1 - window) if window else 0
            keys += length - first
            if not case["causal"]:
                pairs += new * length
            elif not window:
                pairs += new * length - new * (new - 1) // 2
            else:
                pairs += sum(min(window, length - new + i + 1) for i in range(new))
        heads = rows * case["hq"] * case["d"]
        return {"bytes": heads * size + heads * (1 if case["fp8"] else size) + 2 * keys * case["hk"] * case["d"] * size
                + (4 * rows * case["hq"] if case["lse"] else 0), "flops": 4 * pairs * case["hq"] * case["d"]}
    if op in ("prologue", "qkv"):
        heads = case["hq"] + case["hk"] * (1 if op == "prologue" else 2)
        t, d = case["t"], case["d"]
        rows = 2 * min(t, 64 * 3) * case["rot"] // 2 * 4  # cos and sin of the distinct positions, about
        return {"bytes": 2 * t * heads * d * size + 3 * 8 * t + rows + (8 * t if op == "qkv" else 0),
                "flops": t * heads * (4 * d + 3 * case["rot"])}
    page = case["caches"] * case["ps"] * case["hk"] * case["d"] * size
    if op == "copy":
        return {"bytes": 2 * case["n"] * page + 8 * case["n"], "flops": 0}
    counts = [-(-n // case["ps"]) for n in _lengths(case, "rows")]
    if op == "beam":
        copies = max(1, case["rows"] // 2)
        return {"bytes": 2 * copies * page + 4 * case["pages"] + 16 * copies * max(counts), "flops": 0}
    # pages in use lie anywhere in the pool: those past their number move
    used = sum(counts) - case["rows"] // 2
    moved = used * (1 - used / case["pages"])
    return {"bytes": 2 * moved * page + 8 * case["pages"] + 8 * case["rows"] * max(counts), "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] in ("prologue", "qkv"):
        return _exact_rotary(case, s)
    return None  # whole numbers and moved data


def _exact_attend(case, s):
    ps, out, stats = s["ps"], [], []
    at = 0
    for b, (length, new) in enumerate(_chunks(case)):
        pages = s["table"][b, :-(-length // ps)].long()
        slots = (pages[:, None] * ps + torch.arange(ps, device="cuda")).reshape(-1)[:length]
        q = s["q"][at:at + new].double().transpose(0, 1)  # [hq, new, d]
        at += new
        i = torch.arange(length - new, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hidden = torch.zeros(new, length, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > i
            if case["window"]:
                hidden |= j <= i - case["window"]
        rows, lses = [], []
        for h in range(case["hq"]):
            kv = h // (case["hq"] // case["hk"])
            x = q[h] @ s["k"][slots, kv].double().T / math.sqrt(case["d"])
            x = x.masked_fill(hidden, -math.inf)
            lses.append(torch.logsumexp(x, -1))
            rows.append(torch.softmax(x, -1) @ s["v"][slots, kv].double())
        out.append(torch.stack(rows, 1))
        stats.append(torch.stack(lses, 1))
    out = torch.cat(out)
    if case["fp8"]:
        out = (out * s["inv"]).clamp(-448.0, 448.0)
    return (out, torch.cat(stats)) if case["lse"] else out


def _exact_rotary(case, s):
    t, hq, hk, half, c = case["t"], case["hq"], case["hk"], case["rot"] // 2, s["sections"]
    if case["op"] == "prologue":
        x = torch.cat([s["q"], s["k"]], 1)
    else:
        x = s["qkv"].view(t, hq + 2 * hk, -1)[:, :hq + hk]
    weight = torch.cat([s["wq"].double().expand(hq, -1), s["wk"].double().expand(hk, -1)]) + case["offset"]
    y = x.double() / (x.double() ** 2).mean(-1, keepdim=True).add(s["eps"]).sqrt() * weight
    y = y.to(x.dtype).double()
    pos = s["positions"]
    index = torch.zeros(half, dtype=torch.long, device="cuda")
    if case["order"] == "blocks":
        index[c[0]:c[0] + c[1]] = 1
        index[c[0] + c[1]:] = 2
    else:
        index[1:3 * c[1]:3] = 1
        index[2:3 * c[2]:3] = 2
    good = (pos.amin(0) >= 0) & (pos.amax(0) < s["cos"].shape[0])
    at = torch.where(good, pos, torch.zeros_like(pos))[index, :].T
    phase = torch.complex(s["cos"].double().gather(0, at), s["sin"].double().gather(0, at))[:, None]
    z = torch.complex(y[..., :half], y[..., half:2 * half]) * phase
    turned = torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)
    y = torch.where(good[:, None, None], turned, y)
    if case["op"] == "prologue":
        return y[:, :hq], y[:, hq:]
    return y[:, :hq], None, None
