"""A decoder layer whose linear layers run in 8 bits, as a user's program strings the calls together: norm, QKV
product, rotary and cache write, attention over the cache, quantization, output product, norm, gate and up
product, gate, down product."""
import pytest
import torch

import q8_ref as ref
from memory_bound_decode_qk_gb300 import edge_ops

pytestmark = pytest.mark.gpu

HID, HQ, HK, D, INTER, PAGE = 512, 8, 2, 64, 1088, 16


def weights(rows, k, fp8, g):
    w = torch.randn(rows, k, generator=g, device="cuda") * k ** -0.5
    y, step = ref.steps(w.double(), fp8)
    y = y.float()
    return (y.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else y.round().to(torch.int8)), step.float()


class Layer:
    def __init__(self, fp8, seqs, room, dtype):
        g = torch.Generator(device="cuda").manual_seed(11)
        self.fp8, self.dtype = fp8, dtype
        self.qkv, self.o = weights((HQ + 2 * HK) * D, HID, fp8, g), weights(HID, HQ * D, fp8, g)
        self.up, self.down = weights(2 * INTER, HID, fp8, g), weights(HID, INTER, fp8, g)
        self.n1 = (torch.randn(HID, generator=g, device="cuda") * 0.1 + 1).to(dtype)
        self.n2 = (torch.randn(HID, generator=g, device="cuda") * 0.1 + 1).to(dtype)
        pages = seqs * room
        self.k, self.v = (torch.zeros(pages * PAGE, HK, D, dtype=dtype, device="cuda") for _ in range(2))
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda").view(seqs, room)
        at = torch.arange(4096, device="cuda")[:, None] * 1e4 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
        self.cos, self.sin = at.cos().contiguous(), at.sin().contiguous()

    def step(self, x, residual, positions, slots, lens, starts):
        """x is the layer's input, added to the residual; returns the feed-forward block's output."""
        ops, f, dt = edge_ops, self.fp8, self.dtype
        c, s = ops.add_rmsnorm_q8(x, residual, self.n1, fp8=f)
        qkv = ops.matmul_q8(c, self.qkv[0], s, self.qkv[1], dtype=dt)
        q = ops.qkv_rope_cache(qkv, HQ, HK, None, None, positions, self.cos, self.sin, slots, self.k, self.v)
        o = ops.paged_attention(q, self.k, self.v, self.table, lens, page_size=PAGE, q_starts=starts)
        c, s = ops.quantize_q8(o.view(-1, HQ * D), fp8=f)
        y = ops.matmul_q8(c, self.o[0], s, self.o[1], dtype=dt)
        c, s = ops.add_rmsnorm_q8(y, residual, self.n2, fp8=f)
        y = ops.matmul_q8(c, self.up[0], s, self.up[1], dtype=dt)
        c, s = ops.glu_act_q8(y, "silu", fp8=f)
        return ops.matmul_q8(c, self.down[0], s, self.down[1], dtype=dt)

    # ---- the same in 64 bits, with the roundings that the results between calls have

    def linear(self, p, w, factor=None):
        y, step = ref.steps(p, self.fp8)
        y = y.to(torch.float8_e4m3fn).double() if self.fp8 else y.round()
        step = step if factor is None else step * factor
        return (y @ ref.values(w[0], self.fp8).T * step[:, None] * w[1].double()).to(self.dtype)

    def plain(self, x, residual, positions, slots, lens, starts, k, v):
        residual = (x.double() + residual.double()).to(self.dtype)
        eps = 1e-6
        qkv = self.linear(ref.norm_products(residual, self.n1, 0), self.qkv, ref.norm_factor(residual, eps))
        heads = qkv.view(-1, HQ + 2 * HK, D).double()
        w = torch.rsqrt(heads[:, :HQ + HK].square().mean(-1, keepdim=True) + eps)
        normed = (heads[:, :HQ + HK] * w).to(self.dtype).double()
        c, s = (z[positions].double()[:, None] for z in (self.cos, self.sin))
        lo, hi = normed[..., :D // 2], normed[..., D // 2:]
        turned = torch.cat([lo * c - hi * s, hi * c + lo * s], -1).to(self.dtype)
        k[slots], v[slots] = turned[:, HQ:], qkv.view(-1, HQ + 2 * HK, D)[:, HQ + HK:]
        out = []
        for b, n in enumerate(lens.tolist()):
            first, last = (b, b + 1) if starts is None else starts[b:b + 2].tolist()
            j = torch.arange(n, device="cuda")
            at = self.table[b].long()[j // PAGE] * PAGE + j % PAGE
            new = last - first
            for h in range(HQ):
                sc = turned[first:last, h].double() @ k[at, h // (HQ // HK)].double().T * D ** -0.5
                sc = sc.masked_fill(j[None] > torch.arange(n - new, n, device="cuda")[:, None], -float("inf"))
                out.append(torch.softmax(sc, -1) @ v[at, h // (HQ // HK)].double())
            out[-HQ:] = [torch.stack(out[-HQ:], 1)]
        o = torch.cat(out).to(self.dtype).view(-1, HQ * D)
        y = self.linear(o.double(), self.o)
        residual = (y.double() + residual.double()).to(self.dtype)
        y = self.linear(ref.norm_products(residual, self.n2, 0), self.up, ref.norm_factor(residual, eps))
        return self.linear(ref.gate_products(y, "silu")[0], self.down), residual


def near(got, want):
    """The chain rounds to 8 bits four times.  A code that falls to the other side of a tie for a 16-bit rounding
    before it differs by one step, at most 2^-3 (E4M3) of one of the hundreds of terms of every sum behind it; half a step
    of the 16-bit results (2^-8) moves about one E4M3 code in sixteen and one int8 code in four.  In the 2-norm of the
    result that leaves less than 2^-5 for either (four stages of at most 2^-8 + 2^-3 / 16 relative to the
    largest sum, each passed on with a gain of about one)."""
    d = (got.double() - want.double()).norm() / want.double().norm()
    assert d <= 2.0 ** -5, d.item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_and_steps(fp8, dtype):
    seqs, room = 3, 8
    layer = Layer(fp8, seqs, room, dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [70, 1, 33]
    k, v = layer.k.clone(), layer.v.clone()

    def batch(news, lens):
        pos, slot = [], []
        for b, (n, m) in enumerate(zip(news, lens)):
            for p in range(m - n, m):
                pos.append(p)
                slot.append(layer.table[b, p // PAGE].item() * PAGE + p % PAGE)
        t = len(pos)
        starts = torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        return (torch.randn(t, HID, generator=g, device="cuda").to(dtype),
                torch.randn(t, HID, generator=g, device="cuda").to(dtype), torch.tensor(pos, device="cuda"),
                torch.tensor(slot, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"), starts)

    x, r, pos, slot, ln, starts = batch(lens, lens)  # the prompts
    want, want_r = layer.plain(x, r, pos, slot, ln, starts, k, v)
    near(layer.step(x, r, pos, slot, ln, starts), want)
    near(r, want_r)
    for _ in range(3):  # then a token for each
        lens = [n + 1 for n in lens]
        x, r, pos, slot, ln, _ = batch([1] * seqs, lens)
        want, want_r = layer.plain(x, r, pos, slot, ln, None, k, v)
        near(layer.step(x, r, pos, slot, ln, None), want)
        near(r, want_r)


@pytest.mark.parametrize("fp8", [False, True])
def test_step_in_a_graph_and_on_another_stream(fp8):
    layer = Layer(fp8, 4, 4, torch.bfloat16)
    x, r0 = (torch.randn(4, HID, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = torch.tensor([40, 3, 0, 17], device="cuda")
    slot = layer.table[torch.arange(4, device="cuda"), pos // PAGE].long() * PAGE + pos % PAGE
    ln = (pos + 1).int()
    layer.k.normal_()
    layer.v.normal_()
    r = r0.clone()
    eager = layer.step(x, r, pos, slot, ln, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = r0.clone()
        assert torch.equal(layer.step(x, again, pos, slot, ln, None), eager)
    torch.cuda.current_stream().wait_stream(side)
    held = r0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x, held, pos, slot, ln, None)
    for _ in range(2):
        held.copy_(r0)
        graph.replay()
        assert torch.equal(out, eager) and torch.equal(held, r)
