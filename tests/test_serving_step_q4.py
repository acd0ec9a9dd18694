"""The paged 4-bit cache calls together, as a serving step strings them: page table, norm and
rotation, cache append and decode for an FA layer and an SA layer on a ring, eager and captured."""
import math

import numpy as np
import pytest
import torch

import q4_reference as ref
from sparse_attention_flux_b200.flux import Context, kv_q4_pool_shape

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 8, 2, 128, 32
SINK, WINDOW, BLOCK = 1, 3, 64                      # the SA layer's blocks
RING = (SINK * BLOCK // PAGE, WINDOW * BLOCK // PAGE)   # and its pages
LENS = [5, 700, 0, 64, 1]


class Server:
    """Two layers (FA on an ever growing cache, SA on a ring), five requests, one ctx."""

    def __init__(self, steps):
        g = torch.Generator(device="cuda").manual_seed(1)
        top = [n + steps for n in LENS]
        self.ctx = Context(0, 16 << 20)
        self.width = -(-max(top) // PAGE)
        need = [sum(-(-n // PAGE) for n in top), sum(min(-(-n // PAGE), sum(RING)) for n in top)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.free = [torch.randperm(n + 2, generator=g, device="cuda").int() for n in need]
        self.pool = [torch.full(kv_q4_pool_shape(n + 2, HKV, PAGE, D), 0xFF, dtype=torch.uint8, device="cuda")
                     for n in need]
        self.table = [torch.full((5, self.width), -1, **i32) for _ in range(2)]
        self.cursor = [torch.zeros(1, **i32) for _ in range(2)]
        self.mode = torch.tensor([1, 0], dtype=torch.uint8, device="cuda")
        self.old, self.new = torch.zeros(5, **i32), torch.zeros(5, **i32)
        self.inv = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        self.w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
        self.out = [torch.zeros((5, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.lse = [torch.zeros((5, HQ), device="cuda") for _ in range(2)]
        self.k, self.v = [[None] * 5, [None] * 5], [[None] * 5, [None] * 5]     # what was written, per layer

    def buffers(self, n):
        return [(torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"))
                for _ in range(2)]

    def append(self, layer, qkv, slots, pos):
        """Table, norm + rotation in place, cache write."""
        q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
        k = qkv[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D))
        v = qkv[:, (HQ + HKV) * D:].unflatten(1, (HKV, D))
        sink, window = RING if layer else (0, 0)
        self.ctx.build_page_table(self.old, self.new, self.free[layer], self.cursor[layer], self.cursor[layer],
                                  self.table[layer], slots, pos, PAGE, sink, window)
        self.ctx.qk_norm_rope(q, k, q, k, pos, self.inv, *self.w)
        self.ctx.kv_write_q4(k, v, slots, self.pool[layer])
        return q, k, v

    def decode(self, layer, q):
        self.ctx.attn_decode_q4(q, self.pool[layer], self.table[layer], self.new, self.out[layer],
                                1 / math.sqrt(D), layer_mode=self.mode, layer=layer, sink_blocks=SINK,
                                window_blocks=WINDOW, block=BLOCK, lse=self.lse[layer])

    def remember(self, layer, k, v, counts):
        for b, (kk, vv) in enumerate(zip(k.split(counts), v.split(counts))):
            for mem, x in ((self.k, kk), (self.v, vv)):
                x = ref.f64(x)
                mem[layer][b] = x if mem[layer][b] is None else np.concatenate([mem[layer][b], x])

    def check(self, layer, q, lens):
        o, lse, q = ref.f64(self.out[layer]), ref.f64(self.lse[layer]), ref.f64(q)
        for b, n in enumerate(lens):
            u = ref.live_tokens(n, layer == 0, SINK, WINDOW, BLOCK)
            k, v = ref.values(self.k[layer][b])[u], ref.values(self.v[layer][b])[u]
            for h in range(HQ):
                kv = h // (HQ // HKV)
                want, wl, tol, ltol = ref.decode_row(q[b, h], k[:, kv], v[:, kv], 1 / math.sqrt(D))
                assert np.all(np.abs(o[b, h] - want) <= tol), (layer, b, h)
                assert lse[b, h] == wl if np.isinf(wl) else abs(lse[b, h] - wl) <= ltol, (layer, b, h)


def projection(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, (HQ + 2 * HKV) * D), generator=g, device="cuda").to(torch.bfloat16)


def prompt(s):
    s.new.copy_(torch.tensor(LENS, dtype=torch.int32))
    total = sum(LENS)
    for layer, (slots, pos) in enumerate(s.buffers(total)):
        _, k, v = s.append(layer, projection(total, 10 + layer), slots, pos)
        s.ctx.check()
        want = np.concatenate([np.arange(n) for n in LENS])
        assert np.array_equal(pos.cpu().numpy(), want)
        s.remember(layer, k, v, LENS)


@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_steps(captured):
    """A ragged prompt step, then 70 decode steps (the ring wraps) of every request, an empty one
    among them; eager, and as one graph per layer pair that reads its lengths at replay."""
    steps = 70
    s = Server(steps)
    prompt(s)
    qkv = [torch.zeros((5, (HQ + 2 * HKV) * D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bufs = s.buffers(5)

    def step():
        return [(s.append(layer, qkv[layer], *bufs[layer]), s.decode(layer, qkv[layer][:, :HQ * D]
                 .unflatten(1, (HQ, D)).contiguous())) for layer in range(2)]

    graph = None
    if captured:
        s.old.copy_(s.new)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                  # old == new: hands out nothing, writes nothing
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    lens = list(LENS)
    for i in range(steps):
        s.old.copy_(torch.tensor(lens, dtype=torch.int32))
        lens = [n + 1 for n in lens]
        s.new.copy_(torch.tensor(lens, dtype=torch.int32))
        for layer in range(2):
            qkv[layer].copy_(projection(5, 100 + 2 * i + layer))
        graph.replay() if captured else step()
        s.ctx.check()
        for layer in range(2):
            k = qkv[layer][:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D))
            v = qkv[layer][:, (HQ + HKV) * D:].unflatten(1, (HKV, D))
            s.remember(layer, k, v, [1] * 5)
            if i % 23 == 0 or i == steps - 1:
                s.check(layer, qkv[layer][:, :HQ * D].unflatten(1, (HQ, D)), lens)
    s.ctx.close()


def test_captured_steps_equal_eager_ones():
    """The same step replayed twice and run eagerly: the same bits."""
    s = Server(1)
    prompt(s)
    s.old.copy_(s.new)
    q = projection(5, 3)[:, :HQ * D].unflatten(1, (HQ, D)).contiguous()
    got = []
    for layer in range(2):
        s.decode(layer, q)
    want = [(o.clone(), l.clone()) for o, l in zip(s.out, s.lse)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer in range(2):
            s.decode(layer, q)
    for _ in range(2):
        for o, l in zip(s.out, s.lse):
            o.fill_(7), l.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got.append([(o.clone(), l.clone()) for o, l in zip(s.out, s.lse)])
    for g in got:
        for (o, l), (wo, wl) in zip(g, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    s.ctx.close()
