"""A decoding step as a model runs it: the merged projection in 4 bits, rotate-and-append, attention over
the paged cache, and the output projection with the residual joined, captured once and replayed while the
sequences grow.  Every stage of every step is compared with its formula in 64 bits on what the stage
before it left (tolerances of the single operators' tests), the cache with what the steps so far must
have written."""
import math

import pytest

import epilogue_chains_gb300 as fc
from test_paged_attention_gpu import reference as attend
from test_rope_append_gpu import reference as rotate
from test_w4_gemv_gpu import weights

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def near_projection(y, x, wq, s, z, r=None):
    import torch
    w, G = weights(wq, s, z)
    K = x.shape[1]
    want = x.double() @ w.t()
    tol = (G + K / G + 64) * 2.0 ** -22 * (x.double().abs() @ w.abs().t())
    if r is not None:
        want = want + r.double()
        tol = tol + 2.0 ** -23 * want.abs()
    u = torch.finfo(y.dtype).eps / 2
    bound = u * want.abs() + (1 + u) * tol + (2.0 ** -25 if y.dtype is torch.float16 else 0.0)
    assert bool(((y.double() - want).abs() <= bound).all())


class Layer:
    """One attention layer's weights, cache and buffers for `batch` sequences, the last `pad` of them unused."""

    def __init__(self, batch, pad, hidden, hq, hk, D, page, G, dtype, zeros, starts, prefix, steps, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = getattr(torch, DT[dtype])
        self.page, self.prefix, self.live = page, prefix, batch - pad
        width = (hq + 2 * hk) * D

        def weight(N, K):
            return (torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                    ((0.5 + torch.rand(N, K // G, generator=g, device="cuda")) * 0.2 / math.sqrt(K)).to(dt),
                    torch.randint(0, 16, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None)

        self.w_in, self.w_out = weight(width, hidden), weight(hidden, hq * D)
        per = -(-(max(starts) + steps) // page)
        shared = -(-prefix // page)
        order = torch.randperm(batch * per + shared, generator=g, device="cuda").to(torch.int32)
        self.table = order[:batch * per].view(batch, per).contiguous()
        self.ptable = order[batch * per:].contiguous() if prefix else None
        self.k, self.v = (torch.full((len(order), hk, page, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
        for ids, n in [(self.table[b], starts[b]) for b in range(self.live)] + ([(self.ptable, prefix)] if prefix else []):
            at = torch.arange(n, device="cuda")
            for c in (self.k, self.v):
                c[ids.long()[at // page], :, at % page] = torch.randn(n, hk, D, generator=g, device="cuda").to(dt)
        rot, positions = D, prefix + max(starts) + steps
        ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.x = torch.empty(batch, hidden, dtype=dt, device="cuda")
        self.qkv = torch.empty(batch, width, dtype=dt, device="cuda")
        self.q, self.o = (torch.empty(batch, hq, D, dtype=dt, device="cuda") for _ in range(2))
        self.y = torch.empty(batch, hidden, dtype=dt, device="cuda")
        self.pos, self.slots, self.lens = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(3))
        self.scale = 1.0 / math.sqrt(D)
        self.ws = torch.zeros(fc.fuse_paged_attention_workspace_bytes(batch, hq, hk, D, prefix), dtype=torch.uint8, device="cuda")
        self.at = list(starts)

    def advance(self, g):
        """The next token of every live sequence: its input, position, slot and the length with it."""
        import torch
        self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda"))
        for b in range(len(self.lens)):
            n = self.at[b]
            on = b < self.live
            self.pos[b] = self.prefix + n if on else 0
            self.slots[b] = int(self.table[b, n // self.page]) * self.page + n % self.page if on else -1
            self.lens[b] = n + 1 if on else 0
            self.at[b] += 1 if on else 0

    def step(self, interleaved, stream=None):
        fc.fuse_w4_gemv(self.x, *self.w_in[:2], self.qkv, zeros=self.w_in[2], stream=stream)
        fc.fuse_rope_append(self.qkv, self.cs, self.pos, self.slots, self.q, self.k, self.v, interleaved=interleaved, stream=stream)
        fc.fuse_paged_attention(self.q, self.k, self.v, self.table, self.lens, self.o, self.scale, prefix_table=self.ptable,
                                prefix_len=self.prefix, workspace=self.ws, stream=stream)
        fc.fuse_w4_gemv(self.o.view(self.o.shape[0], -1), *self.w_out[:2], self.y, zeros=self.w_out[2], residual=self.x, stream=stream)


@pytest.mark.parametrize("dtype,batch,pad,hq,hk,D,page,G,zeros,prefix,inter", [
    ("bf16", 1, 0, 8, 2, 128, 16, 128, False, 0, False),
    ("f16", 5, 2, 8, 8, 64, 16, 32, True, 0, True),
    ("bf16", 12, 1, 8, 1, 128, 32, 64, True, 300, False),
    ("f16", 40, 0, 16, 2, 64, 64, 64, False, 513, True),
    ("bf16", 3, 1, 4, 2, 256, 128, 128, False, 129, False),
])
def test_captured_step(cuda_device, dtype, batch, pad, hq, hk, D, page, G, zeros, prefix, inter):
    import torch
    steps = 4
    starts = [(0, 14, 31, page - 1, 200)[b % 5] for b in range(batch)]         # from nothing, over page ends
    m = Layer(batch, pad, 1024, hq, hk, D, page, G, dtype, zeros, starts, prefix, steps, seed=batch)
    gen = torch.Generator(device="cuda").manual_seed(1)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        fc.fuse_graph_begin(st)
        m.step(inter, st)
        graph = fc.fuse_graph_end(st)
    for _ in range(steps):
        m.advance(gen)
        k0, v0 = m.k.clone(), m.v.clone()
        torch.cuda.synchronize()
        fc.fuse_graph_launch(graph, st)
        torch.cuda.synchronize()
        assert fc.fuse_check() == fc.FUSE_OK
        near_projection(m.qkv, m.x, *m.w_in)
        want, qm, kk, km, vv = rotate(m.qkv, m.cs, m.pos, m.slots, m.q, k0, v0, inter)
        u = torch.finfo(m.q.dtype).eps / 2
        tiny = 2.0 ** -25 if dtype == "f16" else 0.0
        assert bool(((m.q.double() - want).abs() <= u * want.abs() + (1 + u) * 2.0 ** -22 * qm + tiny).all())
        fresh = km > 0
        assert bool(((m.k.double() - kk).abs() <= u * kk.abs() + (1 + u) * 2.0 ** -22 * km + tiny)[fresh].all())
        assert torch.equal(m.k[~fresh].view(torch.int16), k0[~fresh].view(torch.int16))
        live = m.slots[m.slots >= 0].long()
        assert torch.equal(m.v[live // page, :, live % page].double(), vv[live // page, :, live % page])
        o, tol = attend(dict(q=m.q, k=m.k, v=m.v, table=m.table, lens=m.lens, ptable=m.ptable, prefix=prefix, scale=m.scale))
        assert bool(((m.o.double() - o).abs() <= tol).all())
        near_projection(m.y, m.o.view(batch, -1), *m.w_out, r=m.x)
        # the same step once more, outside the graph: the same slots again, so the same bits
        y = m.y.clone()
        with torch.cuda.stream(st):
            m.step(inter, st)
        torch.cuda.synchronize()
        assert torch.equal(m.y, y)
    fc.fuse_graph_destroy(graph)


def test_two_layers_share_a_workspace(cuda_device):
    """Two captured layers of different shapes with one workspace, replayed in turn on one stream."""
    import torch
    steps = 3

    def make():
        return [Layer(4, 1, 512, 8, 2, 64, 16, 64, "bf16", True, [3, 40, 0, 7], 0, steps, 3),
                Layer(33, 0, 512, 8, 8, 64, 16, 64, "bf16", False, [b * 9 for b in range(33)], 200, steps, 4)]

    want = []
    for share in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(2)
        st = torch.cuda.Stream()
        ms = make()
        ws = max((m.ws for m in ms), key=lambda w: w.numel())
        graphs = []
        torch.cuda.synchronize()
        for m in ms:
            if share:
                m.ws = ws
            with torch.cuda.stream(st):
                fc.fuse_graph_begin(st)
                m.step(False, st)
                graphs.append(fc.fuse_graph_end(st))
        got = []
        for _ in range(steps):
            for m in ms:
                m.advance(gen)
            torch.cuda.synchronize()
            for g in graphs:
                fc.fuse_graph_launch(g, st)
            torch.cuda.synchronize()
            got += [m.y.clone() for m in ms]
        assert fc.fuse_check() == fc.FUSE_OK
        for g in graphs:
            fc.fuse_graph_destroy(g)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once(cuda_device):
    """Steps of two layers on two streams, each with a workspace of its own, give the bits of the same steps one after
    the other."""
    import torch

    def make():
        return [Layer(40, 0, 1024, 16, 4, 128, 32, 128, "bf16", False, [b * 11 for b in range(40)], 700, 1, 5),
                Layer(12, 1, 1024, 8, 8, 64, 16, 32, "bf16", True, [b * 50 for b in range(12)], 0, 1, 6)]

    gen = torch.Generator(device="cuda").manual_seed(3)
    ms = make()
    for m in ms:
        m.advance(gen)
    want = []
    for m in ms:
        m.step(False)
        torch.cuda.synchronize()
        want.append((m.o.clone(), m.y.clone()))
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(25):
        for m, st in zip(ms, streams):
            with torch.cuda.stream(st):
                m.o.zero_()
                m.step(False, st)
        torch.cuda.synchronize()
        assert fc.fuse_check() == fc.FUSE_OK
        for m, (o, y) in zip(ms, want):
            assert torch.equal(m.o, o) and torch.equal(m.y, y)
