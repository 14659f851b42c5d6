"""The operators of a prompt together: 4-bit projections of all tokens, rotary positions with the append to the paged
cache, attention of the packed prompts, the output projection with its residual, the gate of the MLP, and the log
probabilities of the prompt's own tokens; the whole of it as one captured graph, replayed with a second turn."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, HID, MLP, VOCAB = 8, 2, 64, 16, 512, 768, 1000


def quantized(w):
    import torch
    q = torch.empty(w.shape[0], w.shape[1] // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(fc.fuse_mxfp4_scale_bytes(*w.shape), dtype=torch.uint8, device="cuda")
    fc.fuse_mxfp4_quantize(w, q, s)
    v = torch.empty_like(w)
    fc.fuse_mxfp4_dequantize(q, s, v)
    return q, s, v.double()


def values(x):
    """What x stands for in 4 bits, by the library's own round trip (its definition is tested elsewhere)."""
    return quantized(x.contiguous())[2]


class Layer:
    def __init__(self, tokens, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return quantized((torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).bfloat16())
        self.wqkv, self.wo = weight((HQ + 2 * HK) * D, HID), weight(HID, HQ * D)
        self.wgu, self.wd, self.head = weight(2 * MLP, HID), weight(HID, MLP), weight(VOCAB, HID)
        ang = torch.arange(4096, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, device="cuda") / (D / 2))
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.kc, self.vc = (torch.full((64, HK, PAGE, D), float("nan"), **bf) for _ in range(2))
        self.table = torch.randperm(64, generator=g, device="cuda").int().view(2, 32)
        T = tokens
        self.x, self.qkv, self.q, self.o = torch.zeros(T, HID, **bf), torch.zeros(T, (HQ + 2 * HK) * D, **bf), torch.zeros(T, HQ, D, **bf), torch.zeros(T, HQ, D, **bf)
        self.h, self.gu, self.act, self.y, self.logits = (torch.zeros(T, n, **bf) for n in (HID, 2 * MLP, MLP, HID, VOCAB))
        self.pos, self.slots, self.tokens = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(3))
        self.cu, self.lens = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        self.lp, self.H = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
        self.tl, self.ti = torch.zeros(T, 4, device="cuda"), torch.zeros(T, 4, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(fc.fuse_prompt_attention_workspace_bytes(T, HQ, HK, D), dtype=torch.uint8, device="cuda")
        self.buf = {n: (torch.empty(T, n // 2, dtype=torch.uint8, device="cuda"),
                        torch.empty(fc.fuse_mxfp4_scale_bytes(T, n), dtype=torch.uint8, device="cuda")) for n in (HID, HQ * D, MLP)}

    def project(self, x, w, y, s, **kw):
        xq, xs = self.buf[x.shape[1]]
        fc.fuse_mxfp4_quantize(x, xq, xs, stream=s)
        fc.fuse_mxfp4_gemm(xq, xs, w[0], w[1], y, stream=s, **kw)

    def step(self, s):
        T = self.x.shape[0]
        self.project(self.x, self.wqkv, self.qkv, s)
        fc.fuse_rope_append(self.qkv, self.cs, self.pos, self.slots, self.q, self.kc, self.vc, stream=s)
        fc.fuse_prompt_attention(self.q, self.kc, self.vc, self.table, self.cu, self.lens, self.o, 1 / math.sqrt(D), workspace=self.ws, stream=s)
        self.project(self.o.view(T, HQ * D), self.wo, self.h, s, residual=self.x)
        self.project(self.h, self.wgu, self.gu, s)
        self.silu(s)
        self.project(self.act, self.wd, self.y, s, residual=self.h)
        self.project(self.y, self.head, self.logits, s)
        fc.fuse_token_logprobs(self.logits, self.tokens, self.lp, entropy=self.H, top_logprob=self.tl, top_index=self.ti, stream=s)

    def silu(self, s):
        fc.fuse_silu_mul(self.gu[:, :MLP], self.gu[:, MLP:], self.act, stream=s)


def near(got, want, rel):
    """Root mean square difference within `rel` of the values' own."""
    d = (got.double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
    assert float(d) <= rel, float(d)


def test_two_turns_of_a_batch(cuda_device):
    """Every stage against its formula in 64 bits from the stage's own inputs: one rounding to bf16 is 2^-9 (rms at most
    2^-8 / sqrt(3)), two of them (attention's weights and its output) 2^-8."""
    import torch
    T = 150
    L = Layer(T)
    g = torch.Generator(device="cuda").manual_seed(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fc.fuse_graph_begin(s)
    L.step(s)
    graph = fc.fuse_graph_end(s)
    before = [0, 0]
    for new in ([100, 50], [37, 113]):
        L.x.copy_(torch.randn(T, HID, generator=g, device="cuda"))
        L.tokens.copy_(torch.randint(0, VOCAB, (T,), generator=g, device="cuda", dtype=torch.int32))
        pos = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)]).cuda()
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(new)).cuda()
        L.pos.copy_(pos)
        L.slots.copy_(L.table[seq, pos // PAGE] * PAGE + pos % PAGE)
        before = [b + n for b, n in zip(before, new)]
        L.cu.copy_(torch.tensor([0, new[0], T]))
        L.lens.copy_(torch.tensor(before))
        s.wait_stream(torch.cuda.current_stream())
        fc.fuse_graph_launch(graph, s)
        assert fc.fuse_check(s) == fc.FUSE_OK

        near(L.qkv, values(L.x) @ L.wqkv[2].t(), 2.0 ** -8)
        for b in range(2):
            at = slice(0, new[0]) if b == 0 else slice(new[0], T)
            k, v = (c[L.table[b].long()].double().transpose(0, 1).reshape(HK, -1, D)[:, :before[b]] for c in (L.kc, L.vc))
            assert not bool(k.isnan().any())
            q = L.q[at].double().view(-1, HK, HQ // HK, D).permute(1, 2, 0, 3)
            z = q @ k[:, None].transpose(2, 3) / math.sqrt(D)
            n = new[b]
            z = z + torch.full((n, before[b]), -math.inf, device="cuda", dtype=z.dtype).triu(before[b] - n + 1)
            near(L.o[at], (torch.softmax(z, -1) @ v[:, None]).permute(2, 0, 1, 3).reshape(n, HQ, D), 2.0 ** -7)
        near(L.h, values(L.o.view(T, -1)) @ L.wo[2].t() + L.x.double(), 2.0 ** -8)
        near(L.gu, values(L.h) @ L.wgu[2].t(), 2.0 ** -8)
        gate, up = L.gu[:, :MLP].double(), L.gu[:, MLP:].double()
        near(L.act, gate * torch.sigmoid(gate) * up, 2.0 ** -8)
        near(L.y, values(L.act) @ L.wd[2].t() + L.h.double(), 2.0 ** -8)
        near(L.logits, values(L.y) @ L.head[2].t(), 2.0 ** -8)
        lp = torch.log_softmax(L.logits.double(), -1)
        near(L.lp, lp.gather(1, L.tokens.long()[:, None])[:, 0], 2.0 ** -18)
        near(L.H, torch.special.entr(lp.exp()).sum(-1), 2.0 ** -18)
        best = torch.sort(L.logits.float(), dim=-1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(L.ti.long(), best)
        near(L.tl, lp.gather(1, best), 2.0 ** -18)
    fc.fuse_graph_destroy(graph)
