"""Causal attention of packed prompts over a paged cache against its formula in 64 bits.

Tolerance, per output component, with w the exact weights, E = sum w |v| and u = eps / 2 of the type: the weights are
rounded to the type before the product with V (u E); scores are fp32 sums of D products (each step at most 2^-23 of
A = scale sum |q k|, the product by the scale and the exponential's argument 2^-22 of it more) and the exponential is off
by 2^-21, which moves a weight and the sum that divides it: 2 ((D + 4) 2^-23 A + 2^-20) E; the fp32 sums over n keys
n 2^-23 E, twice for numerator and denominator; the result is rounded once (u |o|, fp16 below its normal range 2^-25).
What lies in the pages past the keys in use is NaN throughout, and pages that no key has are not in the table."""
import math
import threading

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def make(seqs, hq, hk, D, page, dtype, seed=0, std=1.0, pad=0, spare=3):
    """seqs: (keys, new tokens) of each sequence."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, DT[dtype])
    counts = [-(-k // page) for k, _ in seqs]
    pages = sum(counts) + spare
    k = torch.full((pages, hk, page, D), float("nan"), dtype=dt, device="cuda")
    v = k.clone()
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(seqs), max(max(counts), 1)), 1 << 30, dtype=torch.int32, device="cuda")   # never read
    at = 0
    for b, (n, _) in enumerate(seqs):
        if not n:
            continue
        ids = order[at:at + counts[b]]
        at += counts[b]
        table[b, :counts[b]] = ids
        for c in (k, v):
            full = torch.full((hk, counts[b] * page, D), float("nan"), dtype=dt, device="cuda")
            full[:, :n] = (std * torch.randn(hk, n, D, generator=g, device="cuda")).to(dt)
            c[ids.long()] = full.view(hk, counts[b], page, D).transpose(0, 1)
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1] + pad, hq, D, generator=g, device="cuda").to(dt)
    return dict(q=q, k=k, v=v, table=table, seqs=seqs, lens=torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda"),
                cu=torch.tensor(starts, dtype=torch.int32, device="cuda"), scale=1.0 / math.sqrt(D))


def reference(p):
    """o, and the bound of the difference, both [tokens, hq, D] in 64 bits (NaN in rows of no sequence)."""
    import torch
    q = p["q"].double()
    T, hq, D = q.shape
    hk, page = p["k"].shape[1], p["k"].shape[2]
    u = torch.finfo(p["q"].dtype).eps / 2
    o, tol = torch.full_like(q, math.nan), torch.zeros_like(q)
    at = 0
    for b, (L, n) in enumerate(p["seqs"]):
        if not n:
            continue
        ids = p["table"][b, :-(-L // page)].long()
        k, v = (p[c][ids].double().transpose(0, 1).reshape(hk, -1, D)[:, :L] for c in "kv")
        for i in range(0, n, 512):
            m = min(512, n - i)
            qb = q[at + i:at + i + m].view(m, hk, hq // hk, D).permute(1, 2, 0, 3)               # [hk, g, m, D]
            seen = torch.arange(L, device="cuda")[None] <= (L - n + i + torch.arange(m, device="cuda"))[:, None]
            z = (qb @ k[:, None].transpose(2, 3) * p["scale"]).masked_fill(~seen, -math.inf)
            w = torch.softmax(z, -1) if L else z
            w = torch.where(seen, w, torch.zeros_like(w))
            A = (qb.abs() @ k[:, None].abs().transpose(2, 3) * p["scale"] * seen).amax(-1, keepdim=True) if L else 0.0
            E = w @ v[:, None].abs()
            o[at + i:at + i + m] = (w @ v[:, None]).permute(2, 0, 1, 3).reshape(m, hq, D)
            t = (u + 2 * ((D + 4) * 2.0 ** -23 * A + 2.0 ** -20) + 2 * L * 2.0 ** -23) * E
            tol[at + i:at + i + m] = t.permute(2, 0, 1, 3).reshape(m, hq, D)
        at += n
    tiny = 2.0 ** -25 if p["q"].dtype is torch.float16 else 0.0
    return o, tol * (1 + u) + u * o.abs() + tiny


def run(p, **kw):
    import torch
    n = p["q"].shape[0] * p["q"].shape[1] * p["q"].shape[2]
    buf = torch.full((n + 64,), 7.0, dtype=p["q"].dtype, device="cuda")       # guards around the output
    o = buf[32:32 + n].view(p["q"].shape)
    fc.fuse_prompt_attention(p["q"], p["k"], p["v"], p["table"], p["cu"], p["lens"], o, p["scale"], **kw)
    assert fc.fuse_check(kw.get("stream")) == fc.FUSE_OK
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + n:] == 7).all())
    return o


def check(p, **kw):
    o = run(p, **kw)
    want, tol = reference(p)
    rows = int(p["cu"][-1])
    assert bool((o[rows:] == 7).all())                     # rows of no sequence are left as they are
    err = (o.double() - want).abs()[:rows]
    tol = tol[:rows]
    assert bool((err <= tol).all()), (float((err / tol.clamp(min=1e-30)).max()), float(err.max()),
                                      (~(err <= tol)).nonzero()[:4].tolist())
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(17, 17)], [(128, 128)], [(129, 129)], [(300, 5)], [(5, 9)], [(0, 3)], [(0, 0), (2, 2)],
                                  [(1000, 1)], [(40, 40), (0, 0), (257, 3), (7, 7), (63, 64)]])
def test_lengths(cuda_device, dtype, D, seqs):
    check(make(seqs, 8, 2, D, 16, dtype, seed=len(seqs), pad=2))


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (5, 1), (16, 16), (24, 3), (14, 2), (20, 1), (40, 2), (64, 1), (127, 1), (128, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(cuda_device, hq, hk, D):
    """Groups of one to 128 query heads, tiles that they do not fill among them."""
    check(make([(37, 37), (130, 66), (0, 0), (200, 1)], hq, hk, D, 32, "bf16", seed=hq))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("cached", [0, 1, 127, 128, 333])
def test_pages(cuda_device, page, cached):
    check(make([(cached + 5, 5), (cached + 300, 300), (cached, 0), (cached + 81, 81)], 8, 2, 128, page, "bf16", seed=page + cached))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_and_ragged(cuda_device, dtype, D):
    check(make([(20000, 33)], 8, 1, D, 64, dtype, seed=1))                        # one item over every CTA
    check(make([(20000, 1), (9000, 200), (1, 1)], 8, 2, D, 64, dtype, seed=2))
    check(make([(2500, 2500)], 8, 2, D, 128, dtype, seed=3))
    check(make([((37 * i) % 611, min((37 * i) % 611, (11 * i) % 97)) for i in range(70)], 8, 2, D, 16, dtype, seed=4, pad=7))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prompts(cuda_device, dtype, D):
    """The form of a step's code for long prompts, also with a cached part, an odd group and a second sequence."""
    check(make([(4100, 4000)], 4, 1, D, 64, dtype, seed=23))
    check(make([(3333, 3333), (3001, 2999)], 6, 2, D, 16, dtype, seed=24, std=3.0, pad=1))


def test_many_sequences(cuda_device):
    check(make([(1 + i % 70, 1 + i % 3 if i % 70 > 2 else 1) for i in range(1500)], 4, 1, 64, 16, "bf16", seed=5))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_grow_along_the_keys(cuda_device, dtype, D):
    """The running reference is replaced again and again, in parts of an item and where they join; and sharp weights."""
    import torch
    p = make([(3000, 200), (500, 500)], 4, 2, D, 16, dtype, seed=6)
    for b, (L, _) in enumerate(p["seqs"]):
        ids = p["table"][b, :-(-L // 16)].long()
        grow = torch.arange(len(ids) * 16, device="cuda").view(len(ids), 1, 16, 1) / 300.0
        p["k"][ids] = (p["k"][ids].float() * 0.3 + grow).to(p["k"].dtype)
    p["q"] = (p["q"].float() * 0.2 + 0.5).to(p["q"].dtype)
    check(p)
    p["scale"] *= 8.0
    check(p)


def test_strided_queries(cuda_device):
    """Queries as the first columns of a merged projection's rows."""
    import torch
    p = make([(90, 90), (200, 30)], 8, 2, 128, 16, "bf16", seed=7, pad=1)
    wide = torch.full((p["q"].shape[0], 12 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :8 * 128] = p["q"].view(-1, 8 * 128)
    want = check(p)
    p["q"] = wide[:, :8 * 128].unflatten(1, (8, 128))
    assert p["q"].stride(0) == 12 * 128
    assert torch.equal(run(p)[:-1], want[:-1])


def test_what_is_past_the_keys_is_not_used(cuda_device):
    """Infinities and NaN in pages past a sequence's keys, also where a page's rows precede others in its tile."""
    import torch
    p = make([(130, 130), (1, 1), (250, 3)], 8, 2, 128, 256, "bf16", seed=8)
    a = check(p)
    for c in ("k", "v"):
        p[c] = torch.where(p[c].isnan(), torch.full_like(p[c], math.inf), p[c])
    assert torch.equal(run(p), a)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tensors_on_16_byte_boundaries(cuda_device, D):
    import torch
    p = make([(300, 280), (40, 40), (129, 2)], 4, 2, D, 16, "bf16", seed=21)
    want = check(p)

    def moved(t):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        out = buf[8:].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % 32 == 16
        return out

    for c in "qkv":
        p[c] = moved(p[c])
    o = moved(torch.full_like(want, 7.0))
    fc.fuse_prompt_attention(p["q"], p["k"], p["v"], p["table"], p["cu"], p["lens"], o, p["scale"])
    assert fc.fuse_check() == fc.FUSE_OK
    assert torch.equal(o, want)


def test_wide_heads(cuda_device):
    """D = 256: strided queries, infinities past the keys, workspaces of any content, parts joined over many runs."""
    import torch
    p = make([(3000, 40), (700, 700), (1, 1), (0, 3), (260, 3)], 8, 2, 256, 32, "f16", seed=22, pad=2)
    want = check(p)
    rows = int(p["cu"][-1])
    for c in "kv":
        p[c] = torch.where(p[c].isnan(), torch.full_like(p[c], -math.inf), p[c])
    wide = torch.full((p["q"].shape[0], 9 * 256), float("nan"), dtype=p["q"].dtype, device="cuda")
    wide[:, :8 * 256] = p["q"].view(-1, 8 * 256)
    p["q"] = wide[:, :8 * 256].unflatten(1, (8, 256))
    ws = torch.full((fc.fuse_prompt_attention_workspace_bytes(rows + 2, 8, 2, 256),), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(run(p, workspace=ws), want)


def test_equal_calls_and_any_workspace(cuda_device):
    import torch
    p = make([(3000, 40), (700, 700)], 8, 2, 128, 32, "f16", seed=9)
    a = check(p)
    need = fc.fuse_prompt_attention_workspace_bytes(740, 8, 2, 128)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(run(p, workspace=ws), a) and torch.equal(run(p, workspace=ws), a)
    with pytest.raises(fc.FuseError):
        run(p, workspace=ws[:-256])


def test_captured_with_other_lengths(cuda_device):
    """A graph keeps its addresses; lengths, row numbers, table and rows may change between replays."""
    import torch
    p = make([(3000, 40), (700, 60)], 8, 2, 128, 32, "bf16", seed=10)
    other = make([(90, 35), (2900, 65)], 8, 2, 128, 32, "bf16", seed=11)
    ws = torch.empty(fc.fuse_prompt_attention_workspace_bytes(100, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(p["q"])
    pages = max(p["k"].shape[0], other["k"].shape[0])
    st = {c: torch.zeros(pages, *p["k"].shape[1:], dtype=p["k"].dtype, device="cuda") for c in "kv"}
    st["table"] = torch.zeros(2, max(p["table"].shape[1], other["table"].shape[1]), dtype=torch.int32, device="cuda")
    for c in ("q", "cu", "lens"):
        st[c] = torch.zeros_like(p[c])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fc.fuse_graph_begin(s)
    fc.fuse_prompt_attention(st["q"], st["k"], st["v"], st["table"], st["cu"], st["lens"], o, p["scale"], workspace=ws, stream=s)
    g = fc.fuse_graph_end(s)
    for x in (p, other, p):
        for c in ("q", "cu", "lens"):
            st[c].copy_(x[c])
        st["table"][:, :x["table"].shape[1]] = x["table"]
        for c in "kv":
            st[c][:x[c].shape[0]] = x[c]
        s.wait_stream(torch.cuda.current_stream())
        fc.fuse_graph_launch(g, s)
        assert fc.fuse_check(s) == fc.FUSE_OK
        want, tol = reference(x)
        assert bool(((o.double() - want).abs() <= tol).all())
    fc.fuse_graph_destroy(g)


def test_streams_and_the_modules_workspace(cuda_device):
    import torch
    p = make([(3000, 40)], 8, 2, 128, 32, "bf16", seed=12)
    want = check(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(ValueError):                       # the module's own serves the current stream only
        run(p, stream=s)
    with torch.cuda.stream(s):
        assert torch.equal(run(p), want)
    ws = torch.empty(fc.fuse_prompt_attention_workspace_bytes(40, 8, 2, 128), dtype=torch.uint8, device="cuda")
    assert torch.equal(run(p, stream=s, workspace=ws), want)


def test_two_threads_on_one_stream(cuda_device):
    import torch
    ps = [make([(3000 + 500 * i, 40)], 8, 2, 128, 32, "bf16", seed=20 + i) for i in range(2)]
    want = [check(p) for p in ps]
    outs = [[torch.zeros_like(p["q"]) for _ in range(30)] for p in ps]

    def work(p, out):
        for o in out:
            fc.fuse_prompt_attention(p["q"], p["k"], p["v"], p["table"], p["cu"], p["lens"], o, p["scale"])

    threads = [threading.Thread(target=work, args=a) for a in zip(ps, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert fc.fuse_check() == fc.FUSE_OK
    for w, out in zip(want, outs):
        assert all(torch.equal(o, w) for o in out)


def test_out_of_range_in_device_memory(cuda_device):
    """Bad pages count as zeros; lengths and rows are taken into range; all are reported."""
    import torch
    p = make([(100, 100), (60, 20)], 4, 2, 64, 16, "bf16", seed=13)
    o = torch.zeros_like(p["q"])

    def call(**kw):
        a = {**p, **kw}
        fc.fuse_prompt_attention(a["q"], a["k"], a["v"], a["table"], a["cu"], a["lens"], o, a["scale"])
        status = fc.fuse_check()
        assert fc.fuse_check() == fc.FUSE_OK
        return status

    table = p["table"].clone()
    table[0, 2], table[1, 0] = -5, p["k"].shape[0]
    assert call(table=table) == fc.FUSE_EINDEX
    zero = {c: torch.cat([p[c], torch.zeros_like(p[c][:1])]) for c in "kv"}
    table[0, 2] = table[1, 0] = p["k"].shape[0]
    want, tol = reference({**p, **zero, "table": table})
    assert bool(((o.double() - want).abs() <= tol).all())
    room = p["table"].shape[1] * 16
    q = p["table"].clone()
    q[q == 1 << 30] = 0
    assert call(lens=torch.tensor([-4, room + 1], dtype=torch.int32, device="cuda"), table=q) == fc.FUSE_EINDEX
    assert bool((o[:100] == 0).all())
    assert call(cu=torch.tensor([0, 500, 120], dtype=torch.int32, device="cuda")) == fc.FUSE_EINDEX
    assert call(cu=torch.tensor([-3, 100, 120], dtype=torch.int32, device="cuda")) == fc.FUSE_EINDEX
    assert call() == fc.FUSE_OK


def test_refusals(cuda_device):
    import torch
    p = make([(100, 100)], 4, 2, 64, 16, "bf16", seed=14)
    for bad in (dict(q=p["q"].float()), dict(cu=p["cu"][:1]), dict(lens=p["lens"].long()), dict(table=p["table"].t()),
                dict(q=p["q"].transpose(0, 1).contiguous().transpose(0, 1)), dict(v=p["v"][:1])):
        with pytest.raises(ValueError):
            run({**p, **bad})
