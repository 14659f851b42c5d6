"""Attention over a paged cache against its formula in 64 bits.

Tolerance, per output component, with w the exact weights, E = sum w |v| and u = eps / 2 of the type:
the weights are rounded to the type before the product with V (u E); scores are fp32 sums of D products
(each step at most 2^-23 of A = scale sum |q k|, the product by the scale and the exponential's argument
2^-22 of it more) and the exponential is off by 2^-21, which moves a weight and the sum that divides it:
2 ((D + 4) 2^-23 A + 2^-20) E; the fp32 sums over n keys n 2^-23 E (half a step each; accumulators that
truncate, a whole one), twice for numerator and denominator; the result is rounded once (u |o|, fp16 below its normal range
2^-25).  What lies in the pages past the keys in use is NaN throughout."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def make(lens, hq, hk, D, page, dtype, prefix=0, seed=0, std=1.0, spare=3):
    """Cache of NaN with the keys in use filled in at random pages."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, DT[dtype])
    B = len(lens)
    counts = [-(-n // page) for n in lens]
    shared = -(-prefix // page)
    pages = sum(counts) + shared + spare
    k = torch.full((pages, hk, page, D), float("nan"), dtype=dt, device="cuda")
    v = k.clone()
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(max(counts), 1)), 1 << 30, dtype=torch.int32, device="cuda")   # never read
    at = 0

    def fill(n):
        nonlocal at
        ids = order[at:at + -(-n // page)]
        at += len(ids)
        for c in (k, v):
            rows = (std * torch.randn(hk, n, D, generator=g, device="cuda")).to(dt)
            full = torch.full((hk, len(ids) * page, D), float("nan"), dtype=dt, device="cuda")
            full[:, :n] = rows
            c[ids.long()] = full.view(hk, len(ids), page, D).transpose(0, 1)
        return ids

    ptable = fill(prefix) if prefix else None
    for b, n in enumerate(lens):
        if n:
            table[b, :counts[b]] = fill(n)
    q = torch.randn(B, hq, D, generator=g, device="cuda").to(dt)
    return dict(q=q, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), ptable=ptable,
                prefix=prefix, scale=1.0 / math.sqrt(D))


def reference(p):
    """o, and the bound of the difference, both [B, hq, D] in 64 bits."""
    import torch
    q = p["q"].double()
    B, hq, D = q.shape
    hk, page = p["k"].shape[1], p["k"].shape[2]
    u = torch.finfo(p["q"].dtype).eps / 2
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        n = int(p["lens"][b])
        ids = p["table"][b, :-(-n // page)].long()
        ks, vs = [], []
        for cache, out in ((p["k"], ks), (p["v"], vs)):
            if p["prefix"]:
                out.append(cache[p["ptable"].long()].double().transpose(0, 1).reshape(hk, -1, D)[:, :p["prefix"]])
            if n:
                out.append(cache[ids].double().transpose(0, 1).reshape(hk, -1, D)[:, :n])
        if not ks:
            continue
        k, v = torch.cat(ks, 1), torch.cat(vs, 1)
        qb = q[b].view(hk, hq // hk, D)
        w = torch.softmax(qb @ k.transpose(1, 2) * p["scale"], 2)
        A = (qb.abs() @ k.abs().transpose(1, 2)).amax(2, keepdim=True) * p["scale"]
        E = w @ v.abs()
        o[b] = (w @ v).reshape(hq, D)
        keys = k.shape[1]
        tol[b] = ((u + 2 * ((D + 4) * 2.0 ** -23 * A + 2.0 ** -20) + 2 * keys * 2.0 ** -23) * E).reshape(hq, D)
    tiny = 2.0 ** -25 if p["q"].dtype is torch.float16 else 0.0
    return o, tol * (1 + u) + u * o.abs() + tiny


def run(p, **kw):
    import torch
    n = p["q"].numel()
    buf = torch.full((n + 64,), 7.0, dtype=p["q"].dtype, device="cuda")       # guards around the output
    o = buf[32:32 + n].view(p["q"].shape)
    fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o, p["scale"], prefix_table=p["ptable"],
                            prefix_len=p["prefix"], **kw)
    assert fc.fuse_check() == fc.FUSE_OK
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + n:] == 7).all())
    return o


def check(p, **kw):
    o = run(p, **kw)
    want, tol = reference(p)
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol.clamp(min=1e-30)).max()), float(err.max()))
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [0], [16], [17, 0, 15], [63, 64, 65, 1], [700], [0, 0, 3, 0]])
def test_own_keys(cuda_device, dtype, D, lens):
    check(make(lens, 8, 2, D, 16, dtype, seed=len(lens)))


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (16, 16), (24, 3), (16, 1), (20, 1), (40, 2), (64, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(cuda_device, hq, hk, D):
    """Groups of one to 32 query heads (past 16 a group takes more than one row tile)."""
    check(make([37, 130, 0, 64], hq, hk, D, 32, "bf16", seed=hq))
    check(make([37, 0], hq, hk, D, 32, "f16", prefix=150, seed=hq))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 333, 1024])
def test_pages_and_prefixes(cuda_device, page, prefix):
    check(make([5, 300, 0, 81], 8, 2, 128, page, "bf16", prefix=prefix, seed=page + prefix))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 200, 2000])
def test_prefix_only_and_types(cuda_device, dtype, D, prefix):
    """Sequences without own keys see the prefix alone; 33 sequences of four heads cross a row tile."""
    check(make([0] * 33, 4, 1, D, 16, dtype, prefix=prefix, seed=D))
    check(make([1, 0, 70], 12, 3, D, 64, dtype, prefix=prefix, seed=D))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_and_ragged(cuda_device, dtype):
    check(make([20000], 8, 1, 128, 64, dtype, seed=1))                       # one sequence over every CTA
    check(make([9000, 1, 0, 4097, 33], 16, 4, 64, 16, dtype, seed=2))
    check(make([(37 * i) % 611 for i in range(70)], 8, 2, 128, 16, dtype, seed=3))
    check(make([(37 * i) % 97 for i in range(70)], 16, 4, 128, 32, dtype, prefix=5000, seed=4))
    check(make([3000, 10], 8, 8, 256, 128, dtype, prefix=2500, seed=5))


def test_many_sequences(cuda_device):
    check(make([i % 5 for i in range(4096)], 2, 1, 64, 16, "bf16", seed=6))
    check(make([i % 3 for i in range(1000)], 2, 2, 64, 16, "f16", prefix=70, seed=7))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_peaked_scores(cuda_device, dtype):
    """Scores of wide range: the running reference moves again and again, most weights vanish."""
    check(make([900, 77], 8, 2, 128, 16, dtype, prefix=700, std=4.0, seed=8))


def test_scores_of_minus_infinity(cuda_device):
    """Keys whose score is -inf have no weight; a row that has no other key gives zeros."""
    import torch
    p = make([40, 20], 2, 1, 64, 16, "bf16", prefix=0, seed=9)
    p["q"].abs_()
    clean = run(p).clone()
    ids = p["table"][1, :2].long()
    p["k"][ids] = torch.where(p["k"][ids].isnan(), p["k"][ids], torch.full_like(p["k"][ids], -math.inf))
    o = run(p)
    assert torch.equal(o[0], clean[0]) and not o[1].any()
    ids = p["table"][0, 0].long()
    p["k"][ids, :, :8] = -math.inf                                           # the first eight keys of sequence 0
    o = run(p)
    q = dict(p, k=p["k"].clone(), v=p["v"].clone())
    q["k"][ids, :, :8], q["v"][ids, :, :8] = 0, 0
    w = torch.softmax(torch.cat([torch.full((2, 8), -math.inf, device="cuda", dtype=torch.float64), p["scale"] * (
        p["q"][0].double() @ q["k"][p["table"][0, :3].long()].double().transpose(0, 1).reshape(-1, 64)[8:40].t())], 1), 1)
    want = w @ q["v"][p["table"][0, :3].long()].double().transpose(0, 1).reshape(-1, 64)[:40]
    assert float((o[0].double() - want).abs().max()) < 2.0 ** -7 * 4         # values up to about 4, two roundings


def test_a_shared_prefix_equals_own_keys(cuda_device):
    """The same keys as a prefix and as every sequence's own ones: equal up to the tolerance's parts."""
    import torch
    p = make([0] * 5, 8, 2, 128, 16, "bf16", prefix=400, seed=10)
    with_prefix = check(p)
    own = dict(p, ptable=None, prefix=0, table=p["ptable"][None].repeat(5, 1).contiguous(),
               lens=torch.full((5,), 400, dtype=torch.int32, device="cuda"))
    check(own)
    assert float((run(own).double() - with_prefix.double()).abs().max()) < 2.0 ** -7


def test_equal_calls_give_equal_bits_in_a_used_workspace(cuda_device):
    import torch
    p = make([9000, 1, 0, 4097, 33], 16, 4, 64, 16, "bf16", prefix=300, seed=11)
    small = make([3000], 8, 8, 128, 32, "bf16", seed=12)
    need = max(fc.fuse_paged_attention_workspace_bytes(5, 16, 4, 64, 300), fc.fuse_paged_attention_workspace_bytes(1, 8, 8, 128))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ws[:8192] = 0                                                            # all that has to be zero
    first, other = run(p, workspace=ws).clone(), run(small, workspace=ws).clone()
    for _ in range(3):
        assert torch.equal(run(p, workspace=ws), first)
        assert torch.equal(run(small, workspace=ws), other)
        assert not ws[:8192].any()


def test_lengths_change_between_replays(cuda_device):
    """One captured graph serves growing lengths (they are read on the device)."""
    import torch
    p = make([700, 60, 333], 8, 2, 128, 16, "bf16", prefix=90, seed=13)
    ws = torch.zeros(fc.fuse_paged_attention_workspace_bytes(3, 8, 2, 128, 90), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(p["q"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fc.fuse_graph_begin(s)
        with pytest.raises(ValueError):                                      # no workspace of the module's own in a graph
            fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o, p["scale"], prefix_table=p["ptable"],
                                    prefix_len=90)
        fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o, p["scale"], prefix_table=p["ptable"],
                                prefix_len=90, workspace=ws)
        g = fc.fuse_graph_end(s)
    assert fc.fuse_graph_kernel_count(g) == 3
    for lens in ([700, 60, 333], [0, 1, 332], [16, 59, 100]):
        p["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        fc.fuse_graph_launch(g, s)
        s.synchronize()
        want, tol = reference(p)
        assert bool(((o.double() - want).abs() <= tol).all())
    fc.fuse_graph_destroy(g)


def test_calls_on_two_streams(cuda_device):
    """Two streams, each with the module's workspace of its own."""
    import torch
    ps = [make([5000, 3, 800], 8, 2, 128, 16, "bf16", seed=20 + i) for i in range(2)]
    want = [run(p).clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[torch.empty_like(p["q"]) for _ in range(4)] for p in ps]
    torch.cuda.synchronize()
    for i in range(4):
        for p, s, o in zip(ps, streams, outs):
            with torch.cuda.stream(s):
                fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o[i], p["scale"])
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for o, w in zip(outs, want) for x in o)


def test_bad_pages_and_lengths_are_reported(cuda_device):
    """A page outside the cache counts as zeros, a length outside the table is taken into it."""
    import torch
    p = make([40, 20, 30], 4, 2, 64, 16, "bf16", prefix=40, seed=14)
    z = dict(p, table=p["table"].clone(), k=p["k"].clone(), v=p["v"].clone(), ptable=p["ptable"].clone())
    free = [i for i in range(p["k"].shape[0]) if i not in set(p["table"][:, :3].flatten().tolist() + p["ptable"].tolist())]
    z["k"][free[0]], z["v"][free[0]] = 0, 0
    z["table"][0, 1], z["ptable"][1] = free[0], free[0]
    want = check(z)
    p["table"][0, 1], p["ptable"][1] = p["k"].shape[0], -5
    o = torch.empty_like(p["q"])

    def call(q):
        fc.fuse_paged_attention(q["q"], q["k"], q["v"], q["table"], q["lens"], o, q["scale"], prefix_table=q["ptable"], prefix_len=q["prefix"])
        return fc.fuse_check()

    assert call(p) == fc.FUSE_EINDEX and fc.fuse_check() == fc.FUSE_OK
    assert torch.equal(o, want)
    z["lens"].copy_(torch.tensor([-3, 20, 30], dtype=torch.int32))
    assert call(z) == fc.FUSE_EINDEX
    z["lens"][0] = 0
    assert torch.equal(o, run(z))
    full = make([48, 48], 4, 2, 64, 16, "bf16", seed=15)
    want = run(full).clone()
    full["lens"][1] = 49
    o = torch.empty_like(full["q"])
    assert call(full) == fc.FUSE_EINDEX and torch.equal(o, want)


def test_wrapper_refusals(cuda_device):
    import torch
    p = make([40, 20], 4, 2, 64, 16, "bf16", prefix=40, seed=16)
    o = torch.empty_like(p["q"])
    good = dict(q=p["q"], k=p["k"], v=p["v"], table=p["table"], lens=p["lens"], o=o, pt=p["ptable"], pl=40, ws=None)
    for bad in (dict(q=p["q"].half()), dict(table=p["table"].long()), dict(lens=p["lens"][:1]), dict(o=o[:1]),
                dict(pl=49), dict(pt=None), dict(k=p["k"].transpose(1, 2)), dict(q=p["q"].cpu()),
                dict(ws=torch.zeros(1 << 20, dtype=torch.uint8))):
        c = dict(good, **bad)
        with pytest.raises(ValueError):
            fc.fuse_paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["o"], 0.1, prefix_table=c["pt"],
                                    prefix_len=c["pl"], workspace=c["ws"])
    with pytest.raises(fc.FuseError):
        fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o, 0.1,
                                workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))


def test_two_threads_on_one_stream(cuda_device):
    """Calls of two threads on the same stream, with the module's own workspace, do not mix."""
    import threading
    import torch
    ps = [make([70 + 13 * b for b in range(24)], 16, 2, 128, 32, "bf16", prefix=900, seed=1),
          make([5 * b for b in range(40)], 8, 8, 64, 16, "bf16", prefix=140, seed=2)]
    want = [run(p) for p in ps]
    outs = [[torch.empty_like(p["q"]) for _ in range(100)] for p in ps]
    errors = []

    def work(p, os):
        try:
            for o in os:
                fc.fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], o, p["scale"], prefix_table=p["ptable"],
                                        prefix_len=p["prefix"])
        except Exception as e:      # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(ps, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and fc.fuse_check() == fc.FUSE_OK
    for w, os in zip(want, outs):
        assert all(torch.equal(o, w) for o in os)


def test_a_timeout_leaves_nothing_in_the_modules_workspace(cuda_device):
    """Counts that a given-up call left in the module's own buffer do not reach the calls after fuse_check()."""
    import torch
    p = make([20000, 300], 8, 1, 128, 64, "bf16", seed=21)
    want = run(p).clone()
    torch.cuda.synchronize()
    for ws in fc._PAGED_WS.values():
        ws[:8192].view(torch.int32)[:1280] = 1                               # one arrival of every item
    fc.fuse_debug_expire_wait(1000)
    assert fc.fuse_check() == fc.FUSE_ETIMEOUT
    for _ in range(3):
        assert torch.equal(run(p), want)


def test_a_refused_call_enqueues_nothing(cuda_device):
    """65536 heads with room for 2^31 - 4112 keys each are more places than a CTA counts: refused, with the shared
    prefix, which could be read, left alone."""
    import torch
    heads, page = 65536, 16
    ld = ((1 << 31) - 4096) // page - 1
    q = torch.zeros(1, heads, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 7.0)
    k, v = (torch.zeros(1, heads, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros(1, ld, dtype=torch.int32, device="cuda")
    lens, ptable = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(fc.fuse_paged_attention_workspace_bytes(1, heads, heads, 64, page), dtype=torch.uint8, device="cuda")
    with pytest.raises(fc.FuseError) as e:
        fc.fuse_paged_attention(q, k, v, table, lens, o, 0.125, prefix_table=ptable, prefix_len=page, workspace=ws)
    assert e.value.status == fc.FUSE_EUNSUPPORTED
    assert fc.fuse_check() == fc.FUSE_OK and not ws.any() and bool((o == 7).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 1000])
def test_infinite_values(cuda_device, D, prefix):
    """A component whose only infinite value has a weight is infinite, however many CTAs share the keys; the
    others are as they would be without it."""
    import torch
    p = make([9000, 200, 40], 8, 2, D, 64, "bf16", prefix=prefix, seed=22, std=0.25)
    clean = run(p).clone()
    v = p["v"] = p["v"].clone()
    at = []
    for b, keys in enumerate(([70, 4000, 8999], [0, 199], [39])):
        for n, key in enumerate(keys):
            v[int(p["table"][b, key // 64]), :, key % 64, n] = -math.inf if n else math.inf
            at.append((b, n, -math.inf if n else math.inf))
    if prefix:
        v[int(p["ptable"][500 // 64]), :, 500 % 64, 9] = math.inf
        at += [(b, 9, math.inf) for b in range(3)]
    o = run(p)
    for b, c, x in at:
        assert bool((o[b, :, c] == x).all()), (b, c, o[b, :, c])
        o[b, :, c] = clean[b, :, c]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_scores(cuda_device, dtype, D):
    """Own keys six times as long at the end of every 1024 as at their start: the reference follows, run after run."""
    import torch
    p = make([30000, 2000, 130], 16, 2, D, 64, dtype, seed=23)
    for b in range(3):
        n = int(p["lens"][b])
        ids = p["table"][b, :-(-n // 64)].long()
        long = 1 + 5 * (torch.arange(len(ids), device="cuda") % 16) / 15
        p["k"][ids] = (p["k"][ids].float() * long[:, None, None, None]).to(p["k"].dtype)
    check(p)


@pytest.mark.parametrize("prefix", [0, 40])
def test_the_largest_tables_in_shared_memory(cuda_device, prefix):
    """4096 sequences at 16 rows of D = 256: what is left of an SM's shared memory holds a ring of one slot."""
    check(make([(7 * i) % 90 if i % 64 == 0 else i % 2 for i in range(4096)], 16, 1, 256, 16, "bf16", prefix=prefix, seed=24))
