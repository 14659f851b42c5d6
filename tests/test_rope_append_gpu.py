"""Rotate-and-append against the formulas in 64 bits.

Tolerance: the kernel rotates in fp32 (two products and a sum of given inputs: at most 2^-22 of
|a cos| + |b sin|) and rounds once to the storage type (half a step, u = eps / 2, of the result; fp16 below
its normal range: 2^-25).  Copied components, values and untouched slots are bit-identical."""
import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def make(tokens, hq, hk, D, rot, page, dtype, seed=0, pad=0, extra_ld=0, max_pos=5000, pages=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, DT[dtype])
    pages = pages or (tokens + page - 1) // page + 2
    width = (hq + 2 * hk) * D
    qkv = torch.randn(tokens, width + extra_ld, generator=g, device="cuda").to(dt)[:, :width]
    order = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    if pad:
        order[torch.randperm(tokens, generator=g, device="cuda")[:pad]] = -1
    pos = torch.randint(0, max_pos, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(1, rot // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    cache = [torch.randn(pages, hk, page, D, generator=g, device="cuda").to(dt) for _ in range(2)]
    return qkv, cs, pos, order, torch.full((tokens, hq, D), float("nan"), dtype=dt, device="cuda"), cache[0], cache[1]


def reference(qkv, cs, pos, slots, q, k, v, inter):
    """(q, k, v) in 64 bits and, for q and k, the sums of magnitudes that the tolerance needs."""
    import torch
    t, hq, D = q.shape
    hk, page, rot = k.shape[1], k.shape[2], cs.shape[1]
    x = qkv.double().view(t, hq + 2 * hk, D)
    c, s = cs[pos.long()].double().split(rot // 2, 1) if rot else (None, None)
    y, mag = x.clone(), x.abs()
    if rot:
        i = torch.arange(0, rot, 2, device="cuda") if inter else torch.arange(rot // 2, device="cuda")
        j = i + (1 if inter else rot // 2)
        a, b = x[:, :hq + hk][..., i], x[:, :hq + hk][..., j]
        c, s = c[:, None], s[:, None]
        y[:, :hq + hk, i], y[:, :hq + hk, j] = a * c - b * s, b * c + a * s
        mag[:, :hq + hk, i], mag[:, :hq + hk, j] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    kk, vv, km = k.double(), v.double(), torch.zeros_like(k, dtype=torch.float64)
    live = (slots >= 0).nonzero()[:, 0]
    at = slots[live].long()
    kk[at // page, :, at % page] = y[live, hq:hq + hk]
    km[at // page, :, at % page] = mag[live, hq:hq + hk]
    vv[at // page, :, at % page] = x[live, hq + hk:]
    return y[:, :hq], mag[:, :hq], kk, km, vv


def check(args, inter):
    import torch
    qkv, cs, pos, slots, q, k, v = args
    want, qm, kk, km, vv = reference(*args, inter)
    fc.fuse_rope_append(qkv, cs, pos, slots, q, k, v, interleaved=inter)
    assert fc.fuse_check() == fc.FUSE_OK
    u = torch.finfo(q.dtype).eps / 2
    tiny = 2.0 ** -25 if q.dtype is torch.float16 else 0.0
    for got, ref, mag in ((q, want, qm), (k, kk, km)):
        err = (got.double() - ref).abs()
        assert bool((err <= u * ref.abs() + (1 + u) * 2.0 ** -22 * mag + tiny).all()), float(err.max())
    assert torch.equal(v.double(), vv)
    D, rot = q.shape[2], cs.shape[1]
    if rot < D:
        assert torch.equal(q[..., rot:].double(), want[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,hq,hk,D,rot,page,pad", [
    (1, 32, 8, 128, 128, 16, 0), (1, 1, 1, 64, 64, 16, 0), (3, 5, 1, 64, 16, 32, 1), (64, 32, 8, 128, 64, 64, 3),
    (257, 7, 7, 256, 256, 128, 17), (2, 3, 2, 80, 48, 16, 0), (5, 2, 1, 512, 32, 256, 5), (4, 6, 2, 16, 16, 16, 0)])
def test_shapes(cuda_device, inter, dtype, tokens, hq, hk, D, rot, page, pad):
    check(make(tokens, hq, hk, D, rot, page, dtype, seed=tokens, pad=pad), inter)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_strided_rows_and_many_tokens(cuda_device, dtype):
    check(make(3001, 8, 2, 128, 128, 64, dtype, extra_ld=72, pad=100), False)


def test_no_rotation_and_no_tokens(cuda_device):
    import torch
    args = make(9, 4, 2, 64, 0, 16, "bf16")
    check(args, False)
    e = make(1, 4, 2, 64, 64, 16, "bf16")
    before = [t.clone() for t in e[5:]]
    fc.fuse_rope_append(e[0][:0], e[1], e[2][:0], e[3][:0], e[4][:0], e[5], e[6])
    torch.cuda.synchronize()
    assert torch.equal(e[5], before[0]) and torch.equal(e[6], before[1])


def test_far_positions(cuda_device):
    """The last row of a long table (an offset past 2^31 elements is out of reach of a test; past 2^27 here)."""
    args = list(make(4, 2, 1, 128, 128, 16, "bf16", max_pos=1 << 20))
    args[2].fill_((1 << 20) - 1)
    check(args, False)


def test_bad_indexes_touch_nothing_and_are_reported(cuda_device):
    import torch
    qkv, cs, pos, slots, q, k, v = make(4, 4, 2, 64, 64, 16, "bf16", max_pos=100, pages=3)
    slots.copy_(torch.tensor([48, 5, 6, -7], dtype=torch.int32))       # one past the cache, two good, padded
    pos.copy_(torch.tensor([1, 100, 2, -1], dtype=torch.int32))        # good, past the table, good, ignored
    k0, v0 = k.clone(), v.clone()
    fc.fuse_rope_append(qkv, cs, pos, slots, q, k, v)
    assert fc.fuse_check() == fc.FUSE_EINDEX
    assert fc.fuse_check() == fc.FUSE_OK                               # cleared once reported
    k1, v1 = k.clone(), v.clone()
    k1[0, :, 6], v1[0, :, 6] = k0[0, :, 6], v0[0, :, 6]                # slot 6 is the only one written
    assert torch.equal(k1, k0) and torch.equal(v1, v0)
    assert torch.equal(v[0, :, 6], qkv.view(4, 8, 64)[2, 6:])
    assert not q[1].any() and not q[3].any() and bool(torch.isfinite(q).all())
    # a padded row alone is not an error, whatever its position
    slots.fill_(-1)
    fc.fuse_rope_append(qkv, cs, pos, slots, q, k, v)
    assert fc.fuse_check() == fc.FUSE_OK


def test_graph_replay_on_another_stream(cuda_device):
    import torch
    args = make(17, 8, 2, 128, 128, 16, "f16", seed=5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fc.fuse_graph_begin(s)
        fc.fuse_rope_append(*args, stream=s)
        g = fc.fuse_graph_end(s)
        assert fc.fuse_graph_kernel_count(g) == 1
        eager = [t.clone() for t in args]
    s.synchronize()
    fc.fuse_rope_append(*eager)
    args[4].zero_()
    torch.cuda.synchronize()
    fc.fuse_graph_launch(g, s)
    s.synchronize()
    fc.fuse_graph_destroy(g)
    assert all(torch.equal(a, b) for a, b in zip(args[4:], eager[4:]))


def test_wrapper_refusals(cuda_device):
    qkv, cs, pos, slots, q, k, v = make(4, 4, 2, 64, 64, 16, "bf16")
    with pytest.raises(ValueError):
        fc.fuse_rope_append(qkv, cs, pos.long(), slots, q, k, v)
    with pytest.raises(ValueError):
        fc.fuse_rope_append(qkv, cs, pos, slots, q.half(), k, v)
    with pytest.raises(ValueError):
        fc.fuse_rope_append(qkv[:, :-64], cs, pos, slots, q, k, v)
    with pytest.raises(ValueError):
        fc.fuse_rope_append(qkv, cs, pos[:3], slots, q, k, v)
    with pytest.raises(ValueError):
        fc.fuse_rope_append(qkv, cs.double(), pos, slots, q, k, v)
    with pytest.raises(fc.FuseError):
        fc.fuse_rope_append(qkv, cs[:, :24].contiguous(), pos, slots, q, k, v)
