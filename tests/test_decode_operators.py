"""Host-side checks of the single-token decode operators (rotate and append, paged attention, 4-bit
projection): refusals, workspace sizes and byte ledgers.  No GPU: every call below is refused, or has
nothing to do, before anything is enqueued."""
import pytest

import epilogue_chains_gb300 as fc

A, B, C, D_, E, F, G = (0x10000000 * i for i in range(1, 8))   # far apart, 256-byte aligned, never read


def rope(**kw):
    p = dict(qkv=A, ld=48 * 128, cs=B, max_pos=1024, rot=128, pos=C, slots=C + 0x1000, q=D_, k=E, v=F, tokens=4,
             hq=32, hk=8, D=128, pages=8, page=16, dtype=fc.FUSE_BF16, flags=0)
    p.update(kw)
    return fc._load().fuse_rope_append(p["qkv"], p["ld"], p["cs"], p["max_pos"], p["rot"], p["pos"], p["slots"], p["q"],
                                       p["k"], p["v"], p["tokens"], p["hq"], p["hk"], p["D"], p["pages"], p["page"],
                                       p["dtype"], p["flags"], None)


def paged(**kw):
    p = dict(q=A, k=B, v=C, table=D_, ld=4, lens=D_ + 0x10000, ptable=None, plen=0, o=E, batch=2, hq=32, hk=8, D=128,
             pages=8, page=16, scale=0.1, dtype=fc.FUSE_BF16, ws=F, ws_bytes=1 << 26)
    p.update(kw)
    return fc._load().fuse_paged_attention(p["q"], p["k"], p["v"], p["table"], p["ld"], p["lens"], p["ptable"], p["plen"],
                                           p["o"], p["batch"], p["hq"], p["hk"], p["D"], p["pages"], p["page"],
                                           p["scale"], p["dtype"], p["ws"], p["ws_bytes"], None)


def w4(**kw):
    p = dict(x=A, wq=B, s=C, z=None, bias=None, R=None, y=D_, M=4, N=4096, K=4096, group=128, gelu=0,
             dtype=fc.FUSE_BF16)
    p.update(kw)
    return fc._load().fuse_w4_gemv(p["x"], p["wq"], p["s"], p["z"], p["bias"], p["R"], p["y"], p["M"], p["N"], p["K"],
                                   p["group"], p["gelu"], p["dtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0, qkv=None, q=None), fc.FUSE_OK),
    (dict(tokens=-1), fc.FUSE_EINVAL),
    (dict(hq=0), fc.FUSE_EINVAL),
    (dict(rot=144), fc.FUSE_EINVAL),             # more than D
    (dict(rot=24), fc.FUSE_EUNSUPPORTED),        # not a multiple of 16
    (dict(D=72, rot=0, ld=4096), fc.FUSE_EUNSUPPORTED),
    (dict(D=1024, ld=48 * 1024), fc.FUSE_EUNSUPPORTED),
    (dict(page=24), fc.FUSE_EUNSUPPORTED),
    (dict(page=8), fc.FUSE_EUNSUPPORTED),
    (dict(page=512), fc.FUSE_EUNSUPPORTED),
    (dict(pages=1 << 27), fc.FUSE_EUNSUPPORTED),
    (dict(ld=48 * 128 - 8), fc.FUSE_EINVAL),
    (dict(ld=48 * 128 + 4), fc.FUSE_EALIGN),
    (dict(dtype=fc.FUSE_F32), fc.FUSE_EINVAL),
    (dict(dtype=7), fc.FUSE_EINVAL),
    (dict(flags=2), fc.FUSE_EINVAL),
    (dict(qkv=None), fc.FUSE_EINVAL),
    (dict(slots=None), fc.FUSE_EINVAL),
    (dict(cs=None), fc.FUSE_EINVAL),
    (dict(pos=None), fc.FUSE_EINVAL),
    (dict(qkv=A + 8), fc.FUSE_EALIGN),
    (dict(slots=C + 2), fc.FUSE_EALIGN),
    (dict(q=A), fc.FUSE_EINVAL),                 # q_out overlaps qkv
    (dict(v=E + 8 * 8 * 16 * 128 * 2 - 16), fc.FUSE_EINVAL),   # the two caches overlap
    (dict(k=B), fc.FUSE_EINVAL),                 # the key cache overlaps the table
])
def test_rope_append_refusals(kw, want):
    assert rope(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0, q=None), fc.FUSE_OK),
    (dict(batch=-1), fc.FUSE_EINVAL),
    (dict(hq=30), fc.FUSE_EINVAL),               # not a multiple of the key/value heads
    (dict(scale=0.0), fc.FUSE_EINVAL),
    (dict(scale=float("nan")), fc.FUSE_EINVAL),
    (dict(scale=float("inf")), fc.FUSE_EINVAL),
    (dict(D=96), fc.FUSE_EUNSUPPORTED),
    (dict(page=48), fc.FUSE_EUNSUPPORTED),
    (dict(page=8), fc.FUSE_EUNSUPPORTED),
    (dict(batch=4097), fc.FUSE_EUNSUPPORTED),
    (dict(pages=1 << 28), fc.FUSE_EUNSUPPORTED),
    (dict(ld=1 << 28), fc.FUSE_EUNSUPPORTED),
    (dict(plen=1 << 31, ptable=G), fc.FUSE_EUNSUPPORTED),
    (dict(plen=-1), fc.FUSE_EINVAL),
    (dict(plen=5), fc.FUSE_EINVAL),              # no prefix table
    (dict(pages=0), fc.FUSE_EINVAL),
    (dict(dtype=fc.FUSE_F32), fc.FUSE_EINVAL),
    (dict(table=None), fc.FUSE_EINVAL),
    (dict(lens=None), fc.FUSE_EINVAL),
    (dict(q=A + 8), fc.FUSE_EALIGN),
    (dict(lens=D_ + 2), fc.FUSE_EALIGN),
    (dict(ws=None), fc.FUSE_EWORKSPACE),
    (dict(ws_bytes=16384), fc.FUSE_EWORKSPACE),
    (dict(ws=F + 128), fc.FUSE_EALIGN),
    (dict(o=A), fc.FUSE_EINVAL),                 # o overlaps q
    (dict(o=C + 256), fc.FUSE_EINVAL),           # o overlaps the value cache
    (dict(ws=B - 4096), fc.FUSE_EINVAL),         # the workspace overlaps the key cache
    (dict(ws=E), fc.FUSE_EINVAL),                # the workspace overlaps o
])
def test_paged_attention_refusals(kw, want):
    assert paged(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(M=0, x=None), fc.FUSE_OK),
    (dict(M=-1), fc.FUSE_EINVAL),
    (dict(N=0), fc.FUSE_EINVAL),
    (dict(K=0), fc.FUSE_EINVAL),
    (dict(M=65), fc.FUSE_EUNSUPPORTED),
    (dict(group=48), fc.FUSE_EUNSUPPORTED),
    (dict(group=256), fc.FUSE_EUNSUPPORTED),
    (dict(K=4096 + 64), fc.FUSE_EUNSUPPORTED),   # not a multiple of the group
    (dict(gelu=2), fc.FUSE_EINVAL),
    (dict(dtype=fc.FUSE_F32), fc.FUSE_EINVAL),
    (dict(x=None), fc.FUSE_EINVAL),
    (dict(y=None), fc.FUSE_EINVAL),
    (dict(x=A + 8), fc.FUSE_EALIGN),
    (dict(wq=B + 4), fc.FUSE_EALIGN),
    (dict(s=C + 1), fc.FUSE_EALIGN),
    (dict(R=D_), fc.FUSE_EINVAL),                # y overlaps the residual
    (dict(y=B + 64), fc.FUSE_EINVAL),            # y overlaps the weight
    (dict(z=D_ + 2), fc.FUSE_EINVAL),            # y overlaps the zero points
])
def test_w4_gemv_refusals(kw, want):
    assert w4(**kw) == want


def test_ledgers():
    # one token, 32 + 2 x 8 heads of 128: read and written once, a table row, a position and a slot
    assert fc.fuse_rope_append_bytes(1, 1, 32, 8, 128, 128) == 2 * 48 * 128 * 2 + 128 * 4 + 8
    # a padded row moves its query only
    assert fc.fuse_rope_append_bytes(2, 1, 32, 8, 128, 0) == 2 * (2 * 32 + 16) * 128 * 2 + 16
    assert fc.fuse_paged_attention_bytes(4, 32, 8, 128, 1000, 500) == 1500 * 8 * 128 * 4 + 4 * 32 * 128 * 4
    assert fc.fuse_paged_attention_flops(4, 32, 128, 1000, 500) == 4 * 128 * 32 * 4500
    assert fc.fuse_w4_gemv_bytes(1, 4096, 4096, 128) == 4096 * 2048 + 4096 * 32 * 2 + 2 * 4096 * 2
    assert fc.fuse_w4_gemv_bytes(2, 64, 256, 32, True, True, True) == 64 * 128 + 64 * 8 * 3 + 2 * 2 * 256 + 2 * 2 * 64 * 2 + 2 * 64
    lib = fc._load()
    assert lib.fuse_rope_append_bytes(1, 2, 32, 8, 128, 128) == fc.FUSE_EINVAL
    assert lib.fuse_paged_attention_bytes(1, 1, 1, 64, -1, 0) == fc.FUSE_EINVAL
    assert lib.fuse_w4_gemv_bytes(1, 64, 100, 32, 0, 0, 0) == fc.FUSE_EINVAL


def test_paged_workspace_is_host_arithmetic():
    ws = fc.fuse_paged_attention_workspace_bytes
    # counters, then (m, l) and fp32 output rows of two parts for each of at most 320 CTAs
    assert ws(1, 32, 8, 128) == 8192 + 640 * 4 * 8 + 640 * 4 * 128 * 4
    assert ws(512, 32, 8, 128) == ws(1, 32, 8, 128)          # independent of the batch
    # with a prefix: where an item's own parts are, every row's own part, and 256-row parts (128 rows up to 128 rows or D = 256) of
    # at most 160 CTAs and one more per item
    assert ws(64, 32, 8, 128, 100) == ws(1, 32, 8, 128) + 64 * 8 * 4 + 64 * 32 * (8 + 512) + (160 + 8) * 256 * (16 + 512)
    assert ws(1, 30, 8, 128) == 0 and ws(0, 32, 8, 128) == 0


def test_wrapper_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    kv = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fc.fuse_paged_attention(q, kv, kv.clone(), i, i[0], q.clone(), 1.0)
    with pytest.raises(ValueError):
        fc.fuse_rope_append(torch.zeros(1, 192, dtype=torch.bfloat16), torch.zeros(4, 64), i[0], i[0].clone(), q, kv, kv.clone())
    with pytest.raises(ValueError):
        fc.fuse_w4_gemv(torch.zeros(1, 32, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.uint8),
                        torch.zeros(8, 1, dtype=torch.bfloat16), torch.zeros(1, 8, dtype=torch.bfloat16))


def test_index_status_has_a_message():
    assert "out of range" in fc.fuse_strerror(fc.FUSE_EINDEX)


class _Status:
    """A library whose fuse_check() returns the given statuses in turn."""

    def __init__(self, *statuses):
        self.statuses = list(statuses)

    def fuse_check(self, stream):
        return self.statuses.pop(0)


def test_a_timeout_drops_the_modules_workspaces(monkeypatch):
    """A call that ran into a timeout leaves arrival counts behind; nobody else can zero the module's buffers."""
    monkeypatch.setattr(fc, "_load", lambda lib=_Status(fc.FUSE_OK, fc.FUSE_EINDEX, fc.FUSE_ECUDA, fc.FUSE_ETIMEOUT): lib)
    monkeypatch.setattr(fc, "_PAGED_WS", {(0, 0): object(), (0, 7): object()})
    for want, kept in ((fc.FUSE_OK, 2), (fc.FUSE_EINDEX, 2), (fc.FUSE_ECUDA, 2), (fc.FUSE_ETIMEOUT, 0)):
        assert fc.fuse_check(7) == want and len(fc._PAGED_WS) == kept
