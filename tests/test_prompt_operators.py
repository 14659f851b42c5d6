"""Host-side checks of the operators that read whole prompts (attention of packed prompts, microscaled 4-bit
floating point, log probabilities of tokens): refusals, workspace and scale sizes, byte ledgers, and what their
kernels' sources say of the order of programmatic launch.  No GPU: every call below is refused, or has nothing to
do, before anything is enqueued."""
import os
import re

import pytest

import epilogue_chains_gb300 as fc

A, B, C, D_, E, F, G = (0x10000000 * i for i in range(1, 8))   # far apart, 256-byte aligned, never read


def prompt(**kw):
    p = dict(q=A, q_ld=32 * 128, k=B, v=C, table=D_, ld=4, cu=D_ + 0x10000, lens=D_ + 0x20000, o=E, tokens=100, batch=2, hq=32,
             hk=8, D=128, pages=8, page=16, scale=0.1, dtype=fc.FUSE_BF16, ws=F, ws_bytes=1 << 27)
    p.update(kw)
    return fc._load().fuse_prompt_attention(p["q"], p["q_ld"], p["k"], p["v"], p["table"], p["ld"], p["cu"], p["lens"], p["o"],
                                            p["tokens"], p["batch"], p["hq"], p["hk"], p["D"], p["pages"], p["page"],
                                            p["scale"], p["dtype"], p["ws"], p["ws_bytes"], None)


def quantize(**kw):
    p = dict(x=A, ld=4096, q=B, s=C, rows=10, cols=4096, dtype=fc.FUSE_BF16)
    p.update(kw)
    return fc._load().fuse_mxfp4_quantize(p["x"], p["ld"], p["q"], p["s"], p["rows"], p["cols"], p["dtype"], None)


def dequantize(**kw):
    p = dict(q=B, s=C, y=A, rows=10, cols=4096, dtype=fc.FUSE_BF16)
    p.update(kw)
    return fc._load().fuse_mxfp4_dequantize(p["q"], p["s"], p["y"], p["rows"], p["cols"], p["dtype"], None)


def gemm(**kw):
    p = dict(xq=A, xs=B, wq=C, ws=D_, bias=None, R=None, y=E, M=10, N=4096, K=4096, gelu=0, dtype=fc.FUSE_BF16)
    p.update(kw)
    return fc._load().fuse_mxfp4_gemm(p["xq"], p["xs"], p["wq"], p["ws"], p["bias"], p["R"], p["y"], p["M"], p["N"], p["K"],
                                      p["gelu"], p["dtype"], None)


def score(**kw):
    p = dict(x=A, ld=1000, t=B, lp=C, h=D_, tl=E, ti=F, rows=7, vocab=1000, top=5, scale=1.0, dtype=fc.FUSE_F32)
    p.update(kw)
    return fc._load().fuse_token_logprobs(p["x"], p["ld"], p["t"], p["lp"], p["h"], p["tl"], p["ti"], p["rows"], p["vocab"],
                                          p["top"], p["scale"], p["dtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0, q=None), fc.FUSE_OK),
    (dict(batch=0, q=None), fc.FUSE_OK),
    (dict(tokens=-1), fc.FUSE_EINVAL),
    (dict(batch=-1), fc.FUSE_EINVAL),
    (dict(hq=30), fc.FUSE_EINVAL),               # not a multiple of the key/value heads
    (dict(scale=0.0), fc.FUSE_EINVAL),
    (dict(scale=float("nan")), fc.FUSE_EINVAL),
    (dict(scale=float("inf")), fc.FUSE_EINVAL),
    (dict(dtype=fc.FUSE_F32), fc.FUSE_EINVAL),
    (dict(q_ld=32 * 128 - 8), fc.FUSE_EINVAL),
    (dict(q_ld=32 * 128 + 4), fc.FUSE_EALIGN),
    (dict(D=96, q_ld=1 << 14), fc.FUSE_EUNSUPPORTED),
    (dict(hq=129 * 8, q_ld=129 * 8 * 128), fc.FUSE_EUNSUPPORTED),   # more than 128 query heads for each
    (dict(page=48), fc.FUSE_EUNSUPPORTED),
    (dict(page=8), fc.FUSE_EUNSUPPORTED),
    (dict(page=512), fc.FUSE_EUNSUPPORTED),
    (dict(batch=4097), fc.FUSE_EUNSUPPORTED),
    (dict(tokens=1 << 24), fc.FUSE_EUNSUPPORTED),
    (dict(pages=1 << 28), fc.FUSE_EUNSUPPORTED),
    (dict(ld=1 << 28), fc.FUSE_EUNSUPPORTED),
    (dict(tokens=(1 << 24) - 1, ld=(1 << 27) - 1024, hk=64, hq=64, q_ld=64 * 128, pages=1), fc.FUSE_EUNSUPPORTED),
    (dict(tokens=(1 << 24) - 1, hk=128, hq=128, q_ld=128 * 128, pages=1), fc.FUSE_EUNSUPPORTED),
    (dict(q=None), fc.FUSE_EINVAL),
    (dict(table=None), fc.FUSE_EINVAL),
    (dict(cu=None), fc.FUSE_EINVAL),
    (dict(lens=None), fc.FUSE_EINVAL),
    (dict(q=A + 8), fc.FUSE_EALIGN),
    (dict(o=E + 8), fc.FUSE_EALIGN),
    (dict(cu=D_ + 0x10002), fc.FUSE_EALIGN),
    (dict(ws=None), fc.FUSE_EWORKSPACE),
    (dict(ws_bytes=1000), fc.FUSE_EWORKSPACE),
    (dict(ws=F + 16), fc.FUSE_EALIGN),
    (dict(o=A), fc.FUSE_EINVAL),                 # o overlaps q
    (dict(o=A + 99 * 32 * 128 * 2), fc.FUSE_EINVAL),
    (dict(ws=B), fc.FUSE_EINVAL),                # the workspace overlaps the cache
    (dict(ws=E), fc.FUSE_EINVAL),
])
def test_prompt_attention_refusals(kw, want):
    assert prompt(**kw) == want


MATRIX = [
    (dict(rows=0, q=None), fc.FUSE_OK),
    (dict(rows=-1), fc.FUSE_EINVAL),
    (dict(cols=0), fc.FUSE_EINVAL),
    (dict(cols=4080), fc.FUSE_EUNSUPPORTED),
    (dict(rows=1 << 22), fc.FUSE_EUNSUPPORTED),
    (dict(dtype=5), fc.FUSE_EINVAL),
    (dict(q=None), fc.FUSE_EINVAL),
    (dict(s=None), fc.FUSE_EINVAL),
    (dict(q=B + 8), fc.FUSE_EALIGN),
    (dict(s=C + 8), fc.FUSE_EALIGN),
    (dict(q=A + 4096), fc.FUSE_EINVAL),          # overlap
    (dict(s=A), fc.FUSE_EINVAL),
]


@pytest.mark.parametrize("kw,want", MATRIX + [
    (dict(ld=4080), fc.FUSE_EINVAL),
    (dict(ld=4104), fc.FUSE_EALIGN),             # rows not 32-byte aligned
    (dict(ld=4104, dtype=fc.FUSE_F32, x=None), fc.FUSE_EINVAL),
    (dict(x=A + 16), fc.FUSE_EALIGN),
    (dict(q=C - 10 * 2048 + 16), fc.FUSE_EINVAL),    # codes and scales overlap
])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


@pytest.mark.parametrize("kw,want", MATRIX + [(dict(y=A + 16), fc.FUSE_EALIGN), (dict(y=None), fc.FUSE_EINVAL)])
def test_dequantize_refusals(kw, want):
    assert dequantize(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(M=0, xq=None), fc.FUSE_OK),
    (dict(M=-1), fc.FUSE_EINVAL),
    (dict(N=0), fc.FUSE_EINVAL),
    (dict(K=0), fc.FUSE_EINVAL),
    (dict(K=48), fc.FUSE_EUNSUPPORTED),
    (dict(M=1 << 22), fc.FUSE_EUNSUPPORTED),
    (dict(N=1 << 22), fc.FUSE_EUNSUPPORTED),
    (dict(M=(1 << 22) - 1, N=(1 << 22) - 1, K=2048), fc.FUSE_EUNSUPPORTED),
    (dict(gelu=2), fc.FUSE_EINVAL),
    (dict(dtype=fc.FUSE_F32), fc.FUSE_EINVAL),
    (dict(xs=None), fc.FUSE_EINVAL),
    (dict(ws=None), fc.FUSE_EINVAL),
    (dict(y=None), fc.FUSE_EINVAL),
    (dict(xq=A + 8), fc.FUSE_EALIGN),
    (dict(ws=D_ + 4), fc.FUSE_EALIGN),
    (dict(y=E + 1), fc.FUSE_EALIGN),
    (dict(bias=F + 1), fc.FUSE_EALIGN),
    (dict(R=E), fc.FUSE_EINVAL),                 # y overlaps an input
    (dict(y=C + 4096), fc.FUSE_EINVAL),
    (dict(bias=E + 10 * 4096 * 2 - 2), fc.FUSE_EINVAL),
])
def test_gemm_refusals(kw, want):
    assert gemm(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, x=None), fc.FUSE_OK),
    (dict(rows=-1), fc.FUSE_EINVAL),
    (dict(vocab=0), fc.FUSE_EINVAL),
    (dict(ld=999), fc.FUSE_EINVAL),
    (dict(top=-1), fc.FUSE_EINVAL),
    (dict(vocab=4, top=5), fc.FUSE_EINVAL),
    (dict(top=33), fc.FUSE_EUNSUPPORTED),
    (dict(vocab=(1 << 31) - 64, ld=1 << 31), fc.FUSE_EUNSUPPORTED),
    (dict(rows=1 << 28), fc.FUSE_EUNSUPPORTED),
    (dict(scale=0.0), fc.FUSE_EINVAL),
    (dict(scale=-1.0), fc.FUSE_EINVAL),
    (dict(scale=float("nan")), fc.FUSE_EINVAL),
    (dict(scale=3e38), fc.FUSE_EINVAL),          # times log2(e) not finite
    (dict(dtype=3), fc.FUSE_EINVAL),
    (dict(x=None), fc.FUSE_EINVAL),
    (dict(t=None), fc.FUSE_EINVAL),
    (dict(lp=None, h=None, top=0), fc.FUSE_EINVAL),
    (dict(tl=None, ti=None), fc.FUSE_EINVAL),
    (dict(x=A + 2), fc.FUSE_EALIGN),
    (dict(x=A + 1, dtype=fc.FUSE_BF16), fc.FUSE_EALIGN),
    (dict(lp=C + 2), fc.FUSE_EALIGN),
    (dict(h=C), fc.FUSE_EINVAL),                 # two outputs overlap
    (dict(tl=A), fc.FUSE_EINVAL),
    (dict(ti=E + 7 * 5 * 4 - 4), fc.FUSE_EINVAL),
])
def test_token_logprobs_refusals(kw, want):
    assert score(**kw) == want


def test_sizes_are_host_arithmetic():
    ws = fc.fuse_prompt_attention_workspace_bytes
    # where 160 runs begin, then (m, l) and fp32 rows of two parts for each of at most 160 CTAs
    assert ws(1000, 32, 8, 128) == 2816 + 320 * 256 * 8 + 320 * 256 * 128 * 4
    assert ws(100000, 32, 8, 128) == ws(1000, 32, 8, 128)
    assert ws(1000, 32, 8, 256) == 2816 + 320 * 128 * 8 + 320 * 128 * 256 * 4       # of 80 pairs of CTAs
    assert ws(17, 32, 8, 128) == 2816 + 320 * 68 * 8 + 320 * 68 * 128 * 4           # 17 tokens of four heads in one tile
    assert ws(1, 30, 8, 128) == 0 and ws(0, 32, 8, 128) == 0 and ws(1, 129, 1, 128) == 0
    assert fc.fuse_mxfp4_scale_bytes(1, 32) == 512
    assert fc.fuse_mxfp4_scale_bytes(129, 160) == 4 * 512
    with pytest.raises(fc.FuseError):
        fc.fuse_mxfp4_scale_bytes(4, 33)


def test_ledgers():
    assert fc.fuse_prompt_attention_bytes(17, 17, 32, 8, 128) == 4 * 128 * (8 * 17 + 17 * 32)
    assert fc.fuse_prompt_attention_flops(17 * 18 // 2, 32, 128) == 4 * 128 * 32 * 153
    assert fc.fuse_mxfp4_gemm_bytes(1, 4096, 4096) == 4097 * (2048 + 128) + 2 * 4096
    assert fc.fuse_mxfp4_gemm_bytes(2, 64, 32, bias=True, residual=True) == 66 * 17 + 4 * 128 + 128
    assert fc.fuse_token_logprobs_bytes(3, 1000, 5, fc.FUSE_BF16) == 3 * (2000 + 12 + 40)


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    kv = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    u = torch.zeros(1, 16, dtype=torch.uint8)
    s = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fc.fuse_prompt_attention(q, kv, kv.clone(), i, torch.zeros(2, dtype=torch.int32), i[0], q.clone(), 1.0)
    with pytest.raises(ValueError):
        fc.fuse_mxfp4_quantize(torch.zeros(1, 32), u, s)
    with pytest.raises(ValueError):
        fc.fuse_mxfp4_dequantize(u, s, torch.zeros(1, 32))
    with pytest.raises(ValueError):
        fc.fuse_mxfp4_gemm(u, s, u.clone(), s.clone(), torch.zeros(1, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fc.fuse_token_logprobs(torch.zeros(1, 32), i[0], torch.zeros(1))


def test_dependents_start_with_the_tensor_memory_in_hand():
    """The kernels that take their tensor memory by tmem_begin() trigger nowhere else, and it triggers after a barrier
    behind the allocation."""
    csrc = os.path.join(os.path.dirname(os.path.abspath(fc.__file__)), "csrc")

    def source(name):
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            return re.sub(r"//[^\n]*", "", f.read())

    tc = source("fc_tc.cuh")
    for name, alloc, barrier in (("tmem_begin", "tmem_alloc(", "__syncthreads();"), ("tmem_begin_pair", "tmem_alloc_pair(", "cluster_sync();")):
        body = re.search(r"uint32_t %s\([^{]*\{(.*?)\n\}" % name, tc, re.S).group(1)
        at = [body.index(x) for x in (alloc, barrier, "pdl_trigger();", "return")]
        assert at == sorted(at)
    for name in ("prompt_attention.cu", "mxfp4.cu"):
        for kernel in re.findall(r"__global__.*?\n\}", source(name), re.S):
            begin = re.search(r"tmem_begin(_pair)?\(", kernel)
            if begin:
                assert "pdl_trigger" not in kernel and "pdl_begin" not in kernel and "tmem_alloc" not in kernel
                assert begin.start() < kernel.index("pdl_wait();")
            else:
                assert kernel.index("pdl_begin();") > 0 and "tmem_dealloc" not in kernel
