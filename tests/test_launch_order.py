"""The order of programmatic launch against tensor memory and earlier writes, read from the kernels' sources.

A kernel lets the next one start with pdl_trigger().  CTAs of the next kernel may then share an SM with its
own, so a kernel that allocates tensor memory has to hold it by then: allocation waits without a bound, and
the next kernel gives columns back only after this one has completed."""
import os
import re

import pytest

import epilogue_chains_gb300 as fc

CSRC = os.path.join(os.path.dirname(os.path.abspath(fc.__file__)), "csrc")


def kernels():
    """{name: source from its name to the end of its body} of every kernel definition, comments left out."""
    found = {}
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+)\(\s*(?:const|float|__half|__nv_bfloat16|int|T\b)", text):
            end = re.compile(r"^}", re.M).search(text, m.end())
            found[m.group(1)] = text[m.start(1):end.end()]
    return found


def test_dependents_start_with_the_tensor_memory_in_hand():
    seen = set()
    for name, body in kernels().items():
        alloc = re.search(r"\btmem_alloc(?:_pair)?\(", body)
        if not alloc:
            continue
        seen.add(name)
        trigger = re.search(r"\bpdl_(?:trigger|begin)\(\)", body)
        assert trigger and trigger.start() > alloc.start(), name
        # one warp allocates; the others know once they have passed a barrier
        assert re.search(r"__syncthreads\(\)|cluster_sync\(\)", body[alloc.end():trigger.start()]), name
    assert seen == {"attn_fwd_kernel", "attn_persist_kernel", "gemm_decode_kernel", "gemm_tc_kernel", "paged_prefix_kernel",
                    "paged_prefix2_kernel", "w4_tile_kernel"}


def test_own_keys_are_read_behind_what_was_written_before():
    """With a shared prefix the own-key kernel starts while the prefix kernel still runs, without a wait for it.
    That it may start does not order its reads behind the writes of earlier kernels: the prefix kernel has to
    release a word after its own wait, the own-key kernel to acquire it before its first read, for its copies
    (another proxy) too, and the join, which comes after both, to take the word back."""
    k = kernels()
    for name in ("paged_prefix_kernel", "paged_prefix2_kernel"):
        at = [k[name].index(x) for x in ("pdl_wait();", "st_release_gpu(a.ready, 1);", "pdl_trigger();")]
        assert at == sorted(at), name
    own = k["paged_own_kernel"]
    acquire = re.search(r"if \(a\.plen == 0\) \{\s*pdl_wait\(\);\s*\} else \{\s*if \(tid == 32\) \(void\)flag_wait_bounded\(a\.ready, 1, a\.flag\);"
                        r"\s*__syncthreads\(\);\s*fence_async_global\(\);\s*\}", own)
    assert acquire
    read = re.search(r"a\.lens|a\.table \+|__ldcg\(|tma_load", own)
    assert read and acquire.end() < read.start()
    join = k["paged_join_kernel"]
    back = join.index("*a.ready = 0;")
    assert join.index("pdl_wait();") < back < join.index("__ldcg(")


@pytest.mark.gpu
def test_small_tensor_memory_kernels_in_a_row(cuda_device):
    """Decode GEMM, dense attention and 4-bit tiles, whose CTAs fit on one SM together, back to back on one
    stream: each reads what the one before it wrote, and every round gives the same bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    H, S = 4096, 128
    x = torch.randn(16, H, generator=g, device="cuda").half()
    w = (torch.randn(H, H, generator=g, device="cuda") / 64).half()
    bias, R = torch.zeros(H, device="cuda").half(), torch.zeros(16, H, device="cuda").half()
    wq = torch.randint(0, 256, (H, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((0.5 + torch.rand(H, H // 128, generator=g, device="cuda")) * 0.2 / 64).half()
    q, k, v = (torch.randn(2, S, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    y, z, o = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q)

    def step():
        fc.fuse_gemm_epilogue(x, w, bias, R, y)
        fc.fuse_w4_gemv(y, wq, s, z)
        fc.fuse_attention(q, k, v, o, 0.125)
        fc.fuse_w4_gemv(z, wq, s, y)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (y, z, o)]
    for _ in range(200):
        step()
    assert fc.fuse_check() == fc.FUSE_OK
    assert all(torch.equal(a, b) for a, b in zip((y, z, o), first))
    assert all(bool(t.isfinite().all()) for t in first)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,D,batch", [(40, 64, 3), (900, 128, 48), (300, 256, 8), (0, 128, 5)])
def test_attention_sees_the_append_before_it(cuda_device, prefix, D, batch):
    """Two tokens in turn overwrite the last place of every sequence, queries, keys and values, each followed at
    once by attention over it, without a wait in between: every output is of its own token."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    hq, hk, page, per = 8, 2, 16, 5
    shared = -(-prefix // page)
    pages = batch * per + shared
    k, v = (torch.randn(pages, hk, page, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(batch * per, dtype=torch.int32, device="cuda").view(batch, per)
    ptable = torch.arange(batch * per, pages, dtype=torch.int32, device="cuda") if prefix else None
    lens = 1 + torch.arange(batch, dtype=torch.int32, device="cuda") * 7 % (page * per)
    last = lens - 1
    slots = table[torch.arange(batch, device="cuda"), last.long() // page] * page + last % page
    cs = torch.cat([torch.ones(100, D // 2), torch.zeros(100, D // 2)], 1).cuda()
    pos = torch.zeros(batch, dtype=torch.int32, device="cuda")
    qkv = [torch.randn(batch, (hq + 2 * hk) * D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    q = torch.empty(batch, hq, D, device="cuda").bfloat16()
    ws = torch.zeros(fc.fuse_paged_attention_workspace_bytes(batch, hq, hk, D, prefix), dtype=torch.uint8, device="cuda")

    def step(i, o):
        fc.fuse_rope_append(qkv[i], cs, pos, slots, q, k, v)
        fc.fuse_paged_attention(q, k, v, table, lens, o, 0.1, prefix_table=ptable, prefix_len=prefix, workspace=ws)

    want = [torch.empty_like(q) for _ in range(2)]
    for i in range(2):
        step(i, want[i])
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    outs = [torch.empty_like(q) for _ in range(400)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        step(i % 2, o)
    assert fc.fuse_check() == fc.FUSE_OK and not ws[:8192].any()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))
