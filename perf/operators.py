"""The measured cases of the single-token decode operators.

One decoder step of a served model runs, between the norms this library already has, three things:
a projection of a few tokens by a weight held in 4 bits (``fuse_w4_gemv``), the rotation of the new
queries and keys with the append of keys and values to a paged cache (``fuse_rope_append``), and the
attention of the new tokens over that cache, part of which may be a prefix that the whole batch
shares (``fuse_paged_attention``).

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()`` one pass (the plain
torch form, or the library's calls where ``own`` is true), ``work()`` what a pass cannot do without
and ``exact()`` the same values in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------- cases
def _rope(name, tokens, q_heads, kv_heads, D, rot, page, dtype, interleaved, pad):
    return {"name": name, "op": "rope_append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "D": D,
            "rot": rot, "page": page, "dtype": dtype, "interleaved": interleaved, "pad": pad}


def _attn(name, batch, q_heads, kv_heads, D, page, dtype, longest, prefix):
    return {"name": name, "op": "paged_attention", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "D": D,
            "page": page, "dtype": dtype, "longest": longest, "prefix": prefix}


def _w4(name, M, N, K, group, dtype, zeros, bias, gelu, residual):
    return {"name": name, "op": "w4_gemv", "M": M, "N": N, "K": K, "group": group, "dtype": dtype, "zeros": zeros,
            "bias": bias, "gelu": gelu, "residual": residual}


def listed():
    return [
        # one user's next token: 32 query and 8 key/value heads of 128, the decoder configuration
        # whose kernels this repository's sources count
        _rope("append 1 token", 1, 32, 8, 128, 128, 16, "bf16", False, 0),
        # a padded decode batch (3 of 64 rows hold no token), pairs interleaved, half of each head rotated
        _rope("append 64 rows, 3 padded", 64, 32, 8, 128, 64, 32, "f16", True, 3),
        # a prompt's keys and values written into the cache
        _rope("append 8192 tokens", 8192, 32, 8, 128, 128, 64, "bf16", False, 0),
        # a short chat of one user: latency
        _attn("attend 1 x 700", 1, 32, 8, 128, 16, "bf16", 700, 0),
        # an ordinary serving batch, every length up to 4096
        _attn("attend 32 x 4096 ragged", 32, 32, 8, 128, 32, "bf16", 4096, 0),
        # few users with long documents: the key axis has to be split
        _attn("attend 3 x 65536", 3, 32, 8, 128, 64, "f16", 65536, 0),
        # a batch under one system prompt that ends inside a page
        _attn("attend 48, shared 8191", 48, 32, 8, 128, 16, "f16", 512, 8191),
        # many samples from one long prompt: the shared part is bound by arithmetic
        _attn("attend 256, shared 16384", 256, 32, 8, 128, 64, "bf16", 256, 16384),
        # 16 ungrouped heads of 256 (this repository's attention benchmark), short shared prompt
        _attn("attend 8 x 2048, D 256", 8, 16, 16, 256, 128, "bf16", 2048, 2048),
        # the output projection of one token (this repository's GEMM width)
        _w4("project 1 x 4096 x 4096", 1, 4096, 4096, 128, "bf16", False, False, False, True),
        # the down projection of a small batch, asymmetric weights in small groups, residual joined
        _w4("project 5 x 4096 x 14336", 5, 4096, 14336, 32, "f16", True, False, False, True),
        # the widest projection (gate and up merged) at the largest batch, whole epilogue
        _w4("project 64 x 28672 x 4096", 64, 28672, 4096, 64, "bf16", False, True, True, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    op = rng.choice(["rope_append", "paged_attention", "paged_attention", "w4_gemv"])
    while True:
        dtype = rng.choice(["bf16", "f16"])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        D = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128])
        if op == "rope_append":
            tokens = _log(rng, 1, 8192)
            c = _rope("", tokens, q_heads, kv_heads, D, rng.choice([D, D, D // 2, D // 4]), page, dtype,
                      rng.random() < 0.5, rng.randint(0, tokens // 8))
        elif op == "paged_attention":
            prefix = _log(rng, 1, 16384) if rng.random() < 0.5 else 0
            c = _attn("", _log(rng, 1, 256), q_heads, kv_heads, D, page, dtype, _log(rng, 1, 65536), prefix)
        else:
            group = rng.choice([32, 64, 128])
            c = _w4("", _log(rng, 1, 64), _log(rng, 64, 28672), group * _log(rng, 1, 14336 // group), group, dtype,
                    rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
        del c["name"]
        if _cost(c) <= most[op]:
            return c


def _lens(c):
    """Own keys of each sequence: spread over 1 .. longest, the longest among them; in a batch of
    eight or more one sequence has none."""
    B, longest = c["batch"], c["longest"]
    lens = [1 + (longest - 1) * ((b * 7 + B - 1) % B + 1) // B for b in range(B)]
    lens[B // 2] = longest
    if B >= 8:
        lens[1] = 0
    return lens


def work(c):
    if c["op"] == "rope_append":
        t, hq, hk, D = c["tokens"] - c["pad"], c["q_heads"], c["kv_heads"], c["D"]
        rows = c["tokens"] * hq + 2 * t * hk
        return {"bytes": 2 * rows * D * 2 + t * c["rot"] * 4 + c["tokens"] * 8, "flops": 3 * (c["tokens"] * hq + t * hk) * c["rot"]}
    if c["op"] == "paged_attention":
        lens, hq, hk, D, B = _lens(c), c["q_heads"], c["kv_heads"], c["D"], c["batch"]
        keys, p = sum(lens), c["prefix"]
        pages = sum(-(-n // c["page"]) for n in lens) + -(-p // c["page"])
        return {"bytes": (keys + p) * hk * D * 4 + 2 * B * hq * D * 2 + 4 * pages + 4 * B,
                "flops": 4 * D * hq * (keys + B * p)}
    M, N, K, G = c["M"], c["N"], c["K"], c["group"]
    extra = 2 * N * c["bias"] + 2 * M * N * c["residual"] + N * K // G * c["zeros"]
    return {"bytes": N * K // 2 + 2 * N * K // G + 2 * M * K + 2 * M * N + extra, "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return dev, g


def prepare(c, seed):
    dev, g = _gen(seed)
    dt = DT.get(c["dtype"])

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    if c["op"] == "rope_append":
        t, hq, hk, D, page, rot = c["tokens"], c["q_heads"], c["kv_heads"], c["D"], c["page"], c["rot"]
        pages = -(-(2 * t) // page) + 2                 # a pool with free pages, the last one never used
        order = torch.randperm((pages - 1) * page, generator=g, device=dev)
        slots = order[:t].to(torch.int32)
        pos = torch.randint(0, 32768, (t,), generator=g, device=dev, dtype=torch.int32)
        if c["pad"]:
            slots[torch.randperm(t, generator=g, device=dev)[:c["pad"]]] = -1
        freq = 500000.0 ** (-torch.arange(0, rot // 2, dtype=torch.float64, device=dev) / (rot // 2))
        ang = torch.arange(32768, dtype=torch.float64, device=dev)[:, None] * freq
        return {"case": c, "qkv": normal(t, (hq + 2 * hk) * D), "cos_sin": torch.cat([ang.cos(), ang.sin()], 1).float(),
                "pos": pos, "slots": slots, "q": torch.empty(t, hq, D, dtype=dt, device=dev),
                "k": normal(pages, hk, page, D), "v": normal(pages, hk, page, D)}
    if c["op"] == "paged_attention":
        B, hq, hk, D, page, p = c["batch"], c["q_heads"], c["kv_heads"], c["D"], c["page"], c["prefix"]
        lens = _lens(c)
        counts = [-(-n // page) for n in lens]
        shared = -(-p // page)
        pages = sum(counts) + shared + 1
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)   # entries past a length are never read
        at = shared
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        return {"case": c, "q": normal(B, hq, D), "k": normal(pages, hk, page, D), "v": normal(pages, hk, page, D),
                "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
                "prefix_table": order[:shared].contiguous() if p else None, "scale": 1.0 / math.sqrt(D),
                "o": torch.empty(B, hq, D, dtype=dt, device=dev)}
    M, N, K, G = c["M"], c["N"], c["K"], c["group"]
    wq = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    scales = ((0.5 + torch.rand(N, K // G, generator=g, device=dev)) * 0.2 / math.sqrt(K)).to(dt)
    return {"case": c, "x": normal(M, K), "wq": wq, "scales": scales,
            "zeros": torch.randint(4, 12, (N, K // G), generator=g, device=dev, dtype=torch.uint8) if c["zeros"] else None,
            "bias": normal(N, std=0.1) if c["bias"] else None, "residual": normal(M, N) if c["residual"] else None,
            "y": torch.empty(M, N, dtype=dt, device=dev)}


# ----------------------------------------------------------------------------- plain forms
def _plain_rope(s):
    c = s["case"]
    t, hq, hk, D, rot, page = c["tokens"], c["q_heads"], c["kv_heads"], c["D"], c["rot"], c["page"]
    x = s["qkv"].view(t, hq + 2 * hk, D)
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    qk = x[:, :hq + hk].float()
    if c["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(x.dtype)
    live = (s["slots"] >= 0)[:, None, None]
    spare = s["k"].shape[0] * page - 1                  # a padded row rewrites the spare slot with its own content
    at = torch.where(s["slots"] >= 0, s["slots"], spare).long()
    pg, off = at // page, at % page
    s["k"][pg, :, off] = torch.where(live, qk[:, hq:], s["k"][pg, :, off])
    s["v"][pg, :, off] = torch.where(live, x[:, hq + hk:], s["v"][pg, :, off])
    return [qk[:, :hq], s["k"], s["v"]]


def _plain_attention(s):
    c = s["case"]
    B, hq, hk, D, page, p = c["batch"], c["q_heads"], c["kv_heads"], c["D"], c["page"], c["prefix"]
    q = s["q"].view(B, hk, hq // hk, D).float() * s["scale"]
    dev = q.device
    pos = torch.arange(s["table"].shape[1] * page, device=dev)
    seen = pos[None, :] < s["lens"][:, None]
    pg = s["table"].clamp(min=0)[:, pos // page].long()
    k, v = s["k"][pg, :, pos % page].float(), s["v"][pg, :, pos % page].float()       # [B, L, hk, D]
    scores = torch.einsum("bhgd,blhd->bhgl", q, k).masked_fill(~seen[:, None, None, :], -math.inf)
    if p:
        pos = torch.arange(p, device=dev)
        pg = s["prefix_table"][pos // page].long()
        kp, vp = s["k"][pg, :, pos % page].float(), s["v"][pg, :, pos % page].float()  # [p, hk, D]
        scores = torch.cat([torch.einsum("bhgd,lhd->bhgl", q, kp), scores], -1)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = (scores - top).exp()
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", e[..., p:], v)
    if p:
        o = o + torch.einsum("bhgl,lhd->bhgd", e[..., :p], vp)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))      # a row that sees no key gives zeros
    return o.reshape(B, hq, D).to(s["q"].dtype)


def _plain_w4(s):
    c = s["case"]
    N, K, G = c["N"], c["K"], c["group"]
    nib = torch.stack([s["wq"] & 15, s["wq"] >> 4], -1).view(N, K // G, G).float()
    zero = s["zeros"].float()[..., None] if c["zeros"] else 8.0
    w = ((nib - zero) * s["scales"].float()[..., None]).view(N, K)
    y = s["x"].float() @ w.t()
    if c["bias"]:
        y = y + s["bias"].float()
    if c["gelu"]:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def run(s):
    c = s["case"]
    if own:
        import epilogue_chains_gb300 as fc
        if c["op"] == "rope_append":
            fc.fuse_rope_append(s["qkv"], s["cos_sin"], s["pos"], s["slots"], s["q"], s["k"], s["v"],
                                interleaved=c["interleaved"])
            return [s["q"], s["k"], s["v"]]
        if c["op"] == "paged_attention":
            fc.fuse_paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["o"], s["scale"],
                                    prefix_table=s["prefix_table"], prefix_len=c["prefix"])
            return s["o"]
        fc.fuse_w4_gemv(s["x"], s["wq"], s["scales"], s["y"], zeros=s["zeros"], bias=s["bias"],
                        residual=s["residual"], gelu=c["gelu"])
        return s["y"]
    if c["op"] == "rope_append":
        return _plain_rope(s)
    return _plain_attention(s) if c["op"] == "paged_attention" else _plain_w4(s)


# ----------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope_append":
        hq, hk, D, rot, page = c["q_heads"], c["kv_heads"], c["D"], c["rot"], c["page"]
        x = s["qkv"].double().view(c["tokens"], hq + 2 * hk, D)
        tab = s["cos_sin"].double()[s["pos"].long()]
        turn = torch.complex(tab[:, :rot // 2], tab[:, rot // 2:])[:, None, :]      # e^(i angle)
        first = torch.arange(0, rot, 2, device=x.device) if c["interleaved"] else torch.arange(rot // 2, device=x.device)
        second = first + (1 if c["interleaved"] else rot // 2)
        z = torch.complex(x[:, :hq + hk, first], x[:, :hq + hk, second]) * turn
        y = x.clone()
        y[:, :hq + hk, first], y[:, :hq + hk, second] = z.real, z.imag
        k, v = s["k"].double(), s["v"].double()
        live = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][live].long()
        k[at // page, :, at % page] = y[live, hq:hq + hk]
        v[at // page, :, at % page] = y[live, hq + hk:]
        return [y[:, :hq], k, v]
    if c["op"] == "paged_attention":
        B, hq, hk, D, page, p = c["batch"], c["q_heads"], c["kv_heads"], c["D"], c["page"], c["prefix"]
        o = torch.zeros(B, hq, D, dtype=torch.float64, device=s["q"].device)

        def rows(cache, pages, n):            # [hk, n, D] of the first n keys in these pages
            return cache[pages.long()].double().transpose(0, 1).reshape(hk, -1, D)[:, :n]

        shared = [rows(s[n], s["prefix_table"], p) for n in "kv"] if p else None
        for b, n in enumerate(_lens(c)):
            pages = s["table"][b, :-(-n // page)]
            parts = ([shared] if p else []) + ([[rows(s["k"], pages, n), rows(s["v"], pages, n)]] if n else [])
            if parts:
                q = s["q"][b].double().view(hk, hq // hk, D)
                z = torch.cat([q @ k.transpose(1, 2) for k, _ in parts], 2) * s["scale"]
                w = torch.softmax(z, 2)
                at = 0
                for k, v in parts:
                    o[b] += (w[:, :, at:at + k.shape[1]] @ v).reshape(hq, D)
                    at += k.shape[1]
        return o
    N, K, G = c["N"], c["K"], c["group"]
    w = torch.empty(N, K, dtype=torch.float64, device=s["x"].device)
    w[:, 0::2], w[:, 1::2] = (s["wq"] % 16).double(), (s["wq"] // 16).double()
    w -= s["zeros"].double().repeat_interleave(G, 1) if c["zeros"] else 8
    w *= s["scales"].double().repeat_interleave(G, 1)
    y = torch.einsum("mk,nk->mn", s["x"].double(), w)
    if c["bias"]:
        y += s["bias"].double()
    if c["gelu"]:
        y = y * torch.special.ndtr(y)
    if c["residual"]:
        y += s["residual"].double()
    return y
