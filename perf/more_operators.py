"""The measured cases of the operators that read whole prompts.

A served model meets a prompt before it answers: the projections of all its tokens, for which both the
weights and the activations can be held in 4-bit floating point with one power-of-two scale per 32 values
(``fuse_mxfp4_quantize``, ``fuse_mxfp4_gemm``); causal attention of the packed prompts over the paged cache
that ``fuse_rope_append`` has filled, earlier turns included (``fuse_prompt_attention``); and, of the logits
at the end, the log probabilities of the given tokens with the entropy and the best alternatives
(``fuse_token_logprobs``).

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()`` one pass (the plain torch
form, or the library's calls where ``own`` is true), ``work()`` what a pass cannot do without and
``exact()`` the same values in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def _attn(name, batch, longest, cached, q_heads, kv_heads, D, page, dtype, pad):
    return {"name": name, "op": "prompt_attention", "batch": batch, "longest": longest, "cached": cached,
            "q_heads": q_heads, "kv_heads": kv_heads, "D": D, "page": page, "dtype": dtype, "pad": pad}


def _round_trip(name, rows, cols, dtype):
    return {"name": name, "op": "mxfp4_quantize", "rows": rows, "cols": cols, "dtype": dtype}


def _project(name, M, N, K, dtype, bias, gelu, residual):
    return {"name": name, "op": "mxfp4_gemm", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias, "gelu": gelu,
            "residual": residual}


def _score(name, rows, vocab, top, dtype, scale, masked, pad):
    return {"name": name, "op": "token_logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "scale": scale, "masked": masked, "pad": pad}


def listed():
    return [
        # a short first message of one user: latency
        _attn("prompt of 17", 1, 17, 0, 32, 8, 128, 16, "bf16", 0),
        # a packed batch of prompts of every length up to 1024, five padded rows behind them
        _attn("32 prompts to 1024", 32, 1024, 0, 32, 8, 128, 32, "f16", 5),
        # one long document
        _attn("prompt of 16384", 1, 16384, 0, 32, 8, 128, 64, "bf16", 0),
        # the next turn of a long conversation: few rows, many keys
        _attn("64 after 65536", 1, 64, 65536, 32, 8, 128, 64, "bf16", 0),
        # 16 ungrouped heads of 256, 8 sequences (this repository's attention benchmark, over a cache)
        _attn("8 prompts to 2048, D 256", 8, 2048, 0, 16, 16, 256, 128, "bf16", 0),
        # the merged gate and up weight quantised, and read back
        _round_trip("quantise 28672 x 4096", 28672, 4096, "bf16"),
        # the output projection of one token (this repository's GEMM width), its activations quantised first
        _project("fp4 1 x 4096 x 4096", 1, 4096, 4096, "bf16", False, False, True),
        # the down projection of a short prompt, ragged against every tile
        _project("fp4 100 x 4096 x 14336", 100, 4096, 14336, "f16", True, False, True),
        # gate and up merged for a long prompt, bias and activation joined
        _project("fp4 8192 x 28672 x 4096", 8192, 28672, 4096, "bf16", True, True, False),
        # one sampled token's report
        _score("score 1 x 128000", 1, 128000, 20, "f32", 1.0, False, 0),
        # a decode batch under a grammar that forbids most tokens, odd vocabulary, sharpened, padded rows
        _score("score 48 x 50257, masked", 48, 50257, 5, "bf16", 1.25, True, 3),
        # every token of a long prompt scored
        _score("score 4096 x 131072", 4096, 131072, 5, "bf16", 1.0, False, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    op = rng.choice(["prompt_attention", "prompt_attention", "mxfp4_gemm", "mxfp4_gemm", "mxfp4_quantize", "token_logprobs"])
    while True:
        dtype = rng.choice(["bf16", "f16"])
        if op == "prompt_attention":
            kv_heads = rng.choice([1, 2, 4, 8])
            q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            cached = _log(rng, 1, 65536) if rng.random() < 0.4 else 0
            c = _attn("", _log(rng, 1, 64), _log(rng, 1, 16384), cached, q_heads, kv_heads, rng.choice([64, 128, 128, 256]),
                      rng.choice([16, 32, 64, 128]), dtype, rng.randint(0, 7))
            lens, own_lens = _lens(c)
            # (the plain form holds the scores of the padded batch)
            if c["batch"] * max(lens) * max(own_lens) * q_heads > 2 ** 33 or c["batch"] * max(lens) * kv_heads * c["D"] > 2 ** 31:
                continue
        elif op == "mxfp4_quantize":
            c = _round_trip("", _log(rng, 1, 28672), 32 * _log(rng, 1, 448), rng.choice(["bf16", "f16", "f32"]))
        elif op == "mxfp4_gemm":
            c = _project("", _log(rng, 1, 8192), _log(rng, 1, 28672), 32 * _log(rng, 1, 448), dtype, rng.random() < 0.5,
                         rng.random() < 0.3, rng.random() < 0.5)
        else:
            rows = _log(rng, 1, 8192)
            c = _score("", rows, _log(rng, 1000, 262144), rng.choice([0, 1, 5, 20, 32]), rng.choice(["bf16", "f16", "f32"]),
                       rng.choice([1.0, 1.0, 0.7, 1.6]), rng.random() < 0.3, rng.randint(0, rows // 8))
        del c["name"]
        if _cost(c) <= most[op]:
            return c


def _spread(n, most, least, step):
    """n whole numbers spread over least .. most, the largest among them."""
    v = [least + (most - least) * ((b * step + n - 1) % n + 1) // n for b in range(n)]
    v[n // 2] = most
    return v


def _lens(c):
    """Keys in the cache and new tokens of each sequence: new tokens spread over 1 .. longest (in a batch
    of eight or more one sequence has none), earlier keys over 0 .. cached."""
    own_lens = _spread(c["batch"], c["longest"], 1, 7)
    if c["batch"] >= 8:
        own_lens[1] = 0
    before = _spread(c["batch"], c["cached"], 0, 5)
    return [p + n for p, n in zip(before, own_lens)], own_lens


def _scale_bytes(rows, cols):
    return -(-rows // 128) * -(-cols // 128) * 512


def work(c):
    if c["op"] == "prompt_attention":
        lens, own_lens = _lens(c)
        hq, hk, D = c["q_heads"], c["kv_heads"], c["D"]
        pairs = sum(n * (k - n) + n * (n + 1) // 2 for k, n in zip(lens, own_lens))
        keys = sum(k for k, n in zip(lens, own_lens) if n)      # a sequence without new tokens is not read
        pages = sum(-(-k // c["page"]) for k, n in zip(lens, own_lens) if n)
        return {"bytes": 4 * keys * hk * D + 4 * sum(own_lens) * hq * D + 4 * pages + 8 * c["batch"], "flops": 4 * D * hq * pairs}
    if c["op"] == "mxfp4_quantize":
        n, size = c["rows"] * c["cols"], 4 if c["dtype"] == "f32" else 2
        # quantised, and read back: the packed form is an output of the first and an input of the second
        return {"bytes": 2 * n * size + 2 * (n // 2 + n // 32), "flops": 4 * n}
    if c["op"] == "mxfp4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        extra = 2 * N * c["bias"] + 2 * M * N * c["residual"]
        return {"bytes": N * K // 2 + N * K // 32 + 2 * M * K + 2 * M * N + extra, "flops": 2 * M * N * K}
    rows, V, size = c["rows"], c["vocab"], 4 if c["dtype"] == "f32" else 2
    return {"bytes": rows * (V * size + 4 + 8 + 8 * c["top"]), "flops": 6 * rows * V}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return dev, g


def prepare(c, seed):
    dev, g = _gen(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    if c["op"] == "prompt_attention":
        B, hq, hk, D, page = c["batch"], c["q_heads"], c["kv_heads"], c["D"], c["page"]
        lens, own_lens = _lens(c)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 1
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)   # entries past a length are never read
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        starts = [0]
        for n in own_lens:
            starts.append(starts[-1] + n)
        tokens = starts[-1] + c["pad"]
        return {"case": c, "q": normal(tokens, hq, D), "k": normal(pages, hk, page, D), "v": normal(pages, hk, page, D),
                "table": table, "cu": torch.tensor(starts, dtype=torch.int32, device=dev),
                "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(D),
                "o": torch.zeros(tokens, hq, D, dtype=dt, device=dev)}
    if c["op"] == "mxfp4_quantize":
        R, K = c["rows"], c["cols"]
        # values of a trained weight's spread, a few rows far larger, one all zeros
        x = normal(R, K, std=0.02)
        big = torch.randperm(R, generator=g, device=dev)[:max(1, R // 64)]
        x[big] *= 40.0
        x[big[0], :K // 2] = 0.0
        return {"case": c, "x": x, "q": torch.empty(R, K // 2, dtype=torch.uint8, device=dev),
                "s": torch.empty(_scale_bytes(R, K), dtype=torch.uint8, device=dev), "y": torch.empty_like(x)}
    if c["op"] == "mxfp4_gemm":
        M, N, K = c["M"], c["N"], c["K"]
        wq = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
        base = 127 + round(-math.log2(2.93 * math.sqrt(K)))         # sums of about one
        ws = torch.randint(base - 1, base + 2, (N, K // 32), generator=g, device=dev, dtype=torch.uint8)
        # the scales as the product takes them: tiles of 128 rows by 4 blocks, 32 rows of 16 bytes each
        nb = -(-K // 128) * 4
        full = torch.zeros(-(-N // 128) * 128, nb, dtype=torch.uint8, device=dev)
        full[:N, :K // 32] = ws
        tiled = full.view(-1, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()
        x = normal(M, K)
        x[:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 256)]] *= 8.0     # outlying channels
        return {"case": c, "x": x, "wq": wq, "ws": ws, "tiled": tiled,
                "bias": normal(N, std=0.1) if c["bias"] else None, "residual": normal(M, N) if c["residual"] else None,
                "xq": torch.empty(M, K // 2, dtype=torch.uint8, device=dev),
                "xs": torch.empty(_scale_bytes(M, K), dtype=torch.uint8, device=dev),
                "y": torch.empty(M, N, dtype=dt, device=dev)}
    R, V, top = c["rows"], c["vocab"], c["top"]
    logits = normal(R, V, std=2.5)
    tokens = torch.randint(0, V, (R,), generator=g, device=dev, dtype=torch.int32)
    rows = torch.arange(R, device=dev)
    sure = torch.rand(R, generator=g, device=dev) < 0.6              # most tokens of a text are likely ones
    logits[rows, tokens.long()] += torch.where(sure, 12.0, 0.0).to(dt)
    if c["masked"]:
        keep = torch.rand(V, generator=g, device=dev) < 0.05
        keep[torch.randperm(V, generator=g, device=dev)[:64]] = True
        keep = keep[None, :].repeat(R, 1)
        keep[rows, tokens.long()] = True
        logits = torch.where(keep, logits, torch.full((), -math.inf, dtype=dt, device=dev))
    if c["pad"]:
        tokens[torch.randperm(R, generator=g, device=dev)[:c["pad"]]] = -1      # rows without a given token
    return {"case": c, "logits": logits, "tokens": tokens, "logprob": torch.empty(R, device=dev),
            "entropy": torch.empty(R, device=dev), "top_logprob": torch.empty(R, top, device=dev),
            "top_index": torch.empty(R, top, dtype=torch.int32, device=dev)}


# ----------------------------------------------------------------------------- plain forms
def _plain_attention(s):
    c = s["case"]
    B, hq, hk, D, page = c["batch"], c["q_heads"], c["kv_heads"], c["D"], c["page"]
    lens, own_lens = _lens(c)
    dev = s["q"].device
    i = torch.arange(max(own_lens), device=dev)
    begin, count, keys = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    there = i[None, :] < count[:, None]                                              # [B, n]
    row = torch.where(there, begin[:, None] + i, torch.zeros_like(begin)[:, None])
    q = s["q"][row].view(B, -1, hk, hq // hk, D).float() * s["scale"]
    pos = torch.arange(max(lens), device=dev)
    last = (keys - count)[:, None] + i                                               # the last key a query sees
    seen = (pos[None, None, :] <= last[:, :, None])                                  # [B, n, L]
    used = pos[None, :] < keys[:, None]
    pg = torch.where(used, s["table"][:, pos // page], torch.zeros((), dtype=torch.int32, device=dev)).long()
    off = (pos % page).expand_as(pg)
    k, v = s["k"][pg, :, off].float(), s["v"][pg, :, off].float()                    # [B, L, hk, D]
    scores = torch.einsum("bnhgd,blhd->bhgnl", q, k)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bhgnd", scores, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))                       # a row that sees no key gives zeros
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, hq, D).to(s["q"].dtype)
    s["o"][row[there]] = o[there]
    return s["o"]


def _power(e):
    """2^e for whole -126 <= e <= 127, exactly (a power function may miss it by a rounding)."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_quantize(x):
    """The values that x [R, K] has in 4 bits: per 32 of them a scale 2^e with 2^(e + 2) <= max |x| < 2^(e + 3),
    each value divided by it and rounded to 0, 1/2, 1, 3/2, 2, 3, 4 or 6, ties to the even mantissa."""
    v = x.float().view(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.zeros((), dtype=torch.int32, device=x.device)).clamp(min=-126)
    v = v / _power(e)
    step = _power(torch.frexp(v).exponent.clamp(min=1) - 2)
    return ((torch.round(v / step) * step).clamp(-6.0, 6.0) * _power(e)).view_as(x)


def _plain_gemm(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=s["x"].device)
    values = torch.cat([values, -values])
    w = values[torch.stack([s["wq"] & 15, s["wq"] >> 4], -1).view(N, K).int()].view(N, K // 32, 32)
    w = (w * _power(s["ws"].int()[..., None] - 127)).view(N, K)
    y = _plain_quantize(s["x"]) @ w.t()
    if c["bias"]:
        y = y + s["bias"].float()
    if c["gelu"]:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_score(s):
    c = s["case"]
    x = s["logits"].float()
    z = x * c["scale"]
    z = z - z.amax(-1, keepdim=True)
    p = z.exp()
    total = p.sum(-1, keepdim=True)
    lse = total.log()
    entropy = lse[:, 0] - torch.where(p > 0, p * z, torch.zeros_like(p)).sum(-1) / total[:, 0]
    given = torch.gather(z - lse, 1, s["tokens"].clamp(min=0).long()[:, None])[:, 0]
    given = torch.where(s["tokens"] >= 0, given, torch.zeros_like(given))            # a padded row
    if not c["top"]:
        return [given, entropy]
    # the largest logits, of equal ones the first: keys whose order is that of (logit, -index)
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * 2 ** 31 - torch.arange(c["vocab"], device=x.device)
    at = torch.topk(order, c["top"], -1).indices
    return [given, entropy, torch.gather(z - lse, 1, at), at.int()]


def run(s):
    c = s["case"]
    if own:
        import epilogue_chains_gb300 as fc
        if c["op"] == "prompt_attention":
            fc.fuse_prompt_attention(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], s["o"], s["scale"])
            return s["o"]
        if c["op"] == "mxfp4_quantize":
            fc.fuse_mxfp4_quantize(s["x"], s["q"], s["s"])
            fc.fuse_mxfp4_dequantize(s["q"], s["s"], s["y"])
            return s["y"]
        if c["op"] == "mxfp4_gemm":
            fc.fuse_mxfp4_quantize(s["x"], s["xq"], s["xs"])
            fc.fuse_mxfp4_gemm(s["xq"], s["xs"], s["wq"], s["tiled"], s["y"], bias=s["bias"], residual=s["residual"],
                               gelu=c["gelu"])
            return s["y"]
        if not c["top"]:
            fc.fuse_token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], scale=c["scale"])
            return [s["logprob"], s["entropy"]]
        fc.fuse_token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], top_logprob=s["top_logprob"],
                               top_index=s["top_index"], scale=c["scale"])
        return [s["logprob"], s["entropy"], s["top_logprob"], s["top_index"]]
    if c["op"] == "prompt_attention":
        return _plain_attention(s)
    if c["op"] == "mxfp4_quantize":
        return _plain_quantize(s["x"]).to(s["x"].dtype)
    return _plain_gemm(s) if c["op"] == "mxfp4_gemm" else _plain_score(s)


# ----------------------------------------------------------------------------- 64 bits
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_quantize(x):
    """The scale by comparison with the powers of two, values by the nearest of the eight (of two as near, the
    one of even code)."""
    v = x.double().view(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    powers = torch.tensor([2.0 ** e for e in range(-126, 129)], dtype=torch.float64, device=x.device)
    scale = powers[(torch.searchsorted(powers, top, right=True) - 3).clamp(min=0)]     # largest with 4 scale <= top
    a = (v / scale).abs()
    out = torch.zeros_like(a)
    for n in range(1, 8):
        mid = (GRID[n - 1] + GRID[n]) / 2
        out = torch.where((a >= mid) if n % 2 == 0 else (a > mid), torch.full_like(a, GRID[n]), out)
    return (torch.sign(v) * out * scale).view_as(x)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "prompt_attention":
        hq, hk, D, page = c["q_heads"], c["kv_heads"], c["D"], c["page"]
        o = s["o"].double()
        at = 0
        for b, (L, n) in enumerate(zip(*_lens(c))):
            pages = s["table"][b, :-(-L // page)].long()
            for h in range(hk if n else 0):
                k, v = (s[x][pages, h].reshape(-1, D)[:L].double() for x in "kv")
                heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
                for i in range(0, n, 1024):          # queries i .. of the sequence see keys up to their own
                    m = min(1024, n - i)
                    last = L - n + i + m
                    z = torch.einsum("mgd,ld->gml", s["q"][at + i:at + i + m, heads].double(), k[:last]) * s["scale"]
                    z = z + torch.full((m, last), -math.inf, dtype=z.dtype, device=z.device).triu(L - n + i + 1)
                    o[at + i:at + i + m, heads] = torch.einsum("gml,ld->mgd", torch.softmax(z, -1), v[:last])
            at += n
        return o
    if c["op"] == "mxfp4_quantize":
        return _exact_quantize(s["x"])
    if c["op"] == "mxfp4_gemm":
        N, K = c["N"], c["K"]
        grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=s["x"].device)
        w = torch.empty(N, K, dtype=torch.float64, device=s["x"].device)
        w[:, 0::2], w[:, 1::2] = grid[(s["wq"] % 16).long()], grid[(s["wq"] // 16).long()]
        w *= torch.tensor([2.0 ** (e - 127) for e in range(255)], dtype=torch.float64, device=w.device)[s["ws"].long()].repeat_interleave(32, 1)
        y = torch.einsum("mk,nk->mn", _exact_quantize(s["x"]), w)
        if c["bias"]:
            y += s["bias"].double()
        if c["gelu"]:
            y = y * torch.special.ndtr(y)
        if c["residual"]:
            y += s["residual"].double()
        return y
    given, entropy, best, index = [], [], [], []
    for a in range(0, c["rows"], 512):               # (a block of rows at a time)
        x = s["logits"][a:a + 512].double()
        tokens = s["tokens"][a:a + 512].long()
        lp = torch.log_softmax(x * c["scale"], -1)
        pick = torch.gather(lp, 1, tokens.clamp(min=0)[:, None])[:, 0]
        given.append(torch.where(tokens >= 0, pick, torch.zeros_like(pick)))
        entropy.append(torch.special.entr(lp.exp()).sum(-1))
        if c["top"]:
            at = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            best.append(torch.gather(lp, 1, at))
            index.append(at.int())
    out = [torch.cat(given), torch.cat(entropy)]
    return out + [torch.cat(best), torch.cat(index)] if c["top"] else out
