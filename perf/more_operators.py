"""Measured cases of the rotary positions with several axes (queries and keys of
video tokens, forward and backward) and of the serving calls on a cache kept in
8 bits: appending rotated keys and values with a scale per block of 16 tokens
and head, the attention of one new token per sequence over it, the same with
the attention weight that each page receives, and the eviction of the pages
that received least.

``own = False`` runs each operator's plain form (elementary torch operations
in fp32), ``own = True`` the framework's calls (``vsa.AxialRope``,
``vsa.PagedCache``).
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128
BLOCK = 16  # tokens that share a scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def _rotate_case(name, back, B, grid, Hq, Hkv, dims, layout, dtype, interleaved, base=10000.0, apart=True):
    """grid: frames x rows x columns; dims: rotated dims of each axis, as text;
    apart: q and k are parts of one projection's output."""
    c = dict(op="back" if back else "rotate", B=B, T=grid[0], H=grid[1], W=grid[2], Hq=Hq, Hkv=Hkv, dims=dims,
             layout=layout, dtype=dtype, interleaved=interleaved, base=base, apart=apart)
    return dict(c, name=name) if name else c


def _cache_case(name, op, B, Hq, Hkv, page, layout, dtype, lo, hi, new_lo=1, new_hi=1, rot=D, interleaved=False, kv="e4m3",
                topk=0, decay=1.0, keep=0, keep_first=0, keep_last=1):
    """lo..hi: tokens in the cache; new_lo..new_hi: of those the appended ones;
    kv: what the cache holds; topk: pages attended to (0: all)."""
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, page=page, layout=layout, dtype=dtype, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi,
             rot=rot, interleaved=interleaved, kv=kv, topk=topk, decay=decay, keep=keep, keep_first=keep_first,
             keep_last=keep_last)
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of the 76,800-token video workload, straight out of the projection
        _rotate_case("rotate-video", False, 1, (20, 48, 80), 40, 40, "44,42,42", "bshd", "bf16", True),
        # two small images with grouped heads: the launch itself is the cost
        _rotate_case("rotate-image", False, 2, (1, 15, 17), 12, 3, "16,56,56", "bshd", "fp16", False),
        # gradients of a video whose last tiles are clipped, head-major
        _rotate_case("back-ragged-video", True, 1, (21, 45, 80), 24, 24, "44,42,42", "bhsd", "bf16", True, apart=False),
        # gradients of packed sequences with two axes (row, column) on part of the head
        _rotate_case("back-packed", True, 1, (1, 57, 101), 12, 3, "48,48", "tnd", "fp16", False),
        # next tokens of a serving batch, contexts of all lengths
        _cache_case("append-batch-tokens", "append", 64, 32, 8, 64, "bhsd", "bf16", 100, 8000),
        # a long video context of 24 heads written at once, 256-token tiles
        _cache_case("append-long-prompt", "append", 2, 24, 24, 256, "bshd", "bf16", 14000, 16000, 14000, 16000,
                    interleaved=True),
        # a serving batch of ragged contexts, grouped heads: the ordinary decode step
        _cache_case("attend-batch", "attend", 64, 32, 8, 64, "bshd", "bf16", 37, 16000),
        # one long video context, every head with its own keys (480 tiles of 256)
        _cache_case("attend-long-video", "attend", 1, 24, 24, 256, "bhsd", "bf16", 122880, 122880),
        # a short context of one sequence with its pages' weights: latency
        _cache_case("weigh-short", "weigh", 1, 12, 3, 16, "bshd", "fp16", 401, 401),
        # the batch's decode step with the weights that an eviction goes by, older ones fading
        _cache_case("weigh-batch", "weigh", 64, 32, 8, 64, "bshd", "bf16", 37, 16000, decay=0.98),
        # a batch over its budget of pages: each sequence gives up its least attended ones
        _cache_case("evict-batch", "evict", 64, 32, 8, 64, "bhsd", "bf16", 2000, 16000, keep=64, keep_first=1, keep_last=4),
        # one long context in small pages
        _cache_case("evict-long", "evict", 1, 24, 24, 16, "bshd", "bf16", 122880, 122880, keep=4000, keep_first=4,
                    keep_last=8),
    ]


def draw(rng):
    """A case of the same ranges: single tokens to long videos, contexts of 1
    to 131,072 tokens, groups of 1 to 16 heads, every page size."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("rotate", "back", "append", "attend", "attend", "weigh", "weigh", "evict"))
    Hkv = rng.choice((1, 2, 3, 4, 8, 12, 24))
    G = rng.choice((1, 2, 3, 4, 5, 8, 16)) if Hkv <= 8 else rng.choice((1, 2))
    style, dtype = rng.random() < 0.5, rng.choice(("bf16", "fp16"))
    if op in ("rotate", "back"):
        dims = rng.choice(("44,42,42", "16,56,56", "32,48,48", "128", "64,64", "48,48", "24,20,20", "32,32,32,32"))
        layout = rng.choice(("bshd", "bhsd", "tnd"))
        B = 1 if layout == "tnd" else rng.choice((1, 1, 2, 3))
        most = 5000000 // (B * Hkv * (G + 1))
        T = log_int(1, 24)
        H = log_int(1, max(2, min(64, most // T)))
        W = log_int(1, max(2, min(96, most // (T * H))))
        return _rotate_case(None, op == "back", B, (T, H, W), G * Hkv, Hkv, dims, layout, dtype, style,
                            base=rng.choice((100.0, 10000.0, 500000.0)), apart=rng.random() < 0.5)
    common = dict(page=rng.choice((16, 32, 64, 128, 256)), layout=rng.choice(("bshd", "bhsd")), dtype=dtype)
    B, page = log_int(1, 96), common["page"]
    if op == "append":
        n = log_int(1, max(2, min(4096, 600000 // (B * Hkv * (G + 2)))))
        hi = n + log_int(1, 4096)
        return _cache_case(None, op, B, G * Hkv, Hkv, lo=n, hi=hi, new_lo=max(1, n // rng.choice((1, 2, 8))), new_hi=n,
                           rot=rng.choice((0, 32, 64, 96, 128, 128)), interleaved=style, **common)
    if op == "evict":
        pages = log_int(4, max(5, min(8000, 1500000 // (B * Hkv))))
        first, last = rng.choice((0, 1, 3)), rng.choice((1, 2))
        hi = pages * page - rng.randrange(page)
        return _cache_case(None, op, B, G * Hkv, Hkv, lo=max(1, hi // rng.choice((1, 2, 16))), hi=hi,
                           keep=max(first + last, rng.randrange(1, pages + 1)), keep_first=first, keep_last=last, **common)
    budget = 2500000  # keys x key heads over the batch
    hi = log_int(1, max(2, min(131072, budget // (B * Hkv))))
    lo = max(1, hi // rng.choice((1, 2, 16, 256)))
    pages = -(-hi // page)
    topk = rng.choice((0, log_int(1, max(2, pages)))) if op == "weigh" else rng.choice((0, 0, log_int(1, max(2, pages))))
    return _cache_case(None, op, B, G * Hkv, Hkv, lo=lo, hi=hi, topk=min(topk, pages),
                       kv=rng.choice(("e4m3", "e4m3", "16")) if op == "weigh" else "e4m3",
                       decay=rng.choice((1.0, 0.9, 0.0)) if op == "weigh" else 1.0, **common)


def _sizes(case):
    """(lengths, new tokens) per sequence: spread over [lo, hi] evenly in
    their logarithm, in an order of the case's own, the longest among them."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))

    def spread(lo, hi):
        n = [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(case["B"])]
        n[r.randrange(len(n))] = hi
        return n

    lens = spread(case["lo"], case["hi"])
    if case["op"] != "append":
        return lens, [0] * len(lens)
    new = spread(case["new_lo"], case["new_hi"])
    return [max(a, b) for a, b in zip(lens, new)], new


def _read_back(lens, new):
    """Tokens of each sequence in the blocks that new ones are written to."""
    return [n - (n - m) // BLOCK * BLOCK for n, m in zip(lens, new)]


def work(case):
    op, B, Hq, Hkv = case["op"], case["B"], case["Hq"], case["Hkv"]
    rows = 256  # bytes of one head of one token in 16 bits
    if op in ("rotate", "back"):
        tokens, dims = B * case["T"] * case["H"] * case["W"], [int(n) for n in case["dims"].split(",")]
        return {"bytes": tokens * (Hq + Hkv) * 2 * rows + tokens // B * 4 * len(dims),
                "flops": tokens * (Hq + Hkv) * sum(dims) * 3}
    page = case["page"]
    lens, new = _sizes(case)
    pages = [-(-n // page) for n in lens]
    total, flops = 0, 0
    if op == "append":
        T, back = sum(new), sum(_read_back(lens, new))
        total += T * (2 * Hkv + 2 * Hq) * rows + T * Hkv * (rows + 16 / BLOCK) + T * case["rot"] * 4
        flops += T * (Hq + Hkv) * case["rot"] * 3 + T * Hkv * D * 6
        for n, m in zip(lens, new):  # means of the pages that fill up: their earlier keys, and the mean
            done = n // page - (n - m) // page
            total += Hkv * (done * 512 + ((n - m) % page * D if done else 0))
        total += back * Hkv * 3 * rows  # the blocks' values, read back
    if op in ("attend", "weigh"):
        held = 2 * rows if case["kv"] == "16" else rows + 8 / BLOCK
        keys = [min(n, case["topk"] * page) if case["topk"] else n for n in lens]
        total += sum(keys) * Hkv * held + B * Hq * (2 * rows + 4)
        flops += sum(keys) * Hq * 4 * D
    if op == "weigh":
        total += sum(pages) * Hkv * 8
        flops += sum(keys) * Hq * 2
    if op == "evict":
        total += B * max(pages) * (Hkv + 1) * 8 + sum(max(0, n - case["keep"]) for n in pages) * 4
        flops += sum(pages) * Hkv
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------ inputs

def _dims(case):
    return [int(n) for n in case["dims"].split(",")]


def _freqs(case, device):
    """Radians per step of each pair, and the pair's axis: the usual geometric
    series within the dims of each axis."""
    dims = _dims(case)
    freq = [case["base"] ** (-2.0 * i / n) for n in dims for i in range(n // 2)]
    axis = [a for a, n in enumerate(dims) for _ in range(n // 2)]
    return torch.tensor(freq, dtype=torch.float64, device=device), torch.tensor(axis, device=device)


def _quantize(x, dim):
    """x fp32 in blocks of BLOCK tokens along `dim` (the last dim is D): e4m3
    values, and the scale of each block, the least power of two that brings
    its largest entry within 448."""
    shape = x.shape[:dim] + (x.shape[dim] // BLOCK, BLOCK) + x.shape[dim + 1:]
    x = x.view(shape)
    top = x.abs().amax((dim + 1, x.dim() - 1), keepdim=True)
    m, e = torch.frexp(top)
    scale = torch.ldexp(torch.ones_like(top), torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126))
    q = (x / scale).to(E4M3)
    return q.view(q.shape[:dim] + (-1,) + q.shape[dim + 2:]), scale.squeeze(dim + 1).squeeze(-1)


def prepare(case, seed):
    B, Hq, Hkv, op = (case[k] for k in ("B", "Hq", "Hkv", "op"))
    dtype, dev = DTYPES[case["dtype"]], torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, scale=1.0, kind=dtype):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(kind)

    if op in ("rotate", "back"):
        T, H, W, layout = (case[k] for k in ("T", "H", "W", "layout"))
        S, n = T * H * W, len(_dims(case))
        lead = (S,) if layout == "tnd" else (B, S)
        s = dict(case=case, dtype=dtype)
        if case["apart"]:
            qkv = torch.empty(*lead, Hq + 2 * Hkv, D, dtype=dtype, device=dev).normal_(generator=g)
            s["q"], s["k"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :]
            if layout == "bhsd":
                s["q"], s["k"] = s["q"].transpose(1, 2), s["k"].transpose(1, 2)
        else:
            s["q"], s["k"] = (torch.empty((B, h, S, D) if layout == "bhsd" else lead + (h, D), dtype=dtype,
                                          device=dev).normal_(generator=g) for h in (Hq, Hkv))
        # frame, row and column of each token, behind those of earlier clips
        at = torch.stack(torch.meshgrid(*(torch.arange(m, device=dev) for m in (T, H, W)), indexing="ij"), -1).view(S, 3)
        at = torch.cat((at, at.sum(1, keepdim=True)), 1) + torch.randint(0, 1000, (4,), generator=g, device=dev)
        s["positions"] = (at[:, 1:3] if n == 2 else at[:, 4 - n:] if n == 1 else at[:, :n]).to(torch.int32).contiguous()
        s["freq"], s["axis"] = _freqs(case, dev)
        if own:
            from bwd_tile_mean_gb300 import vsa
            s["rope"] = vsa.AxialRope(_dims(case), base=case["base"], interleaved=case["interleaved"])
        return s

    page, eight = case["page"], case["kv"] == "e4m3"
    lens, new = _sizes(case)
    need = [-(-n // page) for n in lens]
    max_pages, num_pages = max(need), sum(need) + 3
    s = dict(case=case, dtype=dtype, max_pages=max_pages, num_pages=num_pages)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # pages of the pool in random order, as after many requests came and went
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=dev)
    slots = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table[slots] = order[: sum(need)]
    s["page_table"] = table
    shape = (num_pages, page, Hkv, D) if case["layout"] == "bshd" else (num_pages, Hkv, page, D)
    bshd = case["layout"] == "bshd"
    k = v = ks = vs = mean = None
    if op != "evict":  # which reads no keys
        kind = E4M3 if eight else dtype
        k, v = (torch.empty(shape, dtype=kind, device=dev) for _ in range(2))
        if eight:
            ks, vs = (torch.empty(num_pages, Hkv, page // BLOCK, device=dev) for _ in range(2))
        # keys share a direction within their page, so that the pages' weights differ
        centre = randn(num_pages, Hkv, D, scale=0.5, kind=torch.float32)
        for at in range(0, num_pages, 256):
            to = min(num_pages, at + 256)
            x = randn(to - at, Hkv, page, D, kind=torch.float32) + centre[at:to, :, None]
            y = randn(to - at, Hkv, page, D, kind=torch.float32)
            for c, scales, z in ((k, ks, x), (v, vs, y)):
                if eight:
                    z, scales[at:to] = _quantize(z, 2)
                c[at:to] = (z.transpose(1, 2) if bshd else z).to(kind)
        if op == "append":
            mean = torch.zeros(num_pages, Hkv, D, device=dev)
    s.update(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, k_mean=mean)
    if op == "append":
        T, rot = sum(new), case["rot"]
        # the three parts of one projection's output, as a model hands them over
        qkv = randn(T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        back = _read_back(lens, new)
        start, stop = (torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32) for n in (new, back))
        s["cu_seqlens"] = None if new == [1] * B else start
        s.update(T=T, cu_back=stop, T_back=sum(back), cos=None, sin=None)
        if rot:
            freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
            angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * freq[None]
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # pages that these tokens fill up
        filled = [(b, p) for b, (n, m) in enumerate(zip(lens, new)) for p in range((n - m) // page, n // page)]
        at = torch.tensor(filled, dtype=torch.int64, device=dev).view(-1, 2)
        s["filled"] = table[at[:, 0], at[:, 1]].long()
        # all blocks that they are written to: sequence and number, and which are begun by them
        mine = [(b, i, i * BLOCK >= n - m) for b, (n, m) in enumerate(zip(lens, new))
                for i in range((n - m) // BLOCK, -(-n // BLOCK))]
        s["blocks"] = torch.tensor([(b, i) for b, i, _ in mine], dtype=torch.int64, device=dev)
        s["begun"] = torch.tensor([x for _, _, x in mine], device=dev)
    if op in ("attend", "weigh"):
        s["q"] = randn(B, Hq, D, scale=1.5)
        s["pages"] = None
        if case["topk"]:  # ascending lists of pages, the last one among them
            score = torch.rand(B, Hkv, max_pages, generator=g, device=dev)
            count = torch.tensor(need, device=dev)[:, None, None]
            j = torch.arange(max_pages, device=dev)
            score = torch.where(j < count, torch.where(j == count - 1, 2.0, score), -1.0)
            pick = torch.topk(score, case["topk"], dim=-1).indices
            pick = torch.sort(torch.where(pick < count, pick, max_pages), dim=-1).values
            idx = torch.where(pick < max_pages, pick, -1).to(torch.int32)
            s["pages"] = (idx, (idx >= 0).sum(-1).to(torch.int32))
    if op in ("weigh", "evict"):  # what the pages have received so far
        w = torch.rand(B, Hkv, max_pages, generator=g, device=dev).pow(4)
        s["weight"] = torch.where(slots[:, None], w, 0.0).contiguous()
        s["weight_out"] = torch.empty_like(s["weight"])
    if op == "evict":
        s["table_out"], s["lens_out"] = torch.empty_like(table), torch.empty_like(s["seq_lens"])
    if own:
        from bwd_tile_mean_gb300 import vsa
        s["cache"] = vsa.PagedCache(case["layout"], dtype, B, Hq, Hkv, D, page, num_pages, max_pages, k=k, v=v,
                                    k_mean=mean if mean is not None else False, page_table=table,
                                    seq_lens=s["seq_lens"], kv_dtype=E4M3 if eight else None, k_scale=ks, v_scale=vs,
                                    weigh=op == "weigh", allocate=False)
    return s


# -------------------------------------------------------------- plain forms

def _turned(x, cos, sin, interleaved):
    """x [..., D] in fp32 with its first dims rotated; cos, sin [..., R/2]."""
    h = cos.shape[-1]
    rot, rest = x[..., :2 * h], x[..., 2 * h:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :h], rot[..., h:])
    y1, y2 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, rest), -1)


def _rotate(s, x, back):
    angle = s["positions"].double()[:, s["axis"]] * s["freq"]  # far positions: 32 bits lose the angle
    cos, sin = angle.cos().float(), angle.sin().float()
    if back:
        sin = -sin
    if s["case"]["layout"] != "bhsd":
        cos, sin = cos[:, None], sin[:, None]
    return _turned(x.float(), cos, sin, s["case"]["interleaved"]).to(s["dtype"])


def _values(s, which, phys):
    """fp32 [pages, Hkv, page, D] of the pages `phys` of the k or v cache."""
    c = s["case"]
    x = s[which + "_cache"]
    x = (x.view(torch.uint8)[phys].view(E4M3) if c["kv"] == "e4m3" else x[phys]).float()
    x = x.transpose(-3, -2) if c["layout"] == "bshd" else x
    if c["kv"] == "e4m3":
        x = x * s[which + "_scale"][phys].repeat_interleave(BLOCK, -1)[..., None]
    return x


def _append(s):
    c, page = s["case"], s["case"]["page"]
    lens, table = s["seq_lens"].long(), s["page_table"].long()
    if s["cu_seqlens"] is None:
        seq = torch.arange(c["B"], device=lens.device)
        pos = lens - 1
    else:
        cu = s["cu_seqlens"].long()
        t = torch.arange(s["T"], device=lens.device)
        seq = (t[:, None] >= cu[None, 1:]).sum(1)
        pos = lens[seq] - (cu[seq + 1] - t)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        q, k = _turned(q, cos, sin, c["interleaved"]), _turned(k, cos, sin, c["interleaved"])
    # the blocks that take tokens, as one row each: what they hold, then the new tokens in their places
    b, i = s["blocks"].unbind(1)
    blocks_per = s["max_pages"] * page // BLOCK
    row = torch.full((c["B"] * blocks_per,), -1, dtype=torch.int64, device=lens.device)
    row[b * blocks_per + i] = torch.arange(len(b), device=lens.device)
    r, slot = row[seq * blocks_per + pos // BLOCK], pos % BLOCK
    phys, part = table[b, i * BLOCK // page], i % (page // BLOCK)
    place = part[:, None] * BLOCK + torch.arange(BLOCK, device=lens.device)
    bshd = c["layout"] == "bshd"
    for x, which in ((k, "k"), (v, "v")):
        cache = s[which + "_cache"].view(torch.uint8)
        cache = cache if bshd else cache.transpose(1, 2)  # [pages, page, Hkv, D]
        scale = s[which + "_scale"]
        old = torch.where(s["begun"][:, None], 0.0, scale[phys, :, part])  # [blocks, Hkv]
        top = torch.zeros(len(b), c["Hkv"], device=lens.device)
        top.index_reduce_(0, r, x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        new = torch.ldexp(torch.ones_like(top), torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126))
        new = torch.maximum(new, old)
        held = cache[phys[:, None], place].view(E4M3).float()  # [blocks, BLOCK, Hkv, D]
        held = torch.where(s["begun"][:, None, None, None], 0.0, held * (old / new)[:, None, :, None])
        held[r, slot] = x / new[r][..., None]
        # places behind the sequence's last token keep what they hold
        fresh = (i[:, None] * BLOCK + torch.arange(BLOCK, device=lens.device)) < lens[b][:, None]
        p2, s2 = phys[:, None].expand_as(place)[fresh], place[fresh]
        cache[p2, s2] = held[fresh].to(E4M3).view(torch.uint8)
        scale[phys, :, part] = new
    if len(s["filled"]):
        s["k_mean"][s["filled"]] = _values(s, "k", s["filled"]).mean(2)
    # the values of those blocks, in the order of their tokens
    n = s["cu_back"].long()
    t = torch.arange(s["T_back"], device=lens.device)
    seq = (t[:, None] >= n[None, 1:]).sum(1)
    pos = lens[seq] - (n[seq + 1] - t)
    phys, slot = table[seq, pos // page], pos % page
    got = []
    for which in ("k", "v"):
        cache = s[which + "_cache"].view(torch.uint8)
        cache = cache if bshd else cache.transpose(1, 2)
        got.append((cache[phys, slot].view(E4M3).float() * s[which + "_scale"][phys, :, slot // BLOCK][..., None])
                   .to(s["dtype"]))
    return q.to(s["dtype"]), *got


def _attend(s):
    c, page = s["case"], s["case"]["page"]
    B, Hq, Hkv, P, lens = c["B"], c["Hq"], c["Hkv"], s["max_pages"], s["seq_lens"].long()
    phys = s["page_table"].long()
    j = torch.arange(P, device=lens.device)
    ok = (j[:, None] * page + torch.arange(page, device=lens.device)) < lens[:, None, None]  # [B, P, page]
    ok = ok[:, None].expand(B, Hkv, P, page)
    if s["pages"] is not None:
        listed_ = torch.zeros(B, Hkv, P + 1, dtype=torch.bool, device=lens.device)
        idx = s["pages"][0].long()
        listed_.scatter_(2, torch.where(idx < 0, P, idx), True)
        ok = ok & listed_[..., :P, None]
    ok = ok.reshape(B, Hkv, 1, -1)
    k = _values(s, "k", phys).transpose(1, 2).reshape(B, Hkv, P * page, D)
    x = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    e = e / torch.where(total > 0, total, 1.0)
    v = torch.where(ok.transpose(2, 3), _values(s, "v", phys).transpose(1, 2).reshape(B, Hkv, P * page, D), 0.0)
    o = e @ v
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    got = dict(out=o.reshape(B, Hq, D).to(s["dtype"]), lse=lse.reshape(B, Hq))
    if c["op"] == "weigh":
        mass = e.view(B, Hkv, -1, P, page).sum((2, 4))
        live = j < -(-lens[:, None, None] // page)
        got["weight"] = torch.where(live, s["weight"] * c["decay"] + mass, s["weight"])
    return got


def _evict(s):
    c, page, P, keep = s["case"], s["case"]["page"], s["max_pages"], s["case"]["keep"]
    lens, table = s["seq_lens"].long(), s["page_table"]
    j = torch.arange(P, device=lens.device)[None]
    pages = -(-lens[:, None] // page)
    total = s["weight"].double().sum(1).float()
    held = (j < c["keep_first"]) | ((j >= pages - c["keep_last"]) & (j < pages))
    total = torch.where(held, math.inf, torch.where(j < pages, total, -math.inf))
    rank = torch.sort(torch.sort(total, dim=-1, descending=True, stable=True).indices, dim=-1).indices
    gone = (rank >= keep) & (j < pages)
    count = gone.sum(1)
    order = torch.sort(gone.to(torch.int8), dim=-1, stable=True).indices  # those that stay, then the others
    behind = j >= P - count[:, None]
    new_table = torch.where(behind, -1, table.gather(1, order))
    weight = s["weight"].gather(2, order[:, None].expand_as(s["weight"]))
    weight = torch.where(behind[:, None], 0.0, weight)
    freed = torch.full((c["B"], max(1, P - keep)), -1, dtype=torch.int32, device=lens.device)
    first = torch.sort((~gone).to(torch.int8), dim=-1, stable=True).indices[:, : freed.shape[1]]
    n = first.shape[1]
    freed[:, :n] = torch.where(j[:, :n] < count[:, None], table.gather(1, first), -1)
    return dict(table=new_table, lens=(lens - count * page).to(torch.int32), weight=weight, freed=freed,
                freed_cnt=count.to(torch.int32))


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if op in ("rotate", "back"):
        if own:
            call = s["rope"].backward if op == "back" else s["rope"].forward
            q, k = call(s["q"], s["k"], positions=s["positions"], layout=c["layout"])
            return dict(q=q, k=k)
        return dict(q=_rotate(s, s["q"], op == "back"), k=_rotate(s, s["k"], op == "back"))
    if op == "append":
        if own:
            cache = s["cache"]
            q = cache.append(s["k"], s["v"], s["q"], cu_seqlens=s["cu_seqlens"], cos=s["cos"], sin=s["sin"],
                             interleaved=c["interleaved"])
            k, v = cache.read(s["T_back"], cu_seqlens=s["cu_back"])
        else:
            q, k, v = _append(s)
        return dict(q=q, k=k, v=v, k_scale=s["k_scale"], v_scale=s["v_scale"], k_mean=s["k_mean"])
    if op == "evict":
        if not own:
            return _evict(s)
        freed, count = s["cache"].evict(s["weight"], c["keep"], keep_first=c["keep_first"], keep_last=c["keep_last"],
                                        out=(s["table_out"], s["lens_out"], s["weight_out"]))
        return dict(table=s["table_out"], lens=s["lens_out"], weight=s["weight_out"], freed=freed, freed_cnt=count)
    if not own:
        return _attend(s)
    if op == "attend":
        out, lse = s["cache"].attend(s["q"], s["pages"])
        return dict(out=out, lse=lse)
    out, lse = s["cache"].attend(s["q"], s["pages"], page_weight=s["weight"], weight_out=s["weight_out"],
                                 decay=c["decay"])
    return dict(out=out, lse=lse, weight=s["weight_out"])


# ------------------------------------------------------------------- exact

def _power(top):
    """The least 2^e >= 2^-126 with top <= 448 2^e, for numbers in 64 bits."""
    e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448)).clamp(-126, 127)
    e = torch.where(top > 448 * 2.0 ** e, e + 1, e)
    return 2.0 ** torch.where((top <= 224 * 2.0 ** e) & (e > -126), e - 1, e)


def exact(case, seed):
    """The definition in fp64, one sequence (or one head) at a time."""
    s = prepare(case, seed)
    B, Hq, Hkv, op = (case[k] for k in ("B", "Hq", "Hkv", "op"))
    if op in ("rotate", "back"):
        axis, freq = s["axis"].tolist(), s["freq"].tolist()
        h = len(axis)
        angle = torch.stack([s["positions"][:, a].double() * f for a, f in zip(axis, freq)], 1)
        turn = torch.polar(torch.ones_like(angle), -angle if op == "back" else angle)
        got = {}
        for name in ("q", "k"):
            x = s[name] if case["layout"] != "bhsd" else s[name].transpose(1, 2)
            y = x.double().contiguous()
            for n in range(x.shape[-2]):  # one head at a time, a pair as a complex number
                z = y[..., n, :2 * h]
                if case["interleaved"]:
                    z.copy_(torch.view_as_real(torch.view_as_complex(z.reshape(*z.shape[:-1], h, 2)) * turn).flatten(-2))
                else:
                    w = torch.complex(z[..., :h], z[..., h:]) * turn
                    z.copy_(torch.cat((w.real, w.imag), -1))
            got[name] = y if case["layout"] != "bhsd" else y.transpose(1, 2)
        return got
    if op == "evict":
        weight, page = s["weight"].double(), case["page"]
        for b, n in enumerate(_sizes(case)[0]):
            count = -(-n // page)
            total = weight[b, :, :count].sum(0).float().tolist()
            mine = sorted(range(case["keep_first"], count - case["keep_last"]), key=lambda j: (total[j], -j))
            stay = sorted(set(range(s["max_pages"])) - set(mine[: max(0, count - case["keep"])]))
            weight[b] = torch.nn.functional.pad(weight[b][:, stay], (0, s["max_pages"] - len(stay)))
        return dict(table=None, lens=None, weight=weight, freed=None, freed_cnt=None)
    page, topk, G, bshd = case["page"], case["topk"], Hq // Hkv, case["layout"] == "bshd"
    lens, new = _sizes(case)
    place = s["page_table"].tolist()

    def head(which, pages, h):
        """[tokens, D] of one key head over some pages."""
        x = s[which + "_cache"]
        x = x.view(torch.uint8) if case["kv"] == "e4m3" else x
        x = x[pages, :, h] if bshd else x[pages, h]
        if case["kv"] != "e4m3":
            return x.double().reshape(-1, D)
        x = x.view(E4M3).double().view(len(pages), -1, BLOCK, D)
        return (x * s[which + "_scale"][pages, h].double()[..., None, None]).reshape(-1, D)

    if op == "append":
        q, ks, vs = s["q"].double().clone(), s["k_scale"].double(), s["v_scale"].double()
        kn, vn, mean = s["k"].double(), s["v"].double(), s["k_mean"].double()
        n, t0, keys, values = case["rot"] // 2, 0, [], []
        for b in range(B):
            first = lens[b] - new[b]
            t = slice(t0, t0 + new[b])
            t0 += new[b]
            kb = kn[t].clone()
            if n:
                at = torch.arange(first, lens[b], device=q.device)
                turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
                pair = torch.arange(n, device=q.device)
                i1, i2 = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + n)
                x = q[t]
                z = torch.complex(x[..., i1], x[..., i2]) * turn
                x[..., i1], x[..., i2] = z.real, z.imag
                # which e4m3 value a key next to a border becomes is part of the definition, and so is the rounding of
                # its products and of their sum to 32 bits
                one = lambda y: y.float().double()  # noqa: E731
                a, b2, cos, sin = kb[..., i1].clone(), kb[..., i2].clone(), turn.real, turn.imag
                kb[..., i1] = one(one(a * cos) - one(b2 * sin))
                kb[..., i2] = one(one(b2 * cos) + one(a * sin))
            # from the first block's begin, or the first page's that fills up
            low = min(first // BLOCK * BLOCK, first // page * page if lens[b] // page > first // page else first)
            pages = torch.tensor(place[b][low // page: -(-lens[b] // page)], device=q.device)
            from_ = low // page * page
            skip = first // BLOCK * BLOCK - from_
            for x, which, scales, outs in ((kb, "k", ks, keys), (vn[t], "v", vs, values)):
                old = torch.stack([head(which, pages, h) for h in range(Hkv)], 1)[: lens[b] - from_]
                tops = torch.zeros(len(pages) * page, Hkv, dtype=torch.float64, device=q.device)
                tops[first - from_: lens[b] - from_] = x.abs().amax(-1)
                scale = _power(tops.view(-1, BLOCK, Hkv).amax(1))
                held = scales[pages].transpose(1, 2).reshape(-1, Hkv)
                i0, i1 = (first - from_) // BLOCK, -(-(lens[b] - from_) // BLOCK)
                if first % BLOCK:
                    scale[i0] = torch.maximum(scale[i0], held[i0])
                held = held.clone()
                held[i0:i1] = scale[i0:i1]
                scales[pages] = held.view(len(pages), -1, Hkv).transpose(1, 2)
                old[first - from_:] = x
                each = held.repeat_interleave(BLOCK, 0)[: len(old), :, None]
                stored = (old / each).float().to(E4M3).double() * each  # what the 8 bits stand for
                outs.append(stored[skip:])
                if which == "k":
                    for p in range(first // page, lens[b] // page):
                        mean[place[b][p]] = stored[p * page - from_: (p + 1) * page - from_].mean(0)
        return dict(q=q, k=torch.cat(keys), v=torch.cat(values), k_scale=ks, v_scale=vs, k_mean=mean)
    got = dict(out=torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda"),
               lse=torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda"))
    if op == "weigh":
        got["weight"] = s["weight"].double()
    for b in range(B):
        count = -(-lens[b] // page)
        if op == "weigh":
            got["weight"][b, :, :count] *= case["decay"]
        for h in range(Hkv):
            chosen = torch.arange(count, device="cuda")
            if topk:
                chosen = s["pages"][0][b, h, : int(s["pages"][1][b, h])].long()
            rows = s["page_table"][b, chosen].long()
            live = (chosen[:, None] * page + torch.arange(page, device="cuda")).flatten() < lens[b]
            z = s["q"][b, h * G:(h + 1) * G].double() @ head("k", rows, h).T * (D ** -0.5)
            z[:, ~live] = -math.inf
            p = torch.softmax(z, 1)
            got["lse"][b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            got["out"][b, h * G:(h + 1) * G] = p[:, live] @ head("v", rows, h)[live]
            if op == "weigh":
                got["weight"][b, h, chosen] += p.view(G, len(chosen), page).sum((0, 2))
    return got
