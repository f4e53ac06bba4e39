"""Measured cases of the paged-cache operators: appending rotated keys and
values to a paged cache, choosing pages by their mean key, and the attention
of one new token per sequence over the cache (all pages, or the chosen ones).

``own = False`` runs each operator's plain form (elementary torch operations
in fp32), ``own = True`` the framework's calls (``vsa.PagedCache``).
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases

def _case(name, op, B, Hq, Hkv, page, layout, dtype, lo, hi, new_lo=1, new_hi=1, rot=D, interleaved=False, topk=0,
          keep_first=0, keep_last=1):
    c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, page=page, layout=layout, dtype=dtype, lo=lo, hi=hi, new_lo=new_lo,
             new_hi=new_hi, rot=rot, interleaved=interleaved, topk=topk, keep_first=keep_first, keep_last=keep_last)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence's next token: the launch itself is the cost
        _case("append-one-token", "append", 1, 12, 3, 128, "bshd", "fp16", 400, 400),
        # next tokens of a serving batch, contexts of all lengths
        _case("append-batch-tokens", "append", 64, 32, 8, 64, "bhsd", "bf16", 100, 8000),
        # ragged prompts (the lengths of the varlen workload), rotation of half the head
        _case("append-ragged-prompts", "append", 13, 12, 3, 128, "bshd", "fp16", 400, 900, 7, 360, rot=64,
              interleaved=True),
        # a long video context of 24 heads written at once, 256-token tiles
        _case("append-long-prompt", "append", 2, 24, 24, 256, "bshd", "bf16", 14000, 16000, 14000, 16000),
        # 1,024 tiles of one long video, 24 heads, 5% of the tiles
        _case("select-long-video", "select", 1, 24, 24, 256, "bhsd", "bf16", 245760, 245760, topk=24),
        # a batch of long contexts in small pages, grouped heads, with first and last pages kept
        _case("select-batch", "select", 32, 32, 8, 64, "bshd", "bf16", 20000, 131000, topk=64, keep_first=1,
              keep_last=4),
        # a short context of one sequence: latency
        _case("attend-short", "attend", 1, 12, 3, 128, "bshd", "fp16", 101, 101),
        # one long video context, every head with its own keys (480 tiles of 256)
        _case("attend-long-video", "attend", 1, 24, 24, 256, "bhsd", "bf16", 122880, 122880),
        # a serving batch of ragged contexts, grouped heads: the ordinary decode step
        _case("attend-batch", "attend", 64, 32, 8, 64, "bshd", "bf16", 37, 16000),
        # wide groups (16 query heads on one key head), small pages
        _case("attend-wide-groups", "attend", 16, 32, 2, 16, "bhsd", "fp16", 1000, 9000),
        # the sparse decode step over the long video: choose 24 tiles of 480, attend to them
        _case("sparse-long-video", "sparse", 1, 24, 24, 256, "bshd", "bf16", 122880, 122880, topk=24),
        # a whole decode step of a batch: append the token, choose pages, attend to them
        _case("step-batch", "step", 32, 32, 8, 64, "bshd", "bf16", 5000, 60000, topk=64, keep_first=1, keep_last=2),
    ]


def draw(rng):
    """A case of the same ranges: one token to long prompts, contexts of 1
    to 131,072 tokens, groups of 1 to 16 heads, every page size."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "select", "attend", "sparse", "step"))
    Hkv = rng.choice((1, 2, 3, 4, 8, 12, 24))
    G = rng.choice((1, 2, 3, 4, 5, 8, 16)) if Hkv <= 8 else rng.choice((1, 2))
    page = rng.choice((16, 32, 64, 128, 256))
    B = log_int(1, 96)
    common = dict(layout=rng.choice(("bshd", "bhsd")), dtype=rng.choice(("bf16", "fp16")))
    rot = rng.choice((0, 32, 64, 96, 128, 128))
    style = rng.random() < 0.5
    if op == "append":
        n = log_int(1, max(2, min(4096, 600000 // (B * Hkv * (G + 2)))))
        hi = n + log_int(1, 4096)
        return _case(None, op, B, G * Hkv, Hkv, page, lo=n, hi=hi, new_lo=max(1, n // rng.choice((1, 2, 8))), new_hi=n,
                     rot=rot, interleaved=style, **common)
    budget = 2500000 if op == "attend" else 6000000  # keys x key heads over the batch
    hi = log_int(1, max(2, min(131072, budget // (B * Hkv))))
    lo = max(1, hi // rng.choice((1, 2, 16, 256)))
    topk = max(3, min(128, log_int(3, 1 + max(3, hi // page))))
    if op == "select":  # something to choose: more pages than are asked for
        hi = page * log_int(24, max(25, min(8192, budget // (B * Hkv * page))))
        lo, topk = max(1, hi // rng.choice((1, 2, 16, 256))), log_int(8, max(9, min(128, hi // page // 2)))
    keep_first, keep_last = (rng.choice((0, 1)), rng.choice((1, 2))) if op != "attend" else (0, 1)
    return _case(None, op, B, G * Hkv, Hkv, page, lo=lo, hi=hi, rot=rot, interleaved=style,
                 topk=0 if op == "attend" else topk, keep_first=keep_first, keep_last=keep_last, **common)


def _sizes(case):
    """(lengths, new tokens) per sequence: spread over [lo, hi] evenly in
    their logarithm, in an order of the case's own, the longest among them."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))

    def spread(lo, hi):
        n = [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(case["B"])]
        n[r.randrange(len(n))] = hi
        return n

    lens = spread(case["lo"], case["hi"])
    if case["op"] not in ("append", "step"):
        return lens, [0] * len(lens)
    new = spread(case["new_lo"], case["new_hi"])
    return [max(a, b) for a, b in zip(lens, new)], new


def work(case):
    B, Hq, Hkv, page, op = (case[k] for k in ("B", "Hq", "Hkv", "page", "op"))
    lens, new = _sizes(case)
    T, rows = sum(new), 256  # bytes of one head of one token
    total, flops = 0, 0
    if op in ("append", "step"):
        total += 2 * T * (2 * Hkv + Hq) * rows + T * case["rot"] * 4
        flops += T * (Hq + Hkv) * case["rot"] * 3
        for n, m in zip(lens, new):  # means of the pages that fill up: their earlier keys, and the mean
            done = n // page - (n - m) // page
            total += Hkv * (done * 512 + ((n - m) % page * rows if done else 0))
    if op in ("select", "sparse", "step"):
        full = sum(n // page for n in lens)
        total += full * Hkv * 512 + B * Hq * rows + B * Hkv * case["topk"] * 4
        flops += full * Hkv * 2 * D
    if op in ("attend", "sparse", "step"):
        keys = [n if op == "attend" else min(n, case["topk"] * page) for n in lens]
        total += sum(keys) * Hkv * 2 * rows + B * Hq * (2 * rows + 4)
        flops += sum(keys) * Hq * 4 * D
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    B, Hq, Hkv, page, op = (case[k] for k in ("B", "Hq", "Hkv", "page", "op"))
    dtype, dev = DTYPES[case["dtype"]], torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _sizes(case)
    need = [-(-n // page) for n in lens]
    max_pages, num_pages = max(need), sum(need) + 3

    def randn(*shape, scale=1.0, kind=dtype):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(kind)

    s = dict(case=case, dtype=dtype, max_pages=max_pages, num_pages=num_pages)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # pages of the pool in random order, as after many requests came and went
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=dev)
    slots = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table[slots] = order[: sum(need)]
    s["page_table"] = table
    shape = (num_pages, page, Hkv, D) if case["layout"] == "bshd" else (num_pages, Hkv, page, D)
    if op == "select":  # reads no cache
        k = v = None
        s["k_mean"] = randn(num_pages, Hkv, D, scale=0.5, kind=torch.float32)
    else:
        # keys share a direction within their page, so that the pages' scores differ
        k = torch.empty(shape, dtype=dtype, device=dev)
        v = torch.empty(shape, dtype=dtype, device=dev)
        centre = randn(num_pages, Hkv, D, scale=0.5, kind=torch.float32)
        for at in range(0, num_pages, 256):
            to = min(num_pages, at + 256)
            c = centre[at:to, None] if case["layout"] == "bshd" else centre[at:to, :, None]
            k[at:to] = (randn(to - at, *shape[1:], kind=torch.float32) + c).to(dtype)
            v[at:to] = randn(to - at, *shape[1:])
        s["k_mean"] = torch.empty(num_pages, Hkv, D, device=dev)
        for at in range(0, num_pages, 256):
            s["k_mean"][at:at + 256] = k[at:at + 256].float().mean(1 if case["layout"] == "bshd" else 2)
    s["k_cache"], s["v_cache"] = k, v
    if op in ("append", "step"):
        T, rot = sum(new), case["rot"]
        # the three parts of one projection's output, as a model hands them over
        qkv = randn(T, Hq + 2 * Hkv, D, scale=1.0)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        start = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        s["cu_seqlens"] = None if new == [1] * B else start
        s["cos"] = s["sin"] = None
        if rot:
            freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
            angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * freq[None]
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["T"] = T
        # pages that these tokens fill up
        filled = [(b, p) for b, (n, m) in enumerate(zip(lens, new)) for p in range((n - m) // page, n // page)]
        at = torch.tensor(filled, dtype=torch.int64, device=dev).view(-1, 2)
        s["filled"] = table[at[:, 0], at[:, 1]].long()
    else:
        s["q"] = randn(B, Hq, D, scale=1.5)
    if own:
        from bwd_tile_mean_gb300 import vsa
        s["cache"] = vsa.PagedCache(case["layout"], dtype, B, Hq, Hkv, D, page, num_pages, max_pages, k=k, v=v,
                                    k_mean=s["k_mean"], page_table=table, seq_lens=s["seq_lens"],
                                    allocate=False)
    return s


# -------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] in fp32 with its first dims rotated; cos, sin [T, 1, R/2]."""
    h = cos.shape[-1]
    rot, rest = x[..., :2 * h], x[..., 2 * h:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :h], rot[..., h:])
    y1, y2 = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, rest), -1)


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
    q, k = s["q"].float(), s["k"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        q, k = _rotate(q, cos, sin, c["interleaved"]), _rotate(k, cos, sin, c["interleaved"])
    phys, slot = table[seq, pos // page], pos % page
    bshd = c["layout"] == "bshd"
    kc = s["k_cache"] if bshd else s["k_cache"].transpose(1, 2)
    vc = s["v_cache"] if bshd else s["v_cache"].transpose(1, 2)
    kc[phys, slot] = k.to(s["dtype"])
    vc[phys, slot] = s["v"]
    s["k_mean"][s["filled"]] = kc[s["filled"]].float().mean(1)
    return q.to(s["dtype"])


def _select(s, q):
    c, page, P = s["case"], s["case"]["page"], s["max_pages"]
    B, Hkv, lens = c["B"], c["Hkv"], s["seq_lens"].long()
    j = torch.arange(P, device=lens.device)
    gq = q.double().view(B, Hkv, -1, D).sum(2).float()
    x = s["k_mean"][s["page_table"].long()].transpose(1, 2) * gq[:, :, None]  # [B, Hkv, P, D]
    x = x[..., :64] + x[..., 64:]
    x = x[..., :32] + x[..., 32:]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0::2] + x[..., 1::2]
    x = x[..., 0] + x[..., 1]
    pages = -(-lens // page)
    kept = (j[None] < c["keep_first"]) | (j[None] >= pages[:, None] - c["keep_last"]) | (j[None] >= lens[:, None] // page)
    x = torch.where(kept[:, None], math.inf, x)
    x = torch.where((j[None] < pages[:, None])[:, None], x, -math.inf)
    # kept pages first, then by score, the lower index first among equals
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., : c["topk"]]
    order = torch.where(order < pages[:, None, None], order, P)
    order = torch.sort(order, dim=-1).values
    idx = torch.full((B, Hkv, c["topk"]), -1, dtype=torch.int32, device=lens.device)
    idx[..., : order.shape[-1]] = torch.where(order < P, order, -1).to(torch.int32)
    cnt = pages.clamp(max=c["topk"])[:, None].expand(B, Hkv).to(torch.int32)
    return idx, cnt


def _attend(s, q, idx):
    c, page = s["case"], s["case"]["page"]
    B, Hq, Hkv, lens = c["B"], c["Hq"], c["Hkv"], s["seq_lens"].long()
    if idx is None:
        idx = torch.arange(s["max_pages"], device=lens.device)[None, None].expand(B, Hkv, -1)
    idx = idx.long()
    phys = s["page_table"].long()[:, None].expand(B, Hkv, -1).gather(2, idx.clamp(min=0))
    head = torch.arange(Hkv, device=lens.device)[None, :, None]
    bshd = c["layout"] == "bshd"
    kc = s["k_cache"].transpose(1, 2) if bshd else s["k_cache"]
    vc = s["v_cache"].transpose(1, 2) if bshd else s["v_cache"]
    k = kc[phys, head].float().view(B, Hkv, -1, D)
    pos = idx[..., None] * page + torch.arange(page, device=lens.device)
    ok = ((idx[..., None] >= 0) & (pos < lens[:, None, None, None])).view(B, Hkv, 1, -1)
    x = (q.float().view(B, Hkv, -1, D) @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(ok.transpose(2, 3), vc[phys, head].float().view(B, Hkv, -1, D), 0.0)
    o = (e @ v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return o.reshape(B, Hq, D).to(s["dtype"]), lse.reshape(B, Hq)


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    got = {}
    if own:
        cache = s["cache"]
        q = s["q"]
        if op in ("append", "step"):
            q = cache.append(s["k"], s["v"], q, cu_seqlens=s["cu_seqlens"], cos=s["cos"], sin=s["sin"],
                             interleaved=c["interleaved"])
            got.update(q=q, k_cache=cache.k, v_cache=cache.v, k_mean=cache.k_mean)
        pages = None
        if op in ("select", "sparse", "step"):
            pages = cache.select(q, c["topk"], keep_first=c["keep_first"], keep_last=c["keep_last"])
            got.update(page_idx=pages[0], page_cnt=pages[1])
        if op in ("attend", "sparse", "step"):
            got["out"], got["lse"] = cache.attend(q, pages)
        return got
    q, idx = s["q"], None
    if op in ("append", "step"):
        q = _append(s)
        got.update(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], k_mean=s["k_mean"])
    if op in ("select", "sparse", "step"):
        idx, cnt = _select(s, q)
        got.update(page_idx=idx, page_cnt=cnt)
    if op in ("attend", "sparse", "step"):
        got["out"], got["lse"] = _attend(s, q, idx)
    return got


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The definition in fp64, one sequence at a time."""
    s = prepare(case, seed)
    B, Hq, Hkv, page, op, topk = (case[k] for k in ("B", "Hq", "Hkv", "page", "op", "topk"))
    G, bshd, dtype = Hq // Hkv, case["layout"] == "bshd", s["dtype"]
    lens, new = _sizes(case)
    table = s["page_table"].long()
    place = table.tolist()
    q = s["q"].double()
    k_mean = s["k_mean"].double()
    kc, vc = s["k_cache"], s["v_cache"]
    got = {}
    if op in ("append", "step"):
        q, kc, vc = q.clone(), kc.double(), vc.double()
        kn, t0, h = s["k"].double(), 0, case["rot"] // 2
        for b in range(B):
            at = torch.arange(lens[b] - new[b], lens[b], device=q.device)
            t = slice(t0, t0 + new[b])
            t0 += new[b]
            kb = kn[t]
            if h:
                # the pair of a head as a complex number, turned by its angle
                turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
                at_pair = torch.arange(h, device=q.device)
                i1, i2 = (2 * at_pair, 2 * at_pair + 1) if case["interleaved"] else (at_pair, at_pair + h)
                for x in (q[t], kb):
                    z = torch.complex(x[..., i1], x[..., i2]) * turn
                    x[..., i1], x[..., i2] = z.real, z.imag
            for p in range((lens[b] - new[b]) // page, -(-lens[b] // page)):
                mine = at // page == p
                kp, vp = (c[place[b][p]] if bshd else c[place[b][p]].transpose(0, 1) for c in (kc, vc))
                kp[at[mine] % page] = kb[mine]
                vp[at[mine] % page] = s["v"][t][mine].double()
                if (p + 1) * page <= lens[b]:
                    stored = kp.clone()
                    stored[at[mine] % page] = kb[mine].to(dtype).double()  # the mean is of the keys as stored
                    k_mean[place[b][p]] = stored.mean(0)
        got.update(q=q, k_cache=kc, v_cache=vc, k_mean=k_mean)
        if op == "append":
            return got
        q = q.to(dtype).double()  # what the later parts of the step are given
    if op in ("select", "sparse", "step"):
        got.update(page_idx=None, page_cnt=None)
    if op == "select":
        return None
    got["out"] = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    got["lse"] = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n, count = lens[b], -(-lens[b] // page)
        for h in range(Hkv):
            mine = q[b, h * G:(h + 1) * G]
            if op == "attend" or count <= topk:
                chosen = torch.arange(count, device=q.device)
            else:
                score = k_mean[table[b, :count], h] @ mine.sum(0)
                score[: case["keep_first"]] = math.inf
                score[count - case["keep_last"]:] = math.inf
                score[n // page:] = math.inf
                chosen = torch.sort(torch.sort(score, descending=True, stable=True).indices[:topk]).values
            rows = table[b, chosen]
            kk = (kc[rows, :, h] if bshd else kc[rows, h]).reshape(-1, D)
            vv = (vc[rows, :, h] if bshd else vc[rows, h]).reshape(-1, D)
            live = (chosen[:, None] * page + torch.arange(page, device=q.device)).flatten() < n
            kk, vv = kk[live].to(dtype).double(), vv[live].double()
            z = mine @ kk.T * (D ** -0.5)
            got["lse"][b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            got["out"][b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ vv
    return got
