"""Plain references of the paged-cache calls: the definitions in fp64, and
the fp32 operation orders that make the stored bits and the selection
exact. CPU tensors throughout."""
from __future__ import annotations

import math

import numpy as np
import torch

D = 128
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step of a rounding, relative


class Pool:
    """A paged cache on the CPU: table and lengths as lists, pages in order
    [page, Hkv, D] whatever the layout of the device tensors."""

    def __init__(self, layout, dtype, Hq, Hkv, page, num_pages, max_pages, lens, seed=0, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.layout, self.dtype, self.Hq, self.Hkv, self.page = layout, dtype, Hq, Hkv, page
        self.num_pages, self.max_pages, self.lens = num_pages, max_pages, list(lens)
        self.B = len(self.lens)
        shape = (num_pages, page, Hkv, D)
        self.k = torch.randn(shape, generator=g).to(dtype)
        self.v = torch.randn(shape, generator=g).to(dtype)
        if fill is not None:  # what an unwritten slot holds
            self.k.fill_(fill)
            self.v.fill_(fill)
        self.mean = torch.randn((num_pages, Hkv, D), generator=g)
        need = [-(-n // page) for n in self.lens]
        assert sum(need) <= num_pages and max(need) <= max_pages
        order = torch.randperm(num_pages, generator=g).tolist()
        # entries past a sequence's end are not pages
        self.table = [[order.pop() if j < n else -7 for j in range(max_pages)] for n in need]
        self.gen = g

    def view(self, x):
        """Pages in the device's layout."""
        return (x if self.layout == "bshd" else x.transpose(1, 2)).contiguous()

    def back(self, x):
        x = x.detach().cpu()
        return x if self.layout == "bshd" else x.transpose(1, 2)

    def cache(self, **kw):
        from bwd_tile_mean_gb300 import vsa
        i32 = dict(dtype=torch.int32, device="cuda")
        given = dict(k=self.view(self.k).cuda(), v=self.view(self.v).cuda(), k_mean=self.mean.cuda(),
                     page_table=torch.tensor(self.table, **i32), seq_lens=torch.tensor(self.lens, **i32))
        given.update(kw)
        return vsa.PagedCache(self.layout, self.dtype, self.B, self.Hq, self.Hkv, D, self.page, self.num_pages,
                              self.max_pages, **given)


def rotate(x, cos, sin, interleaved, dtype=np.float32):
    """x [T, H, D] rotated in `dtype`, each product and sum rounded once
    (numpy does not contract)."""
    x = x.to(torch.float64).numpy().astype(dtype)
    c, s = (a.numpy().astype(dtype)[:, None] for a in (cos, sin))
    h = c.shape[-1]
    y = x.copy()
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def append(pool, k, v, q, cu, cos=None, sin=None, positions=None, interleaved=False, means=True):
    """The call on the pool, bits and all: returns q_out with NaN rows where
    nothing is written."""
    q_out = torch.full_like(q, math.nan) if q is not None else None
    for b in range(pool.B):
        n = cu[b + 1] - cu[b]
        touched = set()
        for i in range(n):
            pos, t = pool.lens[b] - n + i, cu[b] + i
            if not 0 <= pos < pool.max_pages * pool.page:
                continue
            kk, qq = k[t:t + 1], None if q is None else q[t:t + 1]
            if cos is not None:
                r = min(max(pos if positions is None else int(positions[t]), 0), cos.shape[0] - 1)
                turn = lambda x: torch.from_numpy(  # noqa: E731
                    rotate(x, cos[r:r + 1], sin[r:r + 1], interleaved)).to(pool.dtype)
                kk = turn(kk)
                qq = None if q is None else turn(qq)
            if q is not None:
                q_out[t] = qq[0]
            p = pool.table[b][pos // pool.page]
            if not 0 <= p < pool.num_pages:
                continue
            pool.k[p, pos % pool.page] = kk[0]
            pool.v[p, pos % pool.page] = v[t]
            if pos % pool.page == pool.page - 1:
                touched.add(p)
        if means:
            for p in touched:
                pool.mean[p] = mean(pool.k[p])
    return q_out


def mean(keys):
    """Mean of a page's stored keys [page, Hkv, D] in the call's fp32 order."""
    x = keys.float().numpy()
    total = None
    for g in range(0, x.shape[0], 16):
        even, odd = np.zeros_like(x[0]), np.zeros_like(x[0])
        for s in range(g, g + 16, 2):
            even, odd = even + x[s], odd + x[s + 1]
        part = even + odd
        total = part if total is None else total + part
    return torch.from_numpy(total / np.float32(x.shape[0]))


def scores(pool, q, b, h):
    """fp32 scores of the full pages of sequence b for key head h."""
    G = pool.Hq // pool.Hkv
    g = q[b, h * G:(h + 1) * G].double().sum(0).float().numpy()
    out = []
    for j in range(pool.lens[b] // pool.page):
        p = pool.table[b][j]
        if not 0 <= p < pool.num_pages:
            out.append(-math.inf)
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            x = g * pool.mean[p, h].numpy()
            x = x[:64] + x[64:]
            x = x[:32] + x[32:]
            while x.size > 1:
                x = x[0::2] + x[1::2]
        out.append(-math.inf if math.isnan(x[0]) else float(x[0]))
    return out


def select(pool, q, topk, keep_first, keep_last):
    """(page_idx [B, Hkv, topk], page_cnt [B, Hkv])."""
    idx = torch.full((pool.B, pool.Hkv, topk), -1, dtype=torch.int32)
    cnt = torch.zeros((pool.B, pool.Hkv), dtype=torch.int32)
    for b in range(pool.B):
        n = -(-pool.lens[b] // pool.page)
        full = pool.lens[b] // pool.page
        for h in range(pool.Hkv):
            r = scores(pool, q, b, h)
            rank = []
            for j in range(n):
                kept = j < keep_first or j >= n - keep_last or j >= full
                rank.append((0 if kept else 1, 0.0 if kept else -r[j], j))
            chosen = sorted(j for _, _, j in sorted(rank)[:topk])
            idx[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            cnt[b, h] = len(chosen)
    return idx, cnt


def attend(pool, q, pages=None, scale=None):
    """(out, lse, bound on out, bound on lse) in fp64; bounds derived below."""
    scale = scale or D ** -0.5
    G = pool.Hq // pool.Hkv
    u = U[pool.dtype]
    out = torch.zeros((pool.B, pool.Hq, D), dtype=torch.float64)
    lse = torch.full((pool.B, pool.Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(pool.B):
        for h in range(pool.Hkv):
            if pages is None:
                listed = range(-(-pool.lens[b] // pool.page))
            else:
                listed = pages[0][b, h, :max(0, min(int(pages[1][b, h]), pages[0].shape[2]))].tolist()
            ks, vs = [], []
            for j in listed:
                if not 0 <= j < pool.max_pages or not 0 <= pool.table[b][j] < pool.num_pages:
                    continue
                live = min(max(pool.lens[b] - j * pool.page, 0), pool.page)
                ks.append(pool.k[pool.table[b][j], :live, h])
                vs.append(pool.v[pool.table[b][j], :live, h])
            if not ks or sum(len(x) for x in ks) == 0:
                continue
            kk, vv = torch.cat(ks).double(), torch.cat(vs).double()
            qq = q[b, h * G:(h + 1) * G].double()
            s = qq @ kk.T * scale
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            rows = slice(h * G, (h + 1) * G)
            out[b, rows] = p @ vv
            # A score is a sum of 128 products in fp32, scaled twice: off by at most
            # 132 * 2^-24 of the products' magnitudes (and 2^-22 of itself in log2 units), so a
            # weight by e^(2 ds) - 1 with its sum; exp2 adds 2^-22, the weight's rounding to
            # 16 bits u (fp16, lifted by 2^15: 2^-40 absolute below its normal range), sums over
            # n keys n * 2^-24 (tree-like: n / 16 steps of a warp), and the output's own rounding
            # u (fp16: 2^-25 absolute below its normal range).
            ds = 132 * 2.0 ** -24 * scale * (qq.abs() @ kk.abs().T).amax(1) + 2.0 ** -22 * s.abs().amax(1)
            rel = u + 2 * ds + (8 + kk.shape[0] / 16) * 2.0 ** -23
            mag = p @ vv.abs()
            tol[b, rows] = u * out[b, rows].abs() + rel[:, None] * mag * 1.01
            if pool.dtype == torch.float16:
                top = torch.exp(s.amax(1) - torch.logsumexp(s, 1))  # 1 / sum of weights relative to the largest
                tol[b, rows] += 2.0 ** -40 * top[:, None] * vv.abs().sum(0)[None] + 2.0 ** -25
            ltol[b, rows] = ds + (8 + kk.shape[0] / 16) * 2.0 ** -23 + 2.0 ** -23 * lse[b, rows].abs()
    return out, lse, tol, ltol


def check_attend(got, want, tag=""):
    out, lse, tol, ltol = want
    o, l = got[0].double().cpu(), got[1].double().cpu()
    assert torch.equal(torch.isnan(o), torch.isnan(out)), f"{tag}: NaN rows"
    d = (o - out).abs()
    fine = ~torch.isnan(out)
    assert (d[fine] <= tol[fine]).all(), f"{tag}: out off by {float((d - tol)[fine].max()):.3e} over its bound"
    empty = lse == -math.inf
    assert (l[empty] == -math.inf).all() and (o[empty] == 0).all(), f"{tag}: rows without keys"
    rest = ~empty & ~torch.isnan(lse)
    assert ((l - lse).abs()[rest] <= ltol[rest]).all(), f"{tag}: lse"
