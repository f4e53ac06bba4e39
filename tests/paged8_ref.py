"""Plain references of the 8-bit paged cache, the page weights and the
eviction, on the CPU: bytes bit for bit, sums in fp64 with bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import paged_ref as ref
from tests.paged_ref import D, U

E4M3 = torch.float8_e4m3fn


def scale_of(top):
    """The least power of two >= 2^-126 that brings `top` within 448."""
    m, e = math.frexp(top)
    return 2.0 ** max(-126, e - 9 + (m > 0.875)) if top > 0 else 2.0 ** -126


def as_bytes(x, scale, dtype):
    """x fp32 (any shape) as e4m3 values of this scale, held in fp32."""
    x = x.float()
    fits = x.abs() < (math.inf if dtype == torch.bfloat16 else 65520.0)
    most = 240.0 if scale == (256.0 if dtype == torch.float16 else 2.0 ** 120) else 448.0
    y = (torch.where(fits, x, 0.0) / scale).clamp(-most, most).to(E4M3).float()  # a power of two: exact
    return torch.where(fits, y, math.nan)


class Pool8:
    """An 8-bit paged cache: e4m3 values (as fp32) [pages, page, Hkv, D] and
    scales [pages, Hkv, page / 16]."""

    def __init__(self, layout, dtype, Hq, Hkv, page, num_pages, max_pages, lens, seed=0, spread=0, garbage=False):
        g = torch.Generator().manual_seed(seed)
        self.layout, self.dtype, self.Hq, self.Hkv, self.page = layout, dtype, Hq, Hkv, page
        self.num_pages, self.max_pages, self.lens = num_pages, max_pages, list(lens)
        self.B = len(self.lens)
        shape, blocks = (num_pages, page, Hkv, D), (num_pages, Hkv, page // 16)
        self.k, self.v = ((torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(E4M3).float() for _ in range(2))
        self.ks, self.vs = (2.0 ** torch.randint(-7 - spread, -6 + spread, blocks, generator=g).float() for _ in range(2))
        self.mean = torch.randn((num_pages, Hkv, D), generator=g)
        need = [-(-n // page) for n in self.lens]
        assert sum(need) <= num_pages and max(need) <= max_pages
        order = torch.randperm(num_pages, generator=g).tolist()
        self.table = [[order.pop() if j < n else -7 for j in range(max_pages)] for n in need]
        if garbage:  # NaN bytes and scales wherever no token is
            live = torch.zeros(num_pages, page, dtype=torch.bool)
            for b, n in enumerate(self.lens):
                for j in range(need[b]):
                    live[self.table[b][j], : min(page, n - j * page)] = True
            for x in (self.k, self.v):
                x[~live] = math.nan
            dead = ~live.view(num_pages, -1, 16).any(2)
            for x in (self.ks, self.vs):
                x.transpose(1, 2)[dead] = math.nan

    def view(self, x):
        return (x if self.layout == "bshd" else x.transpose(1, 2)).contiguous().to(E4M3)

    def back(self, x):
        x = x.detach().cpu().float()
        return x if self.layout == "bshd" else x.transpose(1, 2)

    def cache(self, **kw):
        from bwd_tile_mean_gb300 import vsa
        i32 = dict(dtype=torch.int32, device="cuda")
        given = dict(k=self.view(self.k).cuda(), v=self.view(self.v).cuda(), k_scale=self.ks.cuda(), v_scale=self.vs.cuda(),
                     k_mean=self.mean.cuda(), page_table=torch.tensor(self.table, **i32),
                     seq_lens=torch.tensor(self.lens, **i32), kv_dtype=E4M3)
        given.update(kw)
        return vsa.PagedCache(self.layout, self.dtype, self.B, self.Hq, self.Hkv, D, self.page, self.num_pages,
                              self.max_pages, **given)

    def real(self, x, scale):
        """[pages, page, Hkv, D] in fp32: what the bytes stand for."""
        return x * scale.repeat_interleave(16, 2).transpose(1, 2)[..., None]


def append(pool, k, v, q, cu, cos=None, sin=None, positions=None, interleaved=False, means=True):
    """The call on the pool, bits and all; q_out with NaN rows where nothing is written."""
    q_out = torch.full_like(q, math.nan) if q is not None else None
    filled = set()
    for b in range(pool.B):
        n = cu[b + 1] - cu[b]
        new = {}  # page, block -> slots and their rows
        for i in range(n):
            pos, t = pool.lens[b] - n + i, cu[b] + i
            if not 0 <= pos < pool.max_pages * pool.page:
                continue
            kk, qq = k[t].float(), None if q is None else q[t]
            if cos is not None:
                r = min(max(pos if positions is None else int(positions[t]), 0), cos.shape[0] - 1)
                kk = torch.from_numpy(ref.rotate(k[t:t + 1], cos[r:r + 1], sin[r:r + 1], interleaved))[0]
                if q is not None:
                    qq = torch.from_numpy(ref.rotate(q[t:t + 1], cos[r:r + 1], sin[r:r + 1], interleaved))[0].to(pool.dtype)
            if q is not None:
                q_out[t] = qq
            p = pool.table[b][pos // pool.page]
            if 0 <= p < pool.num_pages:
                new.setdefault((p, pos % pool.page // 16), []).append((pos % pool.page, kk, v[t].float()))
                if pos % pool.page == pool.page - 1:
                    filled.add(p)
        for (p, blk), rows in new.items():
            first = min(s for s, _, _ in rows)
            for h in range(pool.Hkv):
                for what, (cache, scales) in enumerate(((pool.k, pool.ks), (pool.v, pool.vs))):
                    x = torch.stack([r[1 + what][h] for r in rows])
                    fits = x.abs() < (math.inf if pool.dtype == torch.bfloat16 else 65520.0)
                    scale = scale_of(float(torch.where(fits, x.abs(), 0.0).max()))
                    if first % 16:
                        old = float(scales[p, h, blk])
                        scale = max(scale, old)
                        if scale != old:
                            at = slice(blk * 16, first)
                            cache[p, at, h] = (cache[p, at, h] * (old / scale)).to(E4M3).float()
                    scales[p, h, blk] = scale
                    for (s, _, _), row in zip(rows, x):
                        cache[p, s, h] = as_bytes(row, scale, pool.dtype)
    if means:
        for p in filled:
            pool.mean[p] = ref.mean(pool.real(pool.k[p:p + 1], pool.ks[p:p + 1])[0])
    return q_out


def rows_of(pool, b, h, listed):
    """(keys, values, page of each, largest v scale) of some pages, in fp64."""
    ks, vs, at, top = [], [], [], 0.0
    eight = isinstance(pool, Pool8)
    for j in listed:
        if not 0 <= j < pool.max_pages or not 0 <= pool.table[b][j] < pool.num_pages:
            continue
        live = min(max(pool.lens[b] - j * pool.page, 0), pool.page)
        p = pool.table[b][j]
        k, v = pool.k[p, :live, h].double(), pool.v[p, :live, h].double()
        if eight and live:
            of = pool.vs[p, h].repeat_interleave(16)[:live, None].double()
            k, v = k * pool.ks[p, h].repeat_interleave(16)[:live, None].double(), v * of
            top = max(top, float(of.max()))
        ks.append(k)
        vs.append(v)
        at += [j] * live
    if not at:
        return None
    return torch.cat(ks), torch.cat(vs), at, top


def attend(pool, q, pages=None, scale=None, weight=None, decay=1.0):
    """(out, lse, bound on out, bound on lse[, weights, bound on them]) in fp64,
    for either cache; bounds derived below."""
    scale = scale or D ** -0.5
    G = pool.Hq // pool.Hkv
    eight = isinstance(pool, Pool8)
    u = 2.0 ** -11 if eight else U[pool.dtype]   # of a weight: fp16 for 8 bits
    out = torch.zeros((pool.B, pool.Hq, D), dtype=torch.float64)
    lse = torch.full((pool.B, pool.Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    mass = None if weight is None else weight.double().clone()
    wtol = None if weight is None else torch.zeros_like(mass)
    for b in range(pool.B):
        count = -(-pool.lens[b] // pool.page)
        if mass is not None:
            mass[b, :, :count] = mass[b, :, :count] * decay if decay else 0.0
            wtol[b, :, :count] = mass[b, :, :count].abs() * 2.0 ** -23
        for h in range(pool.Hkv):
            if pages is None:
                listed = range(count)
            else:
                listed = pages[0][b, h, :max(0, min(int(pages[1][b, h]), pages[0].shape[2]))].tolist()
            got = rows_of(pool, b, h, listed)
            if got is None:
                continue
            kk, vv, at, top = got
            qq = q[b, h * G:(h + 1) * G].double()
            s = qq @ kk.T * scale
            rows = slice(h * G, (h + 1) * G)
            lse[b, rows] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[b, rows] = p @ vv
            # A score is a sum of 128 products in fp32, scaled twice: off by at most 132 * 2^-24 of the products'
            # magnitudes (and 2^-22 of itself in log2 units), so a weight by e^(2 ds) - 1 with its sum; exp2 adds 2^-22,
            # the weight's rounding to 16 bits u, sums over n keys n * 2^-24 (tree-like: n / 16 steps of a warp), and
            # the output's own rounding U (fp16: 2^-25 absolute below its normal range). 8 bits: q in fp16 is off by
            # 2^-39 of its row's largest entry at most.
            mags = qq.abs() @ kk.abs().T
            if eight:
                mags = mags + 2.0 ** -15 * qq.abs().amax(1, keepdim=True) * kk.abs().sum(1)[None]
            ds = 132 * 2.0 ** -24 * scale * mags.amax(1) + 2.0 ** -22 * s.abs().amax(1)
            n = kk.shape[0]
            rel = u + 2 * ds + (8 + n / 16) * 2.0 ** -23
            tol[b, rows] = U[pool.dtype] * out[b, rows].abs() + rel[:, None] * (p @ vv.abs()) * 1.01
            first = torch.exp(s.amax(1) - torch.logsumexp(s, 1))  # 1 / sum of weights relative to the largest
            if pool.dtype == torch.float16:
                tol[b, rows] += 2.0 ** -25
            if eight:  # weights times a block's scale over the largest one, below 2^-24 lifted by 2^14
                tol[b, rows] += 2.0 ** -38 * first[:, None] * n * 448 * top
            elif pool.dtype == torch.float16:
                tol[b, rows] += 2.0 ** -40 * first[:, None] * vv.abs().sum(0)[None]
            ltol[b, rows] = ds + (8 + n / 16) * 2.0 ** -23 + 2.0 ** -23 * lse[b, rows].abs()
            if mass is not None:
                # each row's weight of a page: off by that of P and of the LSE (twice ds), the exponent's 2^-23 of the
                # scores' size, and sums over up to 256 keys and G rows
                one = torch.zeros(G, pool.max_pages, dtype=torch.float64)
                one.index_add_(1, torch.tensor(at), p)
                off = 3 * ds + 2.0 ** -22 * (s.abs().amax(1) + lse[b, rows].abs()) + (16 + n / 16 + G) * 2.0 ** -23
                mass[b, h] += one.sum(0)
                # and each time a page is listed its sum is added to its weight, rounding that by half a step
                times = torch.bincount(torch.tensor([j for j in listed if 0 <= j < pool.max_pages]), minlength=pool.max_pages)
                wtol[b, h] += (one * off[:, None]).sum(0) * 1.01 + G * 2.0 ** -100
                wtol[b, h] += mass[b, h].abs() * (2.0 ** -23 + times * 2.0 ** -24)
    if mass is None:
        return out, lse, tol, ltol
    return out, lse, tol, ltol, mass, wtol


def evict(table, lens, weight, page, keep, keep_first, keep_last):
    """(table, lens, weight, freed, freed_cnt) as lists and tensors."""
    B, P = len(table), len(table[0])
    cap = max(1, P - keep)
    table, lens, weight = [list(r) for r in table], list(lens), weight.clone()
    freed, cnt = torch.full((B, cap), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = -(-min(max(lens[b], 0), P * page) // page)
        if n <= keep:
            continue
        total = weight[b].double().sum(0).float().tolist()
        total = [-math.inf if math.isnan(x) else x for x in total]
        mine = list(range(keep_first, n - keep_last))
        stay = set(sorted(mine, key=lambda j: (-total[j], j))[: keep - keep_first - keep_last])
        gone = [j for j in mine if j not in stay]
        left = [j for j in range(P) if j not in set(gone)]
        freed[b, :len(gone)] = torch.tensor([table[b][j] for j in gone], dtype=torch.int32)
        cnt[b] = len(gone)
        table[b] = [table[b][j] for j in left] + [-1] * len(gone)
        weight[b] = torch.cat((weight[b][:, left], torch.zeros(weight.shape[1], len(gone))), 1)
        lens[b] = min(lens[b], P * page) - len(gone) * page
    return table, lens, weight, freed, cnt
