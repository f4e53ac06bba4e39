"""The 8-bit paged cache, the page weights of both caches and the eviction
against plain references: bytes and tables bit for bit, sums in fp64 with
bounds from the roundings."""
import itertools
import math

import pytest
import torch

from bwd_tile_mean_gb300 import vsa
from tests import paged8_ref as ref8
from tests import paged_ref as ref
from tests.paged8_ref import D, E4M3, Pool8
from tests.paged_ref import Pool
from tests.test_gpu_paged import BF, HF, angles, new_tokens, same

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def equal_bytes(pool, cache):
    for name, mine, got in (("keys", pool.k, cache.k), ("values", pool.v, cache.v)):
        got = pool.back(got)
        assert torch.equal(torch.isnan(got), torch.isnan(mine)), name + ": NaN"
        assert torch.equal(torch.nan_to_num(got, 0.0), torch.nan_to_num(mine, 0.0)), name
    for name, mine, got in (("k_scale", pool.ks, cache.k_scale), ("v_scale", pool.vs, cache.v_scale)):
        assert same(got, mine), name


# ------------------------------------------------------------------ append

APPEND = [  # layout, dtype, Hq, Hkv, page, rot, interleaved, lengths, new tokens
    ("bshd", BF, 4, 2, 16, 128, False, [1], [1]),
    ("bhsd", HF, 3, 3, 32, 64, True, [40, 31, 64], [40, 31, 64]),
    ("bshd", HF, 12, 3, 128, 96, False, [300, 128, 0, 129, 127], [300, 1, 0, 129, 60]),
    ("bhsd", BF, 8, 8, 256, 128, True, [700, 256, 5], [500, 256, 0]),
    ("bshd", BF, 5, 1, 64, 16, False, [64, 1, 200, 63, 65], [64, 1, 137, 63, 2]),
    ("bhsd", BF, 24, 24, 64, 0, False, [70, 130], [33, 130]),
    ("bshd", HF, 40, 2, 16, 128, True, [17] * 40, [1] * 40),
    ("bhsd", BF, 10, 5, 32, 32, False, [96, 97, 33], [32, 96, 2]),
    ("bshd", BF, 24, 12, 64, 96, True, [1500, 900, 450], [1450, 900, 400]),   # many rows: several key heads per warp
    ("bhsd", HF, 11, 11, 256, 128, False, [1100, 800], [1100, 777]),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-r{c[5]}-{'i' if c[6] else 'h'}")
@pytest.mark.parametrize("rows", ["own-rows", "given-rows", "short-table"])
def test_append(case, rows):
    layout, dtype, Hq, Hkv, page, rot, inter, lens, new = case
    need = sum(-(-n // page) for n in lens)
    pool = Pool8(layout, dtype, Hq, Hkv, page, need + 2, max(-(-n // page) for n in lens) + 1, lens, seed=len(lens))
    T = sum(new) + 3  # tokens behind the last sequence
    qkv, q, k, v = new_tokens(pool, T)
    qkv[:, Hq:] *= torch.exp2(torch.randint(-6, 7, (T, 1, 1)).to(dtype))  # some blocks' scales grow, some stay
    cu = [0] + list(itertools.accumulate(new))
    # a table that ends before the last positions: those take its last row
    cos, sin = angles(max(lens) + 1 if rows != "short-table" else max(1, max(lens) // 2), rot) if rot else (None, None)
    pos = torch.randint(-2, max(lens) + 4, (T,), dtype=torch.int32) if rows == "given-rows" else None
    cache = pool.cache()
    q_out = torch.full((T, Hq, D), math.nan, dtype=dtype, device="cuda")
    gpu = qkv.cuda()
    parts = gpu[:, Hq:Hq + Hkv], gpu[:, Hq + Hkv:], gpu[:, :Hq]
    cud = lambda x: None if x is None else x.cuda()  # noqa: E731
    kw = dict(cu_seqlens=i32(cu), cos=cud(cos), sin=cud(sin), positions=cud(pos), interleaved=inter, q_out=q_out)
    assert cache.append(*parts, **kw) is q_out
    want = ref8.append(pool, k, v, q, cu, cos, sin, pos, inter)
    equal_bytes(pool, cache)
    assert same(cache.k_mean, pool.mean), "means"
    assert torch.equal(torch.isnan(q_out).cpu(), torch.isnan(want)), "q rows written"
    fine = ~torch.isnan(want)
    assert torch.equal(q_out.cpu()[fine], want[fine]), "queries"
    before = [x.clone() for x in (cache.k.view(torch.uint8).int(), cache.v.view(torch.uint8).int(), cache.k_scale,
                                  cache.v_scale, cache.k_mean, q_out)]
    cache.append(*parts, **kw)  # the same call again changes nothing
    after = (cache.k.view(torch.uint8).int(), cache.v.view(torch.uint8).int(), cache.k_scale, cache.v_scale, cache.k_mean,
             q_out)
    assert all(same(a, b) for a, b in zip(before, after))


@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_in_pieces(page):
    """Scales do not depend on how the tokens are cut into calls; bytes only
    below 2^-6 of the scale; the pieces match the reference bit for bit."""
    final = [2 * page + 5, 3 * page]
    one, many = (Pool8("bshd", BF, 6, 3, page, 8, 4, final, seed=9) for _ in range(2))
    _, q, k, v = new_tokens(one, sum(final), seed=10)
    k *= torch.exp2(torch.randint(-3, 4, (k.shape[0], 1, 1)).to(BF))
    whole, pieces = one.cache(), many.cache()
    cu = [0, final[0], sum(final)]
    cos, sin = angles(max(final), 128)
    whole.append(k.cuda(), v.cuda(), cu_seqlens=i32(cu), cos=cos.cuda(), sin=sin.cuda())
    done = [0, 0]
    for step in (1, page - 2, 1, 7, page, 10 * page):
        n = [min(step, f - d) for f, d in zip(final, done)]
        rows = torch.cat([torch.arange(cu[b] + done[b], cu[b] + done[b] + n[b]) for b in range(2)])
        done = [d + m for d, m in zip(done, n)]
        if not len(rows):
            continue
        many.lens = list(done)
        pieces.seq_lens.copy_(i32(done))
        pieces.append(k[rows].cuda(), v[rows].cuda(), cu_seqlens=i32([0, n[0], sum(n)]), cos=cos.cuda(), sin=sin.cuda())
        ref8.append(many, k[rows], v[rows], None, [0, n[0], sum(n)], cos, sin)
        equal_bytes(many, pieces)
        assert same(pieces.k_mean, many.mean)
    assert done == final
    assert same(pieces.k_scale, whole.k_scale) and same(pieces.v_scale, whole.v_scale)
    for a, b in ((pieces.k, whole.k), (pieces.v, whole.v)):
        a, b = a.float(), b.float()
        assert ((a == b) | ((a - b).abs() <= 2.0 ** -9) & (b.abs() < 2.0 ** -6)).all()


@pytest.mark.parametrize("B,Hq,Hkv,page", [(300, 8, 2, 16), (70, 20, 5, 64), (5, 40, 40, 256)])
def test_next_tokens_of_a_batch(B, Hq, Hkv, page):
    """One token per sequence, some at a page's last slot, some at a block's
    first, rows of length 0 among them; twice in a row."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 3 * page, (B,), generator=g).tolist()
    lens[0], lens[1], lens[2], lens[3] = 0, page, 2 * page, 17
    pool = Pool8("bhsd", BF, Hq, Hkv, page, 3 * B + 3, 4, [n + 1 if n else 0 for n in lens], seed=2)
    pool.lens = list(lens)
    cache = pool.cache()
    cos, sin = angles(3 * page + 2, 128)
    for step in range(2):
        _, q, k, v = new_tokens(pool, B, seed=step)
        k *= torch.exp2(torch.randint(-2, 5, (B, Hkv, 1), generator=g).to(BF))
        q_out = cache.append(k.cuda(), v.cuda(), q.cuda(), cos=cos.cuda(), sin=sin.cuda(),
                             q_out=torch.full_like(q, math.nan).cuda())
        want = ref8.append(pool, k, v, q, list(range(B + 1)), cos, sin)
        equal_bytes(pool, cache)
        assert same(cache.k_mean, pool.mean)
        fine = ~torch.isnan(want)
        assert torch.equal(torch.isnan(q_out).cpu(), ~fine) and torch.equal(q_out.cpu()[fine], want[fine])
        pool.lens = [n + 1 if n else 0 for n in pool.lens]
        cache.seq_lens.copy_(i32(pool.lens))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_of_extremes(dtype):
    """Zeros, the smallest and the largest entries, infinities and NaN."""
    pool = Pool8("bshd", dtype, 2, 2, 16, 3, 2, [32], seed=1)
    k, v = torch.zeros(32, 2, D, dtype=dtype), torch.zeros(32, 2, D, dtype=dtype)
    big = torch.finfo(dtype).max
    k[3, 0, :4] = torch.tensor([big, -big, 1.0, torch.finfo(dtype).tiny / 4]).to(dtype)
    k[5, 1, :3] = torch.tensor([math.inf, math.nan, 3.0])
    v[17, 0, :2] = torch.tensor([-math.inf, 500.0])
    v[20, 1] = torch.finfo(dtype).tiny
    cache = pool.cache()
    cache.append(k.cuda(), v.cuda(), cu_seqlens=i32([0, 32]))
    ref8.append(pool, k, v, None, [0, 32])
    equal_bytes(pool, cache)
    rk, rv = cache.read(32, cu_seqlens=i32([0, 32]))
    fine = torch.isfinite(k)
    assert torch.isfinite(rk.cpu()[fine]).all() and torch.isnan(rk.cpu()[~fine]).all()
    top = k.float().abs()
    scale = pool.real(torch.ones(3, 16, 2, 1), pool.ks)[pool.table[0]].reshape(32, 2, 1)
    # half a step of e4m3 (2^-4 relative, 2^-10 of the scale absolute), and what lies beyond the last byte of dtype
    most = 240.0 * (2.0 ** 8 if dtype == HF else 2.0 ** 120)
    bound = top * 2.0 ** -4 + scale * 2.0 ** -10 + (top - most).clamp(min=0.0) + 2.0 ** -25
    assert ((rk.cpu().float() - k.float()).abs() <= bound)[fine].all()


def test_append_leaves_other_memory_alone():
    """Pages that do not exist, positions outside, pages of others."""
    pool = Pool8("bhsd", BF, 2, 1, 16, 6, 2, [20, 32, 5], seed=4)
    pool.table[0][1], pool.table[2][0] = 6, -1
    cache = pool.cache()
    lens = [20, 40, 5]  # the second past what its table holds
    cache.seq_lens.copy_(i32(lens))
    pool.lens = lens
    _, q, k, v = new_tokens(pool, 40, seed=6)
    cu = [0, 10, 35, 40]
    q_out = cache.append(k.cuda(), v.cuda(), q.cuda(), cu_seqlens=i32(cu), q_out=torch.full_like(q, math.nan).cuda())
    want = ref8.append(pool, k, v, q, cu)
    equal_bytes(pool, cache)
    assert torch.equal(torch.isnan(q_out).cpu(), torch.isnan(want)) and same(cache.k_mean, pool.mean)


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("eight", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_read(layout, eight, dtype):
    lens, new = [70, 0, 33, 1, 64], [70, 2, 5, 1, 17]  # the second has no place for its two
    pool = (Pool8 if eight else Pool)(layout, dtype, 6, 3, 32, 9, 4, lens, seed=3)
    pool.table[2][1] = 100  # a page that does not exist
    cache = pool.cache()
    cu = [0] + list(itertools.accumulate(new))
    T = cu[-1] + 2
    k_out, v_out = (torch.full((T, 3, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    got = cache.read(T, cu_seqlens=i32(cu), k_out=k_out, v_out=v_out)
    assert got[0] is k_out and got[1] is v_out
    for x, src, sc in ((k_out, pool.k, getattr(pool, "ks", None)), (v_out, pool.v, getattr(pool, "vs", None))):
        real = pool.real(src, sc) if eight else src
        want = torch.full((T, 3, D), 7.0, dtype=dtype)
        for b in range(5):
            for i in range(new[b]):
                pos = lens[b] - new[b] + i
                p = pool.table[b][pos // 32] if pos >= 0 else -1
                want[cu[b] + i] = real[p, pos % 32].to(dtype) if 0 <= p < 9 else 0.0
        assert same(x, want)
    k1, v1 = cache.read(5)  # the newest of each
    assert torch.equal(k1[0], k_out[cu[1] - 1]) and torch.equal(v1[4], v_out[cu[5] - 1]) and (k1[1] == 0).all()
    assert cache.read(0, cu_seqlens=i32([0] * 6))[0].shape == (0, 3, D)


# ------------------------------------------------------------------ attend

ATTEND = [  # layout, dtype, Hq, Hkv, page, lengths, scales' spread
    ("bshd", BF, 4, 4, 16, [1], 0),
    ("bhsd", HF, 4, 1, 16, [15, 16, 17, 0, 33], 0),
    ("bshd", BF, 12, 3, 128, [101], 1),
    ("bhsd", BF, 16, 1, 64, [2000, 3, 700], 6),
    ("bshd", HF, 40, 2, 32, [500, 77], 1),                 # groups of 20: two chunks
    ("bhsd", HF, 3, 3, 256, [4000], 3),
    ("bshd", BF, 8, 2, 64, [9001, 37, 0, 1200, 5000, 64], 1),
    ("bshd", HF, 10, 2, 16, [3000] + [40] * 30, 0),
    ("bhsd", BF, 130, 10, 32, [513, 31, 0, 100], 2),
    ("bshd", BF, 1, 1, 64, [30001], 0),
    ("bhsd", HF, 64, 8, 64, [131] * 40, 1),
]


def queries(pool, seed=2, size=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((pool.B, pool.Hq, D), generator=g) * size).to(pool.dtype)


def pool_of(case, eight=True, garbage=True, wide=0):
    layout, dtype, Hq, Hkv, page, lens, spread = case
    need = [-(-n // page) for n in lens]
    if eight:
        return Pool8(layout, dtype, Hq, Hkv, page, sum(need) + 3, max(need) + 1 + wide, lens, seed=7, spread=spread,
                     garbage=garbage)
    return Pool(layout, dtype, Hq, Hkv, page, sum(need) + 3, max(need) + 1 + wide, lens, seed=7)


def lists_of(pool, seed=0, ascending=True):
    """Page lists with entries that do not exist, empty and full ones; cap <= max_pages."""
    g = torch.Generator().manual_seed(seed)
    cap = max(1, pool.max_pages - 1)
    idx = torch.full((pool.B, pool.Hkv, cap), -1, dtype=torch.int32)
    cnt = torch.zeros((pool.B, pool.Hkv), dtype=torch.int32)
    for b in range(pool.B):
        n = -(-pool.lens[b] // pool.page)
        for h in range(pool.Hkv):
            m = int(torch.randint(0, cap + 1, (1,), generator=g))
            if ascending:
                pick = sorted(torch.randperm(pool.max_pages, generator=g)[:m].tolist())
            else:
                pick = torch.randint(-2, max(n, 1) + 2, (m,), generator=g).tolist()
            idx[b, h, :m] = torch.tensor(pick, dtype=torch.int32)
            cnt[b, h] = m
    return idx, cnt


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-{max(c[5])}")
@pytest.mark.parametrize("wide", [0, 3000], ids=["", "wide-table"])
def test_attend(case, wide):
    pool = pool_of(case, wide=wide)
    q = queries(pool)
    cache = pool.cache()
    got = cache.attend(q.cuda())
    ref.check_attend(got, ref8.attend(pool, q))
    again = cache.attend(q.cuda())
    assert same(again[0], got[0]) and same(again[1], got[1])
    if not wide:
        for ascending in (True, False):
            idx, cnt = lists_of(pool, ascending=ascending)
            ref.check_attend(cache.attend(q.cuda(), (idx.cuda(), cnt.cuda())), ref8.attend(pool, q, (idx, cnt)), "lists")


@pytest.mark.parametrize("eight", [True, False])
def test_attend_with_a_scale_of_its_own(eight):
    pool = pool_of(ATTEND[4], eight)
    q, w = queries(pool), weights_of(pool)
    wd = w.cuda()
    cache = pool.cache(scale=0.02, weigh=True)
    got = cache.attend(q.cuda(), page_weight=wd)
    want = ref8.attend(pool, q, scale=0.02, weight=w)
    ref.check_attend(got, want[:4])
    check_weights(pool, wd, want, w)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", [1e-4, 1e-2, 1.0, 30.0])
def test_attend_with_queries_of_any_size(dtype, size):
    pool = Pool8("bshd", dtype, 9, 3, 32, 40, 20, [600, 31], seed=8, spread=1)
    q = queries(pool, size=size)
    q[0, 0] = 0
    q[0, 1, 1:] *= 2.0 ** -12
    ref.check_attend(pool.cache().attend(q.cuda()), ref8.attend(pool, q))


def test_attend_with_scales_far_apart():
    """Blocks whose v scales lie up to 2^60 apart, with the large ones attended
    or out of reach; keys likewise."""
    pool = Pool8("bhsd", BF, 4, 2, 16, 12, 10, [160], seed=3)
    pool.vs[:] = torch.exp2(torch.randint(-30, 31, pool.vs.shape).float())
    q = queries(pool, size=0.5)
    ref.check_attend(pool.cache().attend(q.cuda()), ref8.attend(pool, q))
    pool.vs[:] = 2.0 ** -6
    pool.vs[pool.table[0][4]] = 2.0 ** 24       # one block's values 2^30 times the others'
    ref.check_attend(pool.cache().attend(q.cuda()), ref8.attend(pool, q))
    pool.ks[:] = torch.exp2(torch.randint(-9, -4, pool.ks.shape).float())
    ref.check_attend(pool.cache().attend(q.cuda()), ref8.attend(pool, q))
    pool.v[:] = (pool.v / 448).to(E4M3).float()  # the largest scales there are, and none
    pool.vs[:] = torch.exp2(torch.randint(118, 128, pool.vs.shape).float())
    pool.vs[pool.table[0][2]] = 0.0
    ref.check_attend(pool.cache().attend(q.cuda()), ref8.attend(pool, q))


@pytest.mark.parametrize("dtype,value", [(BF, 1.0), (HF, 61440.0), (HF, 60.0), (BF, 3.0e38)])
def test_weights_sum_to_one(dtype, value):
    """A constant comes back as it is: the weights that the output is made
    with sum to one, whatever their roundings (fp32 sums: 2^-20)."""
    pool = Pool8("bshd", dtype, 4, 2, 64, 150, 150, [9001], seed=3)
    scale = ref8.scale_of(value)
    pool.v[:], pool.vs[:] = float(torch.tensor(value / scale).to(E4M3)), scale
    want = float(torch.tensor(value / scale).to(E4M3)) * scale
    out = pool.cache().attend(queries(pool).cuda())[0].double().cpu()
    assert ((out - want).abs() <= want * (2.0 ** -20 + ref.U[dtype])).all()
    assert torch.isfinite(out).all()


def test_nan_and_infinity():
    pool = Pool8("bshd", BF, 4, 2, 16, 8, 4, [40, 20], seed=5)
    q = queries(pool)
    pool.v[pool.table[0][1], 3, 0, 17] = math.nan     # an attended value: its head's dim
    pool.k[pool.table[1][0], 2, 1, 5] = math.nan      # an attended key: its head's rows
    q[0, 3, 2] = math.inf
    out, lse = (x.cpu() for x in pool.cache().attend(q.cuda()))
    assert torch.isnan(out[0, :2, 17]).all() and torch.isfinite(out[0, :2, :17]).all()
    assert torch.isnan(out[1, 2:]).all() and torch.isfinite(out[1, :2]).all()
    assert torch.isfinite(out[0, 2]).all() and torch.isnan(out[0, 3]).all() and torch.isfinite(lse[0, :3]).all()


# ------------------------------------------------------------- page weights

def weights_of(pool, seed=1, wild=False):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand((pool.B, pool.Hkv, pool.max_pages), generator=g)
    return torch.full_like(w, math.nan) if wild else w


def check_weights(pool, got, want, given):
    mass, tol = want[4], want[5]
    for b in range(pool.B):
        n = -(-pool.lens[b] // pool.page)
        assert same(got[b, :, n:], given[b, :, n:]), "entries past the end"
        d = (got[b, :, :n].double().cpu() - mass[b, :, :n]).abs()
        assert (d <= tol[b, :, :n]).all(), float((d - tol[b, :, :n]).max())


@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-{max(c[5])}")
def test_page_weights(case, eight):
    pool = pool_of(case, eight)
    q, cache = queries(pool), pool.cache(weigh=True)
    plain = cache.attend(q.cuda())
    for decay in (0.0, 0.9, 1.0):
        given = weights_of(pool, wild=decay == 0.0)
        w, to = given.cuda(), torch.full_like(given, -1.0).cuda()
        got = cache.attend(q.cuda(), page_weight=w, weight_out=to, decay=decay)
        assert same(got[0], plain[0]) and same(got[1], plain[1]) and same(w, given)
        want = ref8.attend(pool, q, weight=torch.nan_to_num(given, 0.0), decay=decay)
        check_weights(pool, to, want, given)
        cache.attend(q.cuda(), page_weight=w, decay=decay)  # in place
        assert same(w, to)
    # each query head's weights sum to one
    per = (to.double().cpu() - given.double()).sum((1, 2))
    assert ((per - torch.tensor([pool.Hq if n else 0 for n in pool.lens])).abs() <= 2.0 ** -14 * pool.Hq).all()


@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
@pytest.mark.parametrize("ascending", [True, False], ids=["ascending", "any-order"])
def test_page_weights_of_lists(eight, ascending):
    for case in (ATTEND[1], ATTEND[3], ATTEND[4], ATTEND[7]):
        pool = pool_of(case, eight)
        q, cache = queries(pool), pool.cache(weigh=True)
        idx, cnt = lists_of(pool, seed=len(case[5]), ascending=ascending)
        pages = idx.cuda(), cnt.cuda()
        plain = cache.attend(q.cuda(), pages)
        for decay in (0.5, 1.0, 0.0):
            given = weights_of(pool, wild=decay == 0.0)
            w, to = given.cuda(), torch.full_like(given, -1.0).cuda()
            got = cache.attend(q.cuda(), pages, page_weight=w, weight_out=to, decay=decay)
            assert same(got[0], plain[0]) and same(got[1], plain[1])
            check_weights(pool, to, ref8.attend(pool, q, (idx, cnt), weight=torch.nan_to_num(given, 0.0), decay=decay), given)
            cache.attend(q.cuda(), pages, page_weight=w, decay=decay)
            assert same(w, to)


# ------------------------------------------------------------------- evict

EVICT = [  # Hkv, page, max_pages, lengths, keep, keep_first, keep_last
    (1, 16, 1, [16], 1, 0, 1),
    (3, 16, 9, [16 * 9, 16 * 9 - 5, 0, 17, 1], 4, 1, 2),
    (2, 64, 40, [64 * 30 + 1] * 3, 30, 0, 1),
    (4, 32, 700, [32 * 650 + 7, 32 * 699, 40], 100, 3, 1),    # more than one chunk of a CTA
    (24, 16, 1500, [16 * 1500], 2, 1, 1),                      # nothing left to choose
    (8, 128, 33, [128 * 33, 128 * 32 + 1, 128], 3, 2, 1),
    (2, 16, 5000, [16 * 4800 + 3, 16 * 2000], 4000, 4, 8),
    (1, 256, 6, [256 * 6 + 100], 3, 0, 1),                     # a length past the table
    (2, 16, 50, [-5, 16 * 50], 60, 0, 1),                      # keeps more than the table holds
    (24, 32, 300, [32 * 290, 32 * 150 + 1], 140, 2, 3),        # one CTA with rows in several turns
    (40, 16, 700, [16 * 699 + 2], 300, 0, 1),                  # more heads than that
    (3, 16, 20000, [16 * 19990, 16 * 9000], 8500, 100, 50),    # more pages than a CTA holds at once
    (1, 16, 8300, [16 * 8300 - 1], 8299, 0, 1),
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}x{c[2]}-keep{c[4]}")
@pytest.mark.parametrize("kind", ["spread", "ties", "wild"])
def test_evict(case, kind):
    Hkv, page, P, lens, keep, first, last = case
    B = len(lens)
    g = torch.Generator().manual_seed(P)
    table = torch.randint(-3, 10000, (B, P), generator=g).to(torch.int32)  # what a row holds is moved, never looked up
    w = torch.rand((B, Hkv, P), generator=g)
    if kind == "ties":
        w = (w * 3).floor()
    if kind == "wild":
        w[torch.rand(w.shape, generator=g) < 0.1] = math.nan
        w[torch.rand(w.shape, generator=g) < 0.1] = -1.0
        w[torch.rand(w.shape, generator=g) < 0.05] = math.inf
        w[torch.rand(w.shape, generator=g) < 0.05] = -0.0
    cache = vsa.PagedCache("bshd", BF, B, Hkv, Hkv, D, page, 10000, P, page_table=table.cuda(), seq_lens=i32(lens),
                           allocate=False)
    want = ref8.evict(table.tolist(), lens, w, page, keep, first, last)
    wd = w.cuda()
    out = torch.full_like(cache.page_table, 77), torch.full_like(cache.seq_lens, 77), torch.full_like(wd, 77.0)
    freed, cnt = cache.evict(wd, keep, keep_first=first, keep_last=last, out=out)

    def check(got_table, got_lens, got_w, freed, cnt):
        assert got_table.tolist() == want[0] and got_lens.tolist() == want[1]
        assert same(got_w.contiguous(), want[2])
        assert torch.equal(freed.cpu(), want[3]) and torch.equal(cnt.cpu(), want[4])

    check(*out, freed, cnt)
    assert same(wd, w) and torch.equal(cache.page_table.cpu(), table) and cache.seq_lens.tolist() == lens
    freed2, cnt2 = cache.evict(wd, keep, keep_first=first, keep_last=last, freed=torch.full_like(freed, 5),
                               freed_cnt=torch.full_like(cnt, 5))  # in place
    check(cache.page_table, cache.seq_lens, wd, freed2, cnt2)
    freed3, cnt3 = cache.evict(wd, keep, keep_first=first, keep_last=last)  # nothing over the budget any more
    assert (cnt3 == 0).all() and (freed3 == -1).all()
    assert cache.page_table.tolist() == want[0] and cache.seq_lens.tolist() == want[1] and same(wd, want[2])


# ----------------------------------------------------------- used together

def test_decoding_within_a_budget():
    """Prompts, then steps of append (rotated by frame, row and column), attention
    with page weights, eviction and new pages from what it freed; the same steps
    on plain references, and the steps captured in a graph."""
    B, Hq, Hkv, page, P, keep, dtype = 3, 6, 2, 16, 8, 5, BF
    lens = [60, 79, 3]
    pool = Pool8("bshd", dtype, Hq, Hkv, page, B * P, P, [0] * B, seed=12)
    ids = iter(torch.randperm(B * P).tolist())
    pool.table = [[next(ids) for _ in range(P)] for _ in range(B)]
    pool.lens = list(lens)
    cache = pool.cache(weigh=True)
    rope = vsa.AxialRope((44, 42, 42), interleaved=True)
    g = torch.Generator().manual_seed(1)

    def tokens(n):
        qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g).to(dtype)
        pos = torch.randint(0, 50, (n, 3), generator=g).to(torch.int32)
        return qkv, pos

    weight = torch.zeros(B, Hkv, P, device="cuda")
    mass, slack = torch.zeros(B, Hkv, P, dtype=torch.float64), torch.zeros(B, Hkv, P, dtype=torch.float64)
    qkv, pos = tokens(sum(lens))
    cu = [0] + list(itertools.accumulate(lens))
    cos, sin = rope.table(pos.cuda())
    d = qkv.cuda()
    rows = torch.arange(sum(lens), dtype=torch.int32)
    cache.append(d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cu_seqlens=i32(cu), cos=cos, sin=sin, positions=rows.cuda(),
                 interleaved=True)
    ref8.append(pool, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], None, cu, cos.cpu(), sin.cpu(), rows, True)
    equal_bytes(pool, cache)
    evicted = 0
    own = torch.arange(B, dtype=torch.int32).cuda()
    buf, at = torch.zeros(B, Hq + 2 * Hkv, D, dtype=dtype, device="cuda"), torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    res = {}

    def step():
        cache.seq_lens.add_(1)
        c, s = rope.table(at)
        res["q"] = cache.append(buf[:, Hq:Hq + Hkv], buf[:, Hq + Hkv:], buf[:, :Hq], cos=c, sin=s, positions=own,
                                interleaved=True)
        res["out"], res["lse"] = cache.attend(res["q"], page_weight=weight)
        res["freed"], res["cnt"] = cache.evict(weight, keep, keep_first=1, keep_last=2)
        res["cos"], res["sin"] = c, s

    graph = None
    for i in range(45):
        qkv, pos = tokens(B)
        buf.copy_(qkv)
        at.copy_(pos)
        if i == 10:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        pool.lens = [n + 1 for n in pool.lens]
        q = ref8.append(pool, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], qkv[:, :Hq], list(range(B + 1)), res["cos"].cpu(),
                        res["sin"].cpu(), torch.arange(B), True)
        assert torch.equal(res["q"].cpu(), q)
        equal_bytes(pool, cache)
        want = ref8.attend(pool, q, weight=mass)
        ref.check_attend((res["out"], res["lse"]), want[:4], f"step {i}")
        # what the device holds decides (two pages may weigh the same to rounding): it is near the reference's, and the
        # eviction is right for it
        mass, slack = want[4], slack + want[5]
        counts = [-(-n // page) for n in pool.lens]
        tables, new_lens = cache.page_table.tolist(), cache.seq_lens.tolist()
        for b in range(B):
            gone = int(res["cnt"][b])
            assert gone == max(0, counts[b] - keep)
            if not gone:
                continue
            evicted += gone
            out_ids = res["freed"][b, :gone].tolist()
            left = [j for j in range(P) if pool.table[b][j] not in out_ids]
            went = [j for j in range(P) if pool.table[b][j] in out_ids]
            assert all(1 <= j < counts[b] - 2 for j in went)
            total, err = mass[b].sum(0), slack[b].sum(0)
            rest = [j for j in range(1, counts[b] - 2) if j not in went]
            assert max(float(total[j] - err[j]) for j in went) <= min(float(total[j] + err[j]) for j in rest)
            assert tables[b] == [pool.table[b][j] for j in left] + [-1] * gone
            pool.lens[b] -= gone * page
            pad = torch.zeros(Hkv, gone, dtype=torch.float64)
            mass[b] = torch.cat((mass[b][:, left], pad), 1)
            slack[b] = torch.cat((slack[b][:, left], pad), 1)
            # the freed pages go behind the sequence's others, to be filled anew
            pool.table[b] = [pool.table[b][j] for j in left] + out_ids
            cache.page_table[b, P - gone:] = i32(out_ids)
        assert new_lens == pool.lens
        assert ((weight.double().cpu() - mass).abs() <= slack).all()
    assert evicted > 4


def test_prefill_from_an_8_bit_cache():
    """A prompt read back from the cache attends to itself: append, read, block-sparse
    attention on packed sequences."""
    Hq, Hkv, dtype, lens = 4, 2, HF, [200, 131]
    pool = Pool8("bhsd", dtype, Hq, Hkv, 64, 8, 4, lens, seed=2)
    cache = pool.cache()
    T = sum(lens)
    _, q, k, v = new_tokens(pool, T)
    cu = i32([0, 200, 331])
    cache.append(k.cuda(), v.cuda(), cu_seqlens=cu)
    kk, vv = cache.read(T, cu_seqlens=cu)
    ref8.append(pool, k, v, None, [0, 200, 331])
    plan = vsa.Plan("tnd", dtype, 2, Hq, Hkv, D, 128, 128, 2, 2, T, T, 2, cu_seqlens_q=cu, cu_seqlens_kv=cu)
    plan.mask_to_index(torch.ones(2, Hq, 2, 2, dtype=torch.uint8, device="cuda"))
    out, _, _ = plan.forward(q.cuda(), kk, vv)
    for b, (s, e) in enumerate(((0, 200), (200, 331))):
        for h in range(Hq):
            kb, vb, _, _ = ref8.rows_of(pool, b, h // 2, range(-(-lens[b] // 64)))
            want = torch.softmax(q[s:e, h].double() @ kb.T / math.sqrt(D), 1) @ vb
            rel = float((out[s:e, h].double().cpu() - want).norm() / want.norm())
            assert rel <= 4 * ref.U[dtype], rel  # P and the output round to fp16, the values read are exact


def test_selected_pages_of_an_8_bit_cache():
    """append's means feed select, whose lists feed attend."""
    pool = Pool8("bshd", BF, 8, 2, 32, 30, 15, [460, 333], seed=6)
    cache = pool.cache(weigh=True)
    _, q, k, v = new_tokens(pool, 793)
    cu = [0, 460, 793]
    cache.append(k.cuda(), v.cuda(), cu_seqlens=i32(cu))
    ref8.append(pool, k, v, None, cu)
    qq = queries(pool)
    pages = cache.select(qq.cuda(), 6, keep_first=1, keep_last=2)
    want = ref.select(pool, qq, 6, 1, 2)
    assert torch.equal(pages[0].cpu(), want[0]) and torch.equal(pages[1].cpu(), want[1])
    w = torch.zeros(2, 2, 15)
    wd = w.cuda()
    got = cache.attend(qq.cuda(), pages, page_weight=wd)
    full = ref8.attend(pool, qq, want, weight=w)
    ref.check_attend(got, full[:4])
    check_weights(pool, wd, full, w)


def test_streams_shared_workspace_and_graphs():
    """Two layers on one workspace and table, eager and captured, on a side stream."""
    pool = Pool8("bshd", BF, 8, 2, 64, 60, 20, [1200, 37, 800], seed=5)
    a = pool.cache(weigh=True)
    other = Pool8("bshd", BF, 8, 2, 64, 60, 20, [1200, 37, 800], seed=6)
    b = other.cache(page_table=a.page_table, seq_lens=a.seq_lens, workspace=a.workspace, weigh=True)
    q = queries(pool).cuda()
    w = [weights_of(pool, s).cuda() for s in (1, 2)]
    to = [torch.empty_like(x) for x in w]
    want = [(c.attend(q, page_weight=x, weight_out=y, decay=0.5), y.clone()) for c, x, y in zip((a, b), w, to)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [c.attend(q, page_weight=x, weight_out=torch.empty_like(x), decay=0.5, stream=side) for c, x in zip((a, b), w)]
    side.synchronize()
    for (got, _), g in zip(want, outs):
        assert same(got[0], g[0]) and same(got[1], g[1])
    graph = torch.cuda.CUDAGraph()
    lay = [torch.empty_like(want[0][0][0]) for _ in range(2)]
    with torch.cuda.graph(graph):
        for c, x, y, o in zip((a, b), w, to, lay):
            c.attend(q, page_weight=x, weight_out=y, decay=0.5, out=o)
            c.attend(q, out=o)
            c.attend(q, page_weight=x, weight_out=y, decay=0.5, out=o)
    for y in to:
        y.fill_(-1.0)
    for _ in range(3):
        graph.replay()
    for (got, y0), o, y in zip(want, lay, to):
        assert same(got[0], o) and same(y0, y)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: pages at its far end."""
    Hkv, page = 64, 256
    size = page * Hkv * D
    pages = (1 << 32) // size + 6
    k = torch.empty(pages, page, Hkv, D, dtype=E4M3, device="cuda")
    v = torch.empty_like(k)
    last = [pages - 1, 2, pages - 4]
    cache = vsa.PagedCache("bshd", BF, 1, Hkv, Hkv, D, page, pages, 3, k=k, v=v,
                           k_scale=torch.ones(pages, Hkv, page // 16, device="cuda"),
                           v_scale=torch.ones(pages, Hkv, page // 16, device="cuda"), k_mean=False,
                           page_table=i32([last]), seq_lens=i32([600]), kv_dtype=E4M3)
    g = torch.Generator(device="cuda").manual_seed(3)
    kk, vv = (torch.randn(600, Hkv, D, generator=g, device="cuda").to(BF) for _ in range(2))
    cache.append(kk, vv, cu_seqlens=i32([0, 600]))
    rk, rv = cache.read(600, cu_seqlens=i32([0, 600]))
    near = vsa.PagedCache("bshd", BF, 1, Hkv, Hkv, D, page, 3, 3, k_mean=False, kv_dtype=E4M3, page_table=i32([[0, 1, 2]]),
                          seq_lens=i32([600]))
    near.append(kk, vv, cu_seqlens=i32([0, 600]))
    nk, nv = near.read(600, cu_seqlens=i32([0, 600]))
    assert same(rk, nk) and same(rv, nv)
    assert ((rk - kk).float().abs() <= kk.float().abs() * 2.0 ** -4 + 2.0 ** -7).all()
    q = torch.randn(1, Hkv, D, generator=g, device="cuda").to(BF)
    for x, y in zip(cache.attend(q), near.attend(q)):
        assert same(x, y)
