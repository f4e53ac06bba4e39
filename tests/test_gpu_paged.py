"""Paged-cache calls against plain references: appending (bit for bit),
page selection (index for index) and one-token attention (fp64, bounds from
the roundings)."""
import itertools
import math

import pytest
import torch

from bwd_tile_mean_gb300 import vsa
from tests import paged_ref as ref
from tests.paged_ref import D, Pool

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def angles(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def new_tokens(pool, T, seed=5):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, pool.Hq + 2 * pool.Hkv, D), generator=g).to(pool.dtype)
    return qkv, qkv[:, :pool.Hq], qkv[:, pool.Hq:pool.Hq + pool.Hkv], qkv[:, pool.Hq + pool.Hkv:]


def split(pool, x):
    return x[:, :pool.Hq], x[:, pool.Hq:pool.Hq + pool.Hkv], x[:, pool.Hq + pool.Hkv:]


def same(a, b):
    """Equal bit for bit (NaN included)."""
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16)) if a.dtype in (BF, HF) else \
        torch.equal(a.cpu().view(torch.int32), b.cpu().view(torch.int32))


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
    ("bshd", BF, 48, 24, 64, 96, True, [1500, 900, 450], [1450, 900, 400]),   # many rows: four key heads per warp
    ("bhsd", HF, 23, 23, 256, 128, False, [2100, 800], [2100, 777]),
    ("bhsd", HF, 15, 5, 64, 96, False, [130, 64, 128, 71, 70] * 6, [70, 64, 70, 71, 3] * 6),  # two key heads per warp
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-r{c[5]}-{'i' if c[6] else 'h'}")
@pytest.mark.parametrize("with_pos", [False, True], ids=["own-rows", "given-rows"])
def test_append(case, with_pos):
    layout, dtype, Hq, Hkv, page, rot, inter, lens, new = case
    need = sum(-(-n // page) for n in lens)
    pool = Pool(layout, dtype, Hq, Hkv, page, need + 2, max(-(-n // page) for n in lens) + 1, lens, seed=len(lens))
    tail = 3  # tokens behind the last sequence
    T = sum(new) + tail
    qkv, q, k, v = new_tokens(pool, T)
    cu = [0] + list(itertools.accumulate(new))
    cos, sin = angles(max(lens) + 1, rot) if rot else (None, None)
    pos = torch.randint(-2, max(lens) + 4, (T,), dtype=torch.int32) if with_pos else None
    cache = pool.cache()
    dq, dk, dv = split(pool, qkv.cuda())
    q_out = torch.full((T, Hq, D), math.nan, dtype=dtype, device="cuda")
    cud = lambda x: None if x is None else x.cuda()  # noqa: E731
    got = cache.append(dk, dv, dq, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), cos=cud(cos), sin=cud(sin),
                       positions=cud(pos), interleaved=inter, q_out=q_out)
    assert got is q_out
    want = ref.append(pool, k, v, q, cu, cos, sin, pos, inter)
    assert same(pool.back(cache.k).contiguous(), pool.k), "keys"
    assert same(pool.back(cache.v).contiguous(), pool.v), "values"
    assert same(cache.k_mean, pool.mean), "means"
    assert torch.equal(torch.isnan(q_out).cpu(), torch.isnan(want)), "q rows written"
    fine = ~torch.isnan(want)
    assert torch.equal(q_out.cpu()[fine], want[fine]), "queries"
    # the rotation against fp64: three fp32 roundings and one of dtype
    if rot and not with_pos:
        for b in range(pool.B):
            for t in range(cu[b], cu[b + 1]):
                r = lens[b] - new[b] + t - cu[b]
                y = torch.from_numpy(ref.rotate(q[t:t + 1], cos[r:r + 1], sin[r:r + 1], inter, "f8"))[0]
                size = q[t].double().abs().amax()
                assert ((q_out[t].cpu().double() - y).abs() <= ref.U[dtype] * y.abs() + 8 * 2.0 ** -24 * size).all()
    # the same call again changes nothing
    before = [x.clone() for x in (cache.k, cache.v, cache.k_mean, q_out)]
    cache.append(dk, dv, dq, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), cos=cud(cos), sin=cud(sin),
                 positions=cud(pos), interleaved=inter, q_out=q_out)
    assert all(same(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_mean, q_out)))


@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_in_pieces_gives_the_same_bits(page):
    lens, final = [1, 1], [2 * page + 5, 3 * page]
    pool = Pool("bshd", BF, 6, 3, page, 8, 4, final, seed=9)
    qkv, q, k, v = new_tokens(pool, sum(final), seed=10)
    cos, sin = (x.cuda() for x in angles(max(final), 128))
    whole, pieces = pool.cache(), pool.cache()
    cu = torch.tensor([0, final[0], sum(final)], dtype=torch.int32).cuda()
    dk, dv = k.cuda(), v.cuda()
    whole.append(dk, dv, cu_seqlens=cu, cos=cos, sin=sin)
    done = [0, 0]
    for step in (1, page - 2, 1, 7, page, 10 * page):  # page ends inside, at and after a piece
        n = [min(step, f - d) for f, d in zip(final, done)]
        part = [torch.arange(o + d, o + d + m) for o, d, m in zip((0, final[0]), done, n)]
        at = torch.cat(part).cuda()
        done = [d + m for d, m in zip(done, n)]
        pieces.seq_lens.copy_(torch.tensor(done, dtype=torch.int32))
        pieces.append(dk[at], dv[at], cu_seqlens=torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32).cuda(),
                      cos=cos, sin=sin)
    assert done == final
    for a, b in ((whole.k, pieces.k), (whole.v, pieces.v), (whole.k_mean, pieces.k_mean)):
        assert same(a, b)


@pytest.mark.parametrize("B", [3, 200, 1300])
def test_append_one_token_each(B):
    """Without offsets; one, two and four key heads per warp."""
    lens = [0 if b % 13 == 7 else (b % 3 + 1) * 32 if b % 4 == 0 else 1 + b % 70 for b in range(B)]
    pool = Pool("bshd", BF, 6, 3, 32, sum(-(-n // 32) for n in lens), 4, lens, seed=18)
    qkv, q, k, v = new_tokens(pool, B, seed=19)
    cos, sin = angles(100, 128)
    cache = pool.cache()
    dq, dk, dv = split(pool, qkv.cuda())
    q_out = torch.full((B, 6, D), math.nan, dtype=BF, device="cuda")
    cache.append(dk, dv, dq, cos=cos.cuda(), sin=sin.cuda(), q_out=q_out)
    want = ref.append(pool, k, v, q, list(range(B + 1)), cos, sin)
    assert same(cache.k, pool.k) and same(cache.v, pool.v) and same(cache.k_mean, pool.mean)
    fine = ~torch.isnan(want)
    assert torch.equal(torch.isnan(q_out).cpu(), ~fine) and torch.equal(q_out.cpu()[fine], want[fine])


def test_append_to_many_sequences():
    """More sequences than two steps of the search hold, some without tokens."""
    new = [b % 3 if b % 11 else 0 for b in range(1100)]
    lens = [n + (b % 29 if n else 0) for b, n in enumerate(new)]
    pool = Pool("bshd", BF, 2, 1, 16, sum(-(-n // 16) for n in lens), 2, lens, seed=17)
    cu = [0] + list(itertools.accumulate(new))
    qkv, q, k, v = new_tokens(pool, cu[-1])
    cos, sin = angles(32, 128)
    cache = pool.cache()
    got = cache.append(k.cuda(), v.cuda(), q.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                       cos=cos.cuda(), sin=sin.cuda())
    want = ref.append(pool, k, v, q, cu, cos, sin)
    assert same(cache.k, pool.k) and same(cache.v, pool.v) and same(cache.k_mean, pool.mean) and same(got, want)


def test_append_ignores_what_has_no_place():
    # lengths past the table, more new tokens than the length, page ids outside the pool, no tokens
    pool = Pool("bshd", HF, 4, 2, 16, 8, 3, [48, 20, 7, 5], seed=3)
    pool.table[1][0], pool.table[2][0] = 8, -1
    pool.lens = [60, 20, 7, 5]      # three pages hold 48
    new = [30, 20, 3, 9]            # the last sequence's first four would sit before 0
    cu = [0] + list(itertools.accumulate(new))
    qkv, q, k, v = new_tokens(pool, cu[-1])
    cos, sin = angles(8, 128)       # fewer rows than positions: the last row is taken
    cache = pool.cache()
    q_out = torch.full((cu[-1], 4, D), math.nan, dtype=HF, device="cuda")
    cache.append(k.cuda(), v.cuda(), q.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), cos=cos.cuda(),
                 sin=sin.cuda(), q_out=q_out)
    want = ref.append(pool, k, v, q, cu, cos, sin)
    assert same(cache.k, pool.k) and same(cache.v, pool.v) and same(cache.k_mean, pool.mean)
    assert torch.equal(torch.isnan(q_out).cpu(), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(q_out.cpu()[fine], want[fine])
    # no tokens at all
    before = cache.k.clone()
    assert cache.append(k[:0].cuda(), v[:0].cuda(), cu_seqlens=torch.zeros(5, dtype=torch.int32).cuda()) is None
    assert same(cache.k, before)


def test_append_without_means_or_queries_and_in_halves_of_one_buffer():
    pool = Pool("bhsd", BF, 4, 2, 32, 5, 2, [64, 33, 1], seed=12)
    both = torch.randn(5, 2, 2, 32, D, device="cuda").to(BF)
    k0, v0 = both[:, 0], both[:, 1]
    k0.copy_(pool.view(pool.k).cuda())
    v0.copy_(pool.view(pool.v).cuda())
    cache = pool.cache(k=k0, v=v0, k_mean=False)
    qkv, q, k, v = new_tokens(pool, 3)
    assert cache.append(*(x.cuda() for x in (k, v))) is None
    ref.append(pool, k, v, None, [0, 1, 2, 3], means=False)
    assert same(pool.back(both[:, 0]).contiguous(), pool.k) and same(pool.back(both[:, 1]).contiguous(), pool.v)
    out = cache.attend(q.cuda())
    ref.check_attend(out, ref.attend(pool, q))


# ------------------------------------------------------------------ select

SELECT = [  # layout, dtype, Hq, Hkv, page, lengths, topk, keep_first, keep_last
    ("bshd", BF, 4, 2, 16, [1000, 0, 1, 16, 17, 15 * 16, 999], 8, 0, 1),
    ("bhsd", HF, 3, 3, 64, [64 * 300 + 5], 24, 1, 2),
    ("bshd", BF, 40, 5, 16, [16 * 1000, 16 * 129, 16 * 128 + 1], 64, 2, 3),
    ("bshd", HF, 1, 1, 256, [256 * 40], 39, 0, 1),
    ("bhsd", BF, 6, 2, 32, [32 * 50, 32 * 49 + 7], 1, 0, 1),
    ("bhsd", BF, 16, 1, 16, [16 * 5000 + 3, 16 * 700], 300, 4, 4),
    ("bshd", BF, 4, 2, 16, [100, 16, 0, 333], 64, 0, 1),                          # fewer pages than are asked for
    ("bhsd", HF, 24, 24, 16, [b * 71 % 1400 for b in range(20)], 20, 1, 1),       # many heads: two groups, many clusters
    ("bshd", BF, 96, 3, 64, [64 * 900, 64 * 350 + 9, 64 * 41], 33, 0, 2),         # 32 query heads each
    ("bhsd", HF, 4, 1, 16, [16 * 30000 + 5, 16 * 21], 900, 2, 2),
]


def select_pool(case, seed=21):
    layout, dtype, Hq, Hkv, page, lens = case[:6]
    need = [-(-n // page) for n in lens]
    pool = Pool(layout, dtype, Hq, Hkv, page, sum(need) + 1, max(need), lens, seed=seed)
    q = torch.randn((pool.B, Hq, D), generator=pool.gen).to(dtype)
    return pool, q


def check_select(pool, q, topk, first, last):
    """With the table as it is and with much wider ones: the call takes
    other variants for tables of many pages."""
    want = ref.select(pool, q, topk, first, last)
    for wide in (0, 4000, 25000):
        table = torch.nn.functional.pad(torch.tensor(pool.table, dtype=torch.int32), (0, wide), value=-9)
        cache = vsa.PagedCache(pool.layout, pool.dtype, pool.B, pool.Hq, pool.Hkv, D, pool.page, pool.num_pages,
                               pool.max_pages + wide, k_mean=pool.mean.cuda(), page_table=table.cuda(),
                               seq_lens=torch.tensor(pool.lens, dtype=torch.int32).cuda(), allocate=False)
        idx, cnt = cache.select(q.cuda(), topk, keep_first=first, keep_last=last)
        assert torch.equal(cnt.cpu(), want[1])
        assert torch.equal(idx.cpu(), want[0])


@pytest.mark.parametrize("case", SELECT, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-k{c[6]}")
def test_select(case):
    pool, q = select_pool(case)
    check_select(pool, q, *case[6:])


def test_select_ties_and_special_scores():
    case = ("bshd", BF, 4, 2, 16, [16 * 400, 16 * 300 + 1], 0, 0, 0)
    pool, q = select_pool(case)
    pool.mean[:] = pool.mean[:1]                      # all pages score alike: the lowest indices
    check_select(pool, q, 20, 0, 1)
    pool, q = select_pool(case)
    pool.mean[torch.rand(pool.num_pages, generator=pool.gen) < 0.6] = 0.0   # zero of either sign
    pool.mean[torch.rand(pool.num_pages, generator=pool.gen) < 0.3] *= -0.0
    check_select(pool, q, 150, 1, 1)
    pool, q = select_pool(case)
    q = q.abs()
    for value in (math.nan, math.inf, -math.inf):
        pool.mean[torch.rand(pool.num_pages, generator=pool.gen) < 0.2] = value
    for k in (30, 200, 390):
        check_select(pool, q, k, 2, 2)
    pool.table[0][3], pool.table[0][5], pool.table[1][0] = -1, pool.num_pages, 1 << 30  # no such pages
    for k in (30, 390):
        check_select(pool, q, k, 0, 1)


def test_select_batch_of_many_sequences():
    """More sequences than one scan of a CTA holds, most without a choice."""
    lens = [16 * 40 + 3 if b % 37 == 5 else b % 90 for b in range(300)]
    pool, q = select_pool(("bhsd", HF, 2, 2, 16, lens, 0, 0, 0))
    check_select(pool, q, 7, 1, 2)


def test_select_strided_queries():
    pool, q = select_pool(SELECT[2])
    wide = torch.randn((pool.B, pool.Hq + 7, D), device="cuda").to(BF)
    wide[:, :pool.Hq] = q.cuda()
    cache = pool.cache(k=None, v=None, allocate=False)
    idx, cnt = cache.select(wide[:, :pool.Hq], 64, keep_first=2, keep_last=3)
    want = ref.select(pool, q, 64, 2, 3)
    assert torch.equal(idx.cpu(), want[0]) and torch.equal(cnt.cpu(), want[1])


# ------------------------------------------------------------------ attend

EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300]
ATTEND = [  # layout, dtype, Hq, Hkv, page, lengths
    ("bshd", BF, 1, 1, 16, EDGE),
    ("bhsd", HF, 3, 3, 32, EDGE),
    ("bshd", HF, 12, 3, 128, EDGE),
    ("bhsd", BF, 8, 1, 64, EDGE),
    ("bshd", BF, 32, 2, 256, EDGE),
    ("bhsd", HF, 34, 2, 16, [5, 64, 200]),
    ("bshd", BF, 80, 2, 16, [1, 100, 0, 333]),
    ("bhsd", BF, 64, 2, 128, [129, 1, 257]),
    ("bshd", BF, 2, 2, 64, [6000, 1, 0, 3001]),
    ("bhsd", HF, 16, 1, 16, [20011]),
    ("bshd", BF, 10, 2, 32, [7] * 200),
    ("bhsd", BF, 80, 80, 64, [1100]),                # clusters of two CTAs
    ("bshd", HF, 60, 20, 32, [700, 321, 0]),         # of four
    ("bshd", BF, 64, 4, 64, [1000, 999]),            # of eight
    ("bhsd", HF, 40, 2, 16, [3000]),                 # of sixteen, two chunks of a group's heads
]


def attend_pool(case, seed=31, fill=None):
    layout, dtype, Hq, Hkv, page, lens = case
    need = [-(-n // page) for n in lens]
    pool = Pool(layout, dtype, Hq, Hkv, page, sum(need) + 3, max(need) + 1, lens, seed=seed, fill=fill)
    q = (torch.randn((pool.B, Hq, D), generator=pool.gen) * 2).to(dtype)
    return pool, q


def spoil(pool):
    """NaN and infinities in every slot that no sequence holds."""
    held = torch.zeros(pool.num_pages, pool.page, dtype=torch.bool)
    for b, n in enumerate(pool.lens):
        for pos in range(n):
            held[pool.table[b][pos // pool.page], pos % pool.page] = True
    for x, value in ((pool.k, math.nan), (pool.v, math.inf)):
        x[~held] = value


def widened(pool, entries):
    """The pool's cache with a page table that much wider: the call takes
    another variant for tables that allow long sequences."""
    table = torch.nn.functional.pad(torch.tensor(pool.table, dtype=torch.int32), (0, entries), value=-9)
    return vsa.PagedCache(pool.layout, pool.dtype, pool.B, pool.Hq, pool.Hkv, D, pool.page, pool.num_pages,
                          pool.max_pages + entries, k=pool.view(pool.k).cuda(), v=pool.view(pool.v).cuda(),
                          k_mean=pool.mean.cuda(), page_table=table.cuda(),
                          seq_lens=torch.tensor(pool.lens, dtype=torch.int32).cuda())


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-b{len(c[5])}")
def test_attend(case):
    pool, q = attend_pool(case)
    spoil(pool)
    want = ref.attend(pool, q)
    for cache in (pool.cache(), widened(pool, 70000 // pool.page)):
        got = cache.attend(q.cuda())
        ref.check_attend(got, want, "all pages")
        again = cache.attend(q.cuda())
        assert same(got[0], again[0]) and same(got[1], again[1])


RAGGED = [9000, 1, 0, 300, 5003, 17, 0, 0, 64, 2048, 1, 777, 4096, 33, 15, 6001]


@pytest.mark.parametrize("Hq,Hkv,page", [(16, 1, 16), (3, 3, 64), (20, 1, 32), (8, 2, 128)])
def test_attend_ragged_batch_in_equal_runs(Hq, Hkv, page):
    """Segments that end inside a warp's run, a CTA's run, and span many."""
    pool, q = attend_pool(("bhsd", BF, Hq, Hkv, page, RAGGED), seed=33)
    spoil(pool)
    got = widened(pool, 70000 // page).attend(q.cuda())
    ref.check_attend(got, ref.attend(pool, q), "ragged")


def test_attend_long_list_in_equal_runs():
    pool, q = attend_pool(("bhsd", HF, 16, 1, 16, [20011, 300]), seed=34)
    g = torch.Generator().manual_seed(8)
    idx = torch.full((2, 1, 2200), -1, dtype=torch.int32)
    cnt = torch.tensor([[1251], [7]], dtype=torch.int32)
    for b in range(2):
        n = int(cnt[b, 0])
        idx[b, 0, :n] = torch.randperm(-(-pool.lens[b] // 16), generator=g)[:n].int()
    got = widened(pool, 3000).attend(q.cuda(), (idx.cuda(), cnt.cuda()))
    ref.check_attend(got, ref.attend(pool, q, (idx, cnt)), "long list")


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-b{len(c[5])}")
def test_attend_listed_pages(case):
    pool, q = attend_pool(case, seed=32)
    spoil(pool)
    g = torch.Generator().manual_seed(4)
    cap = 9
    idx = torch.full((pool.B, pool.Hkv, cap), -1, dtype=torch.int32)
    cnt = torch.zeros((pool.B, pool.Hkv), dtype=torch.int32)
    for b, h in itertools.product(range(pool.B), range(pool.Hkv)):
        n = -(-pool.lens[b] // pool.page)
        some = torch.randperm(n, generator=g)[:int(torch.randint(0, cap + 1, (1,), generator=g))]
        idx[b, h, :len(some)] = some.int()            # in any order
        cnt[b, h] = len(some)
    # entries that are no pages hold no key; a page twice counts twice; counts are clamped
    idx[0, 0, :4] = torch.tensor([-1, pool.max_pages, pool.max_pages - 1, 1 << 30], dtype=torch.int32)
    cnt[0, 0] = 4
    if pool.B > 2:
        idx[2, 0] = 0
        cnt[2, 0] = 100
        cnt[1, 0] = -5
    got = pool.cache().attend(q.cuda(), (idx.cuda(), cnt.cuda()))
    ref.check_attend(got, ref.attend(pool, q, (idx, cnt)), "listed")


def test_attend_scale_strides_and_bad_lengths():
    pool, q = attend_pool(("bshd", BF, 8, 2, 32, [90, 33, 64]), seed=40)
    wide = torch.randn((3, 17, D), device="cuda").to(BF)
    wide[:, 3:11] = q.cuda()
    got = pool.cache(scale=0.25).attend(wide[:, 3:11])
    ref.check_attend(got, ref.attend(pool, q, scale=0.25), "scale")
    pool.table[2][1] = pool.num_pages + 5              # a page that does not exist: 32 of 64 keys remain
    ref.check_attend(pool.cache().attend(q.cuda()), ref.attend(pool, q), "bad page")
    cache = pool.cache(seq_lens=torch.tensor([90, -4, 1 << 30], dtype=torch.int32, device="cuda"))
    out, lse = cache.attend(q.cuda())
    pool.lens = [90, 0, pool.max_pages * pool.page]
    ref.check_attend((out, lse), ref.attend(pool, q), "clamped lengths")


def test_attend_special_values():
    pool, q = attend_pool(("bhsd", HF, 4, 2, 16, [40, 40, 40, 40, 40]), seed=41)
    q = q.abs()
    p = lambda b, pos: (pool.table[b][pos // 16], pos % 16)  # noqa: E731
    pool.v[p(0, 5)] = math.inf                          # an infinity that is attended
    pool.k[p(1, 7)] = math.nan                          # a score that is NaN
    for pos in range(40):
        pool.k[p(2, pos)] = -math.inf                   # every score -inf: as without keys
    pool.k[p(3, 20)] = -math.inf                        # one key that gets no weight
    pool.k[p(4, 39)] = 65504.0                          # one key that gets all of it
    pool.v[p(4, 0)] = 65504.0
    out, lse = pool.cache().attend(q.cuda())
    w = ref.attend(pool, q)
    assert torch.isinf(out[0]).all() and (out[0] > 0).all()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    o, l = out.double().cpu(), lse.double().cpu()
    assert ((o[4] - w[0][4]).abs() <= w[2][4]).all()
    # row 3 is the row without its key 20: scores of a few units, 39 keys; weights off by 2^-11
    # (rounded) + 2^-14 (scores), the output by 2^-11 of itself
    live = [x for x in range(40) if x != 20]
    k, v = (torch.stack([c[p(3, x)] for x in live]).double() for c in (pool.k, pool.v))
    for h in range(4):
        s = k[:, h // 2] @ q[3, h].double() * D ** -0.5
        want = torch.softmax(s, 0) @ v[:, h // 2]
        assert ((o[3, h] - want).abs() <= 2.5 * 2.0 ** -11 * v[:, h // 2].abs().amax()).all()
        assert abs(float(l[3, h] - torch.logsumexp(s, 0))) < 1e-4


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [[9001], [9001, 33, 5000]])
def test_attend_one_large_score_before_a_long_tail(dtype, lens):
    """The first key's weight is e^16 times every other's, and its value 0:
    the output is the sum of thousands of weights of 1e-7 each."""
    pool, q = attend_pool(("bshd", dtype, 4, 2, 64, lens), seed=44)
    q.fill_(1.0)
    pool.k.zero_()
    pool.v.copy_(pool.v.abs())
    for b in range(pool.B):
        first = pool.table[b][0]
        pool.k[first, 0] = 16.0 / (D * D ** -0.5)
        pool.v[first, 0] = 0.0
    want = ref.attend(pool, q)
    assert float(want[0][0].amax()) < 2e-3
    for cache in (pool.cache(), widened(pool, 70000 // pool.page)):
        ref.check_attend(cache.attend(q.cuda()), want, "long tail")


@pytest.mark.parametrize("dtype,value", [(BF, 1.0), (BF, -2.984375), (HF, 1.0), (HF, 65504.0)])
@pytest.mark.parametrize("lens", [[300], [9001], [9001, 33, 5000]])
def test_attend_gives_a_constant_value_back(dtype, value, lens):
    """Every 16th score 0 (one for each block of a warp's run), the others
    between -0.69 and -0.77, the same within a head, so that all weights of a
    head round the same way (by up to half a step: the heads differ), and
    every value the same: so is the output, from clusters, equal runs and page
    lists. The 16-bit weights' sum is taken as their products with V are, so
    their roundings cancel; what is left is that of fp32 sums of at most
    9,001 / 16 steps: 563 * 2^-23 = 6.7e-5, below half a step of either type
    (fp16 at 65504: 2.4e-4)."""
    pool, q = attend_pool(("bshd", dtype, 16, 2, 64, lens), seed=46)
    q.copy_((1 + torch.arange(16) / 128)[None, :, None].expand_as(q))
    pool.k.fill_(-0.69 / D ** 0.5)
    pool.v.fill_(value)
    pool.k[:, ::16] = 0.0
    want = ref.attend(pool, q)
    every = torch.full((pool.B, 2, pool.max_pages), -1, dtype=torch.int32)
    cnt = torch.zeros((pool.B, 2), dtype=torch.int32)
    for b, n in enumerate(lens):
        cnt[b] = -(-n // 64)
        every[b, :, :cnt[b, 0]] = torch.arange(int(cnt[b, 0]), dtype=torch.int32)
    for cache, pages in itertools.product((pool.cache(), widened(pool, 70000 // 64)), (None, (every.cuda(), cnt.cuda()))):
        out, lse = cache.attend(q.cuda(), pages)
        assert (out == value).all(), float(out[0, 0, 0])
        assert ((lse.double().cpu() - want[1]).abs() <= want[3]).all()


@pytest.mark.parametrize("Hq,Hkv,page", [(16, 1, 16), (3, 3, 64), (20, 1, 32), (8, 2, 128)])
@pytest.mark.parametrize("classes", [128, 127, 101])
def test_attend_counts_every_block_once(Hq, Hkv, page, classes):
    """Equal scores, and dim d of V set in the 16-key blocks d, d + classes,
    ... only: dim d of the output is the share of those keys, so a block that
    is lost, doubled or taken for its neighbour shows. All weights are alike
    and counts are exact, so a share is off by its own rounding and a few of
    fp32's (2^-20)."""
    pool, q = attend_pool(("bhsd", BF, Hq, Hkv, page, RAGGED), seed=47)
    q.zero_()
    pool.v.zero_()
    spoil(pool)
    counts = torch.zeros((pool.B, D), dtype=torch.float64)
    for b, n in enumerate(pool.lens):
        for pos in range(n):
            pool.v[pool.table[b][pos // page], pos % page, :, pos // 16 % classes] = 1.0
            counts[b, pos // 16 % classes] += 1
    lens = torch.tensor(pool.lens, dtype=torch.float64)
    share = (counts / lens.clamp(min=1)[:, None])[:, None].expand(-1, Hq, -1)
    logs = lens.log()[:, None].expand(-1, Hq)
    idx = torch.full((pool.B, Hkv, pool.max_pages + 2), -1, dtype=torch.int32)
    cnt = torch.zeros((pool.B, Hkv), dtype=torch.int32)
    for b, n in enumerate(pool.lens):
        order = torch.randperm(-(-n // page), generator=pool.gen).int()
        cnt[b] = len(order)
        idx[b, :, :len(order)] = order
    for cache, pages in itertools.product((pool.cache(), widened(pool, 70000 // page)), (None, (idx.cuda(), cnt.cuda()))):
        out, lse = (x.double().cpu() for x in cache.attend(q.cuda(), pages))
        assert ((out - share).abs() <= (ref.U[BF] + 2.0 ** -20) * share).all()
        assert torch.equal(lse == -math.inf, logs == -math.inf)
        held = logs > -math.inf
        assert ((lse - logs).abs()[held] <= 2.0 ** -20 * (1 + logs[held])).all()


@pytest.mark.parametrize("lens", [[40], [9001], [9001, 33, 5000]])
def test_attend_scores_past_the_exponents_last_bit(lens):
    """Scores of 1e13, whose last bit is worth thousands: the largest one's
    weight is 1 all the same and the output its value."""
    pool, q = attend_pool(("bhsd", BF, 4, 2, 64, lens), seed=45)
    q = (q.float().abs() + 1).to(BF) * 1e6
    pool.k.copy_((pool.k.float().abs() * 1e5).to(BF))
    best = [n // 3 for n in lens]
    for b, pos in enumerate(best):
        pool.k[pool.table[b][pos // 64], pos % 64] = 3e6
    for cache in (pool.cache(), widened(pool, 70000 // pool.page)):
        out, lse = cache.attend(q.cuda())
        for b, pos in enumerate(best):
            v = pool.v[pool.table[b][pos // 64], pos % 64]
            assert torch.equal(out[b].cpu(), v.repeat_interleave(2, 0))
            s = q[b].double().sum(1) * 3e6 * D ** -0.5  # 3e6 in bf16 is off by less than 2^-8
            assert ((lse[b].cpu().double() / s - 1).abs() < 2.0 ** -8).all()


def test_attend_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, pages at both ends."""
    page, Hkv = 256, 8
    per = page * Hkv * D
    n = (1 << 31) // per + 9
    free, _ = torch.cuda.mem_get_info()
    if free < 5 * n * per:
        pytest.skip("needs 21 GB")
    k, v = (torch.empty((n, page, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
    small = Pool("bshd", BF, 16, 8, page, 6, 3, [700, 513], seed=50)
    where = [0, n - 1, n - 2, 5, n - 3, n // 2]
    for i, w in enumerate(where):
        k[w], v[w] = small.k[i].cuda(), small.v[i].cuda()
    table = [[where[j] for j in row] for row in small.table]
    mean = torch.zeros((n, Hkv, D), device="cuda")
    cache = vsa.PagedCache("bshd", BF, 2, 16, 8, D, page, n, 3, k=k, v=v, k_mean=mean,
                           page_table=torch.tensor(table, dtype=torch.int32, device="cuda"),
                           seq_lens=torch.tensor(small.lens, dtype=torch.int32, device="cuda"))
    qkv, q, kn, vn = new_tokens(small, 2)
    q_out = cache.append(kn.cuda(), vn.cuda(), q.cuda())
    ref.append(small, kn, vn, q, [0, 1, 2])
    for i, w in enumerate(where):
        assert same(k[w], small.k[i]) and same(v[w], small.v[i])
    ref.check_attend(cache.attend(q_out), ref.attend(small, q))


# -------------------------------------------------------------- used together

def test_decode_steps_together_eager_and_captured():
    """Prompts appended, then steps of append, select and attend; the steps
    run eagerly and as one captured graph replayed, lengths advanced on the
    device, one row of the batch unused."""
    steps, topk, page = 40, 6, 16
    start = [100, 0, 31, 257]
    final = [n + steps if n else 0 for n in start]
    pool = Pool("bshd", BF, 8, 2, page, 64, 20, final, seed=60)
    pool.lens = list(start)
    cu = [0] + list(itertools.accumulate(start))
    qkv, q, k, v = new_tokens(pool, cu[-1])
    cos, sin = angles(512, 128)
    dc, ds = cos.cuda(), sin.cuda()
    eager, graph = pool.cache(), pool.cache()
    g = torch.Generator().manual_seed(61)
    tokens = torch.randn((steps, 4, 12, D), generator=g).to(BF)
    live = torch.tensor([1, 0, 1, 1], dtype=torch.int32, device="cuda")
    for c in (eager, graph):
        c.append(k.cuda(), v.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), cos=dc, sin=ds)
    ref.append(pool, k, v, None, cu, cos, sin)

    cur = torch.zeros((4, 12, D), dtype=BF, device="cuda")
    bufs = dict(q=torch.zeros((4, 8, D), dtype=BF, device="cuda"),
                idx=torch.zeros((4, 2, topk), dtype=torch.int32, device="cuda"),
                cnt=torch.zeros((4, 2), dtype=torch.int32, device="cuda"),
                out=torch.zeros((4, 8, D), dtype=BF, device="cuda"), lse=torch.zeros((4, 8), device="cuda"))

    def step(c, x, **kw):
        c.seq_lens.add_(live)
        qq, kk, vv = split(pool, x)
        qr = c.append(kk, vv, qq, cos=dc, sin=ds, q_out=kw.get("q"))
        pages = c.select(qr, topk, keep_first=1, keep_last=2, page_idx=kw.get("idx"), page_cnt=kw.get("cnt"))
        return (qr, *pages, *c.attend(qr, pages, out=kw.get("out"), lse=kw.get("lse")))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first launches outside the capture, on a state that is put back
        keep = [x.clone() for x in (graph.k, graph.v, graph.k_mean, graph.seq_lens)]
        step(graph, cur, **bufs)
        for x, y in zip((graph.k, graph.v, graph.k_mean, graph.seq_lens), keep):
            x.copy_(y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        step(graph, cur, **bufs)
    for s in range(steps):
        x = tokens[s]
        got = step(eager, x.cuda())
        cur.copy_(x)
        cg.replay()
        torch.cuda.synchronize()
        rows = torch.tensor([0, 2, 3])  # q_out of the unused row is not written
        assert same(got[0][rows.cuda()], bufs["q"][rows.cuda()])
        for a, b in zip(got[1:], (bufs["idx"], bufs["cnt"], bufs["out"], bufs["lse"])):
            assert same(a, b)
        pool.lens = [n + 1 if n else 0 for n in pool.lens]
        qq, kk, vv = split(pool, x)
        qr = ref.append(pool, kk, vv, qq, [0, 1, 2, 3, 4], cos, sin)
        assert torch.equal(got[0].cpu()[rows], qr[rows])
        qr[1] = 0
        want = ref.select(pool, qr, topk, 1, 2)
        assert torch.equal(got[1].cpu(), want[0]) and torch.equal(got[2].cpu(), want[1])
        if s % 8 == 0 or s == steps - 1:
            ref.check_attend(got[3:], ref.attend(pool, qr, want), f"step {s}")
    for a, b in ((eager.k, graph.k), (eager.v, graph.v), (eager.k_mean, graph.k_mean)):
        assert same(a, b)
    assert same(eager.k, pool.k) and same(eager.k_mean, pool.mean)


def test_layers_share_table_lengths_and_workspace_on_another_stream():
    pool, q = attend_pool(("bhsd", HF, 12, 3, 64, [500, 64, 3]), seed=70)
    other, _ = attend_pool(("bhsd", HF, 12, 3, 64, [500, 64, 3]), seed=71)
    other.table = pool.table
    a = pool.cache()
    b = other.cache(page_table=a.page_table, seq_lens=a.seq_lens, workspace=a.workspace)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dq = q.cuda()
    s.wait_stream(torch.cuda.current_stream())
    got = [c.attend(dq, stream=s) for c in (a, b, a)]
    picked = a.select(dq, 4, stream=s)
    listed = a.attend(dq, picked, stream=s)
    s.synchronize()
    for x, p in zip(got, (pool, other, pool)):
        ref.check_attend(x, ref.attend(p, q))
    ref.check_attend(listed, ref.attend(pool, q, [x.cpu() for x in picked]))


def test_graphs_that_share_a_workspace_and_streams_that_do_not():
    """Captured calls of two caches with one workspace, replayed in turns;
    then the two caches on two streams at once, each with its own."""
    case = ("bshd", BF, 8, 2, 32, RAGGED)
    pools = [attend_pool(case, seed=80 + i) for i in range(2)]
    first = widened(pools[0][0], 3000)
    shared = [first, widened(pools[1][0], 3000)]
    shared[1] = vsa.PagedCache("bshd", BF, len(RAGGED), 8, 2, D, 32, shared[1].num_pages, shared[1].max_pages,
                               k=shared[1].k, v=shared[1].v, k_mean=shared[1].k_mean, page_table=shared[1].page_table,
                               seq_lens=shared[1].seq_lens, workspace=first.workspace)
    qs = [q.cuda() for _, q in pools]
    want = [ref.attend(p, q) for p, q in pools]

    def run(c, q):
        pages = c.select(q, 20, keep_first=1)
        return (*pages, *c.attend(q, pages), *c.attend(q))

    eager = [run(c, q) for c, q in zip(shared, qs)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, q in zip(shared, qs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(c, q))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(a, b) for a, b in zip(eager[i], outs[i]))
        ref.check_attend(outs[i][4:], want[i], f"graph {i}")
    apart = [widened(p, 3000) for p, _ in pools]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append([])
        for c, q, s in zip(apart, qs, streams):
            with torch.cuda.stream(s):
                got[-1].append(run(c, q))
    torch.cuda.synchronize()
    for round_ in got:
        for i in range(2):
            assert all(same(a, b) for a, b in zip(eager[i], round_[i]))


def test_pages_of_a_shared_prefix():
    pool, q = attend_pool(("bshd", BF, 6, 2, 32, [100, 80, 64]), seed=72)
    pool.table[1][:2] = pool.table[0][:2]
    pool.table[2][:2] = pool.table[0][:2]
    ref.check_attend(pool.cache().attend(q.cuda()), ref.attend(pool, q))


def test_profile_names_and_launch_count():
    pool, q = attend_pool(("bshd", BF, 2, 2, 16, [100]), seed=73)
    cache = pool.cache()
    dq = q.cuda()
    n = vsa.vsa_launch_count()
    with vsa.profile() as pr:
        pages = cache.select(dq, 3)
        cache.attend(dq, pages)
        torch.cuda.synchronize()
    assert vsa.vsa_launch_count() - n == len(pr.records)
    assert {name for name, _ in pr.records} == {"page_select", "paged_attn"}
