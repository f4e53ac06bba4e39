"""The paged attention where numbers lie far apart: v scales of an 8-bit cache,
scores past the last bit of an exponent, queries and keys near the ends of
bf16's range, the largest entries under the largest scales."""
import pytest
import torch

from bwd_tile_mean_gb300 import vsa
from tests import paged8_ref as ref8
from tests import paged_ref as ref
from tests.paged8_ref import D, E4M3, Pool8
from tests.paged_ref import Pool, U
from tests.test_gpu_paged import BF, HF, attend_pool, widened
from tests.test_gpu_paged8 import pool_of, queries

pytestmark = pytest.mark.gpu


def share_pages(pool, B):
    """The pool's one sequence, B times over the same pages."""
    pool.table, pool.lens, pool.B = pool.table * B, pool.lens * B, B
    return pool


# ------------------------------------------------- v scales of 8 bits, far apart

def tail(Hq, Hkv, dtype, apart, B, n=9001):
    """Values of 1. Every 24 blocks: a strong key (score 0), then a block with
    scores of -60, a v scale 2^apart times the others' and dim 0 full, then
    a tail of equal keys (-7: together a third of the strong one)."""
    pool = Pool8("bshd", dtype, Hq, Hkv, 64, -(-n // 64) + 1, -(-n // 64), [n], seed=1)
    pool.k[:], pool.ks[:] = 0.0, 1.0
    pool.k[..., 0] = -7.0
    pool.v[:], pool.vs[:] = 64.0, 2.0 ** -6
    for blk in range(1, n // 16, 24):
        pool.k[pool.table[0][(blk - 1) // 4], 16 * ((blk - 1) % 4) + 5, :, 0] = 0.0
        p, i = pool.table[0][blk // 4], blk % 4
        at = slice(16 * i, 16 * i + 16)
        pool.k[p, at, :, 0] = -60.0
        pool.v[p, at] = 0.0
        pool.v[p, at, :, 0] = 448.0
        pool.vs[p, :, i] = 2.0 ** (apart - 6)
    q = torch.zeros(B, Hq, D, dtype=dtype)
    q[..., 0] = 1.0
    return share_pages(pool, B), q


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (24, 2)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("apart", [0, 6, 7, 16, 22, 25, 27, 29, 60])
def test_a_block_of_no_weight_takes_nothing_from_the_others(Hq, Hkv, dtype, apart):
    """A constant comes back as it is however large the scale of a block that
    is hardly attended: all weights together are 1 (they round alike: fp32
    sums, 2^-18, and e^-60 of the large block are what is left)."""
    pool, q = tail(Hq, Hkv, dtype, apart, 24)
    for wide in (0, 3000):
        table = torch.nn.functional.pad(torch.tensor(pool.table, dtype=torch.int32), (0, wide), value=-1).cuda()
        cache = pool.cache(scale=1.0) if not wide else vsa.PagedCache(
            pool.layout, dtype, pool.B, Hq, Hkv, D, 64, pool.num_pages, pool.max_pages + wide, k=pool.view(pool.k).cuda(),
            v=pool.view(pool.v).cuda(), k_scale=pool.ks.cuda(), v_scale=pool.vs.cuda(), page_table=table,
            seq_lens=torch.tensor(pool.lens, dtype=torch.int32).cuda(), kv_dtype=E4M3, scale=1.0)
        out = cache.attend(q.cuda())[0].double().cpu()
        assert ((out[..., 1:] - 1).abs() <= U[dtype] + 2.0 ** -18).all(), float((out[..., 1:] - 1).abs().max())


def by_products(pool, q, scale=None):
    """(out, bound) in fp64, the bound on what is lost in weights' products
    with the v scales relative to the largest product of a row: weights round
    to 11 bits, and where the product lies below 2^-20 of the largest to 2^-32 of
    that (2^-33 by rounding to nearest)."""
    want = ref8.attend(pool, q, scale=scale)
    out, tol = want[0], torch.zeros_like(want[0])
    scale, G = scale or D ** -0.5, pool.Hq // pool.Hkv
    for b in range(pool.B):
        for h in range(pool.Hkv):
            pages = [pool.table[b][j] for j in range(-(-pool.lens[b] // pool.page))]
            of = torch.cat([pool.vs[p, h].repeat_interleave(16) for p in pages])[: pool.lens[b]].double()
            k, v, _, _ = ref8.rows_of(pool, b, h, range(len(pages)))
            rows = slice(h * G, (h + 1) * G)
            qq = q[b, rows].double()
            s = qq @ k.T * scale
            p = torch.softmax(s, 1)
            mags = qq.abs() @ k.abs().T + 2.0 ** -15 * qq.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]
            ds = 132 * 2.0 ** -24 * scale * mags.amax(1) + 2.0 ** -22 * s.abs().amax(1)
            n = k.shape[0]
            rel = 2.0 ** -11 + 2 * ds + (8 + n / 16) * 2.0 ** -23
            tol[b, rows] = U[pool.dtype] * out[b, rows].abs() + rel[:, None] * (p @ v.abs()) * 1.01
            top = (p * of[None]).amax(1)
            units = (v / torch.where(of > 0, of, 1.0)[:, None]).abs().sum(0)  # e4m3 values
            tol[b, rows] += 2.0 ** -33 * top[:, None] * units[None]
    return out, tol


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (32, 2)])
@pytest.mark.parametrize("size", [0.5, 4.0, 12.0])
@pytest.mark.parametrize("lens", [[160], [5000, 77, 3000]])
def test_attend_by_products(Hq, Hkv, size, lens):
    """Scales up to 2^60 apart with weights as far apart, so that products of
    the two decide."""
    need = sum(-(-n // 16) for n in lens)
    pool = Pool8("bhsd", BF, Hq, Hkv, 16, need + 1, -(-max(lens) // 16), lens, seed=3)
    g = torch.Generator().manual_seed(4)
    q = queries(pool, size=size)
    for lo, hi in ((-30, 31), (-4, 5), (60, 120), (-120, -60)):
        pool.vs[:] = torch.exp2(torch.randint(lo, hi, pool.vs.shape, generator=g).float())
        out, tol = by_products(pool, q)
        got = pool.cache().attend(q.cuda())[0].double().cpu()
        assert torch.isfinite(got).all()
        assert ((got - out).abs() <= tol).all(), (lo, float(((got - out).abs() / tol).max()))


def test_weights_tiny_and_scales_huge():
    """Weights of 2^-100 of the largest whose values' scale is 2^110 times the
    others': their products are what the output is made of."""
    pool = Pool8("bshd", BF, 8, 1, 16, 40, 40, [640], seed=5)
    pool.k[:], pool.ks[:] = 0.0, 1.0
    pool.k[..., 0] = -72.0                      # 2^-103.9
    pool.k[pool.table[0][7], 3, 0, 0] = 0.0
    pool.v[:] = (pool.v / 4).to(E4M3).float()
    pool.vs[:] = 2.0 ** 110
    pool.vs[pool.table[0][7]] = 1.0
    q = torch.zeros(1, 8, D, dtype=BF)
    q[..., 0] = 1.0
    out, tol = by_products(pool, q, scale=1.0)
    got = pool.cache(scale=1.0).attend(q.cuda())[0].double().cpu()
    assert ((got - out).abs() <= tol).all(), float(((got - out).abs() / tol).max())


@pytest.mark.parametrize("Hq,small", [(1, -60), (1, -20), (12, -60)])
def test_scores_that_creep_up_behind_a_large_scale(Hq, small):
    """16,384 keys of scores that rise by 1/64 from block to block; every 330
    blocks one with a v scale of 2^100, the others with a small one: what the
    large ones add stays what outputs are relative to, for hundreds of steps
    whose maximum moves a little."""
    n, B = 16384, 400
    pool = Pool8("bshd", BF, Hq, 1, 64, n // 64, n // 64, [n], seed=2)
    g = torch.Generator().manual_seed(9)
    pool.k[:], pool.ks[:] = 0.0, 1.0
    pool.v[:] = (torch.randint(1, 16, pool.v.shape, generator=g) * 1.0)
    pool.vs[:] = 2.0 ** small
    for blk in range(n // 16):
        p, at = pool.table[0][blk // 4], slice(16 * (blk % 4), 16 * (blk % 4) + 16)
        pool.k[p, at, 0, 0], pool.k[p, at, 0, 1], pool.k[p, at, 0, 2] = blk // 64, blk // 4 % 16, blk % 4
        if blk % 330 == 5:
            pool.vs[p, 0, blk % 4] = 2.0 ** 100
    q = torch.zeros(1, Hq, D, dtype=BF)
    q[..., 0], q[..., 1], q[..., 2] = 1.0, 2.0 ** -4, 2.0 ** -6
    out, tol = by_products(pool, q, scale=1.0)
    share_pages(pool, B)
    got = pool.cache(scale=1.0).attend(q.expand(B, -1, -1).contiguous().cuda())[0].double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - out).abs() <= tol).all(), float(((got - out).abs() / tol).max())


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (32, 2)])
@pytest.mark.parametrize("apart", [2, 12])
def test_negative_scales_are_used_as_they_are(Hq, Hkv, apart):
    """Not what an append makes, but what a caller may give: the sign in the
    scale is the sign in the values, bit for bit."""
    pool = Pool8("bshd", BF, Hq, Hkv, 32, 60, 30, [900, 700], seed=7, spread=apart)
    q = queries(pool, size=3.0)
    want = pool.cache().attend(q.cuda())
    sign = torch.randint(0, 2, pool.vs.shape) * 2.0 - 1
    pool.vs = pool.vs * sign
    pool.v = pool.real(pool.v, sign)
    got = pool.cache().attend(q.cuda())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------- large scores

def plain_row(eight, n, seed=3, heads=2):
    """A cache of one head per query head whose keys are zero but for dims 0
    and 1, which q takes by 2^15 and 1: scores are whole numbers, exact in fp32."""
    kind = Pool8 if eight else Pool
    pool = kind("bshd", BF, heads, heads, 64, -(-n // 64) + 1, -(-n // 64), [n], seed=seed)
    pool.k[:] = 0.0
    if eight:
        pool.ks[:] = 1.0
    q = torch.zeros(1, heads, D, dtype=BF)
    q[..., 0], q[..., 1] = 2.0 ** 15, 1.0
    return pool, q


@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
@pytest.mark.parametrize("wide", [0, 3000], ids=["", "wide-table"])
def test_pieces_are_joined_by_exact_differences(eight, wide):
    """Two keys in different pieces of a row whose scores, 8,388,609 and
    8,388,610 and so on, differ by 1 and 2: by less than what their products
    with log2(e) are rounded by."""
    pool, q = plain_row(eight, 9001)
    at = lambda pos: (pool.table[0][pos // 64], pos % 64)  # noqa: E731
    for step, (near, far) in enumerate([(1, 2), (3, 5), (2, 1), (6, 7), (9, 8)]):
        pool.k[:] = 0.0
        for pos, x in ((70, near), (8100, far)):
            pool.k[at(pos)][:, 0], pool.k[at(pos)][:, 1] = 256.0, float(x)
        if eight:
            cache = vsa.PagedCache("bshd", BF, 1, 2, 2, D, 64, pool.num_pages, pool.max_pages + wide,
                                   k=pool.view(pool.k).cuda(), v=pool.view(pool.v).cuda(), k_scale=pool.ks.cuda(),
                                   v_scale=pool.vs.cuda(), kv_dtype=E4M3, scale=1.0)
        else:
            cache = vsa.PagedCache("bshd", BF, 1, 2, 2, D, 64, pool.num_pages, pool.max_pages + wide,
                                   k=pool.view(pool.k).cuda(), v=pool.view(pool.v).cuda(), scale=1.0)
        cache.page_table[:, : pool.max_pages] = torch.tensor(pool.table, dtype=torch.int32)
        cache.seq_lens.fill_(9001)
        out = cache.attend(q.cuda())[0][0].double().cpu()
        p = torch.softmax(torch.tensor([near, far], dtype=torch.float64), 0)
        v = [(pool.v[at(x)] * (pool.vs[at(x)[0], :, at(x)[1] // 16, None] if eight else 1.0)).double() for x in (70, 8100)]
        want = p[0] * v[0] + p[1] * v[1]
        # the weights' rounding to 16 bits, the output's, and fp32
        tol = (U[BF] + 2.0 ** -18) * (p[0] * v[0].abs() + p[1] * v[1].abs()) + U[BF] * want.abs()
        assert ((out - want).abs() <= tol).all(), (step, float(((out - want).abs() / tol).max()))


@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
@pytest.mark.parametrize("n", [40, 9001])
def test_the_largest_softmax_scale(eight, n):
    """A scale whose product with a score is beyond fp32 takes the largest
    score's value, whichever piece holds it."""
    pool, q = plain_row(eight, n)
    best = n // 3
    p, slot = pool.table[0][best // 64], best % 64
    pool.k[p, slot, :, 1] = 64.0
    out = pool.cache(scale=2.2e38).attend(q.cuda())[0][0].cpu()
    v = pool.v[p, slot].float() * (pool.vs[p, :, slot // 16, None] if eight else 1.0)
    assert torch.equal(out, v.to(BF))


def sums_of(weight):
    return weight.double().sum(-1).cpu()


@pytest.mark.parametrize("lens", [[40], [9001], [9001, 33, 5000]])
@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
def test_page_weights_of_the_largest_scores(lens, eight):
    """Scores of 1e13 and more: every row's weights are still 1 together, all
    of it on the page of its largest score."""
    if eight:
        pool = pool_of(("bhsd", BF, 4, 2, 64, lens, 0), garbage=False)
        q = (queries(pool).float().abs() + 1).to(BF) * 1e6
        pool.k, pool.ks[:] = pool.k.abs().clamp(max=120), 2.0 ** 13
        big, apart = 448.0, 1.0
    else:
        pool, q = attend_pool(("bhsd", BF, 4, 2, 64, lens), seed=45)
        q = (q.float().abs() + 1).to(BF) * 1e6
        pool.k.copy_((pool.k.float().abs() * 1e5).to(BF))
        big = 3e6
    best = [n // 3 for n in lens]
    for b, pos in enumerate(best):
        pool.k[pool.table[b][pos // 64], pos % 64] = big
    caches = [pool.cache(weigh=True)]
    if not eight:
        wide = widened(pool, 1000)
        caches.append(vsa.PagedCache("bhsd", BF, pool.B, 4, 2, D, 64, pool.num_pages, pool.max_pages + 1000, k=wide.k, v=wide.v,
                                     page_table=wide.page_table, seq_lens=wide.seq_lens, weigh=True))
    for cache in caches:
        every = torch.arange(cache.max_pages, dtype=torch.int32).expand(pool.B, 2, -1).contiguous().cuda()
        count = torch.tensor([[-(-n // 64)] * 2 for n in lens], dtype=torch.int32).cuda()
        for pages in (None, (every, count)):
            w = torch.zeros(pool.B, 2, cache.max_pages, device="cuda")
            cache.attend(q.cuda(), pages, page_weight=w)
            assert ((sums_of(w) - 2).abs() <= 2 * 2.0 ** -14).all()
            for b, pos in enumerate(best):
                assert ((w[b, :, pos // 64].cpu() - 2).abs() <= 2 * 2.0 ** -14).all()


@pytest.mark.parametrize("eight", [True, False], ids=["8", "16"])
@pytest.mark.parametrize("size", [30.0, 3e3, 3e5, 3e7])
@pytest.mark.parametrize("Hq,Hkv,lens", [(6, 3, [37, 4000]), (24, 2, [9001]), (8, 8, [3000, 0, 100])])
def test_weights_of_a_row_are_one(Hq, Hkv, lens, eight, size):
    """Random scores of any size: whatever their fp32 errors are, a row's
    weights are what its output is made with, 1 together."""
    pool = pool_of(("bshd", BF, Hq, Hkv, 32, lens, 1), eight, garbage=eight)
    q = queries(pool, size=size)
    cache = pool.cache(weigh=True)
    w = torch.zeros(pool.B, Hkv, cache.max_pages, device="cuda")
    cache.attend(q.cuda(), page_weight=w)
    want = torch.tensor([Hq / Hkv if n else 0.0 for n in lens], dtype=torch.float64)[:, None]
    assert ((sums_of(w) - want).abs() <= want * 2.0 ** -14).all(), float((sums_of(w) - want).abs().max())


# --------------------------------------------------- appends under large scales

@pytest.mark.parametrize("dtype,top", [(HF, 8), (BF, 120)])
@pytest.mark.parametrize("more", [0, 1, 6, 13, 14, 16, 17, 20])
def test_append_under_a_scale_larger_than_any_of_its_own(dtype, top, more):
    """A begun block whose scale (given with the cache) is 2^more times the
    largest that an append makes: the type's largest entry still reads back
    finite, as the nearest byte that stays within it."""
    if top + more > 127:
        pytest.skip("no such scale in fp32")
    scale, big = 2.0 ** (top + more), torch.finfo(dtype).max
    cache = vsa.PagedCache("bshd", dtype, 1, 2, 2, D, 16, 2, 2, kv_dtype=E4M3)
    cache.k_scale.fill_(scale), cache.v_scale.fill_(scale)
    cache.page_table.copy_(torch.tensor([[1, 0]], dtype=torch.int32))
    cache.seq_lens.fill_(6)
    x = torch.zeros(1, 2, D, dtype=dtype, device="cuda")
    x[..., 0], x[..., 1], x[..., 2] = big, -big, big / 2
    cache.append(x, x)
    assert (cache.k_scale[1] == scale).all() and (cache.v_scale[1] == scale).all()
    e4m3 = torch.arange(127, dtype=torch.uint8).view(E4M3).double() * scale
    e4m3 = e4m3[e4m3 <= big]
    for got in cache.read(1):
        got = got.double().cpu()[0]
        for d, want in ((0, big), (1, -big), (2, big / 2)):
            nearest = (e4m3 - abs(want)).abs().min()
            assert ((got[:, d].abs() - abs(want)).abs() == nearest).all() and torch.isfinite(got).all()
            assert (got[:, d] * want >= 0).all()


# --------------------------------------------- queries and keys near bf16's ends

def scaled(pool, q, k_by=0, q_by=0):
    pool.ks = pool.ks * 2.0 ** k_by
    return (q.double() * 2.0 ** q_by).to(q.dtype)


@pytest.mark.parametrize("heads", [(6, 3), (24, 2)])
@pytest.mark.parametrize("k_by,q_by,scale", [
    (0, -110, 2.0 ** -40), (0, -120, 2.0 ** -120), (0, -60, 1e-38),  # the softmax scale times q below fp32's least number
    (105, -105, 0.0), (112, -110, 0.0), (118, -118, 0.0), (112, -98, 2.0 ** -20),  # keys of 2^112 and more
    (-118, 118, 0.0), (-100, 60, 2.0 ** 40),
])
def test_attend_near_the_ends_of_the_range(heads, k_by, q_by, scale):
    Hq, Hkv = heads
    pool = pool_of(("bshd", BF, Hq, Hkv, 64, [900, 17], 1))
    q = scaled(pool, queries(pool), k_by, q_by)
    got = pool.cache(scale=scale).attend(q.cuda())
    ref.check_attend(got, ref8.attend(pool, q, scale=scale or None))


def test_zero_scores_of_large_queries_and_keys():
    """q of 2^120 against zeros in blocks of a scale of 2^30: scores of 0."""
    pool = Pool8("bshd", BF, 2, 1, 16, 3, 2, [32], seed=6)
    pool.k[..., 0], pool.ks[:] = 0.0, 2.0 ** 30
    q = torch.zeros(1, 2, D, dtype=BF)
    q[..., 0] = 2.0 ** 120
    out, lse = pool.cache().attend(q.cuda())
    want = ref8.attend(pool, q)
    ref.check_attend((out, lse), want)
