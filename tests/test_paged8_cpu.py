"""The 8-bit paged cache, page weights and eviction on a machine without a
GPU: refusals of both layers, and the references' own logic."""
import ctypes as C
import math

import pytest
import torch

from bwd_tile_mean_gb300 import build as libbuild
from bwd_tile_mean_gb300 import vsa
from tests import paged8_ref as ref8
from tests.test_paged_cpu import BAD_ARRAYS, BAD_DESC, FAKE, ODD, desc

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return vsa.lib()


def append(L, d=None, **kw):
    a = dict(T=2, k=FAKE, ks=0, v=FAKE, vs=0, q=FAKE, qs=0, q_out=FAKE, cu=None, pos=None, cos=FAKE, sin=FAKE,
             rows=9, rot=128, inter=0, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE, mean=FAKE)
    a.update(kw)
    return L.vsa_paged8_append(C.byref(d or desc()), *a.values(), None)


def attn(L, d=None, **kw):
    a = dict(q=FAKE, qs=0, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE, idx=None, cnt=None, cap=0, out=FAKE, lse=FAKE, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return L.vsa_paged8_attn(C.byref(d or desc()), *a.values(), None)


def weigh(L, d=None, **kw):
    a = dict(q=FAKE, qs=0, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE, idx=None, cnt=None, cap=0, out=FAKE, lse=FAKE, w=FAKE,
             wo=FAKE, decay=1.0, ws=FAKE, wsb=1 << 60)
    a.update(kw)
    return L.vsa_paged_attn_weigh(C.byref(d or desc()), *a.values(), None)


def read(L, d=None, **kw):
    a = dict(T=2, cu=None, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE, k=FAKE, v=FAKE)
    a.update(kw)
    return L.vsa_paged_read(C.byref(d or desc()), *a.values(), None)


def evict(L, d=None, **kw):
    a = dict(w=FAKE, keep=3, first=1, last=1, table=FAKE, lens=FAKE, wo=FAKE, freed=FAKE, cnt=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.vsa_page_evict(C.byref(d or desc()), *a.values(), None)


@pytest.mark.parametrize("bad,code", BAD_DESC + BAD_ARRAYS, ids=lambda x: str(x))
def test_descriptor_errors(L, bad, code):
    for call in (append, attn, weigh, read, evict):
        assert call(L, desc(**bad)) == code, call
    size = L.vsa_paged_weigh_workspace_size(C.byref(desc(**bad)))
    assert (size > 0) == ((bad, code) in BAD_ARRAYS)


def test_append_errors(L):
    for name in ("k", "v", "kc", "vc", "q", "q_out", "cos", "sin", "kscale", "vscale"):
        assert append(L, **{name: None}) == 1, name
    for name in ("k", "v", "q", "q_out", "kc", "vc", "mean", "cos", "sin", "cu", "pos", "kscale", "vscale"):
        assert append(L, **{name: ODD}) == 4, name
    assert append(L, desc(page_stride=64 * 2 * 128 + 8)) == 2    # bytes: a multiple of 16
    assert append(L, T=-1) == 2 and append(L, T=3) == 2 and append(L, rot=120) == 5 and append(L, rows=0) == 2
    assert append(L, T=0, cu=FAKE) == 0


def test_attention_errors(L):
    for call in (attn, weigh):
        for name in ("q", "kc", "vc", "out", "lse", "kscale", "vscale"):
            assert call(L, **{name: None}) == 1, name
            assert call(L, **{name: ODD}) == 4, name
        assert call(L, desc(page_stride=64 * 2 * 128 + 8)) == 2
        assert call(L, idx=FAKE, cap=3) == 1 and call(L, cnt=FAKE, cap=3) == 1
        assert call(L, idx=FAKE, cnt=FAKE, cap=0) == 2
        assert call(L, idx=ODD, cnt=FAKE, cap=3) == 4
        assert call(L, qs=12) == 2
        assert call(L, ws=None) == 7 and call(L, ws=C.c_void_p((1 << 20) + 128)) == 7
    assert attn(L, idx=FAKE, cnt=FAKE, cap=1 << 26) == 5
    assert weigh(L, idx=FAKE, cnt=FAKE, cap=5) == 5              # longer than the table
    plain, large = (f(C.byref(desc())) for f in (L.vsa_paged_workspace_size, L.vsa_paged_weigh_workspace_size))
    assert large == plain + 8 * 2 * 2 * 4 * (4 * 64 // 16)       # sums: B, Hkv, rows, blocks
    assert attn(L, wsb=plain - 1) == 7 and weigh(L, wsb=large - 1) == 7
    for name in ("w", "wo"):
        assert weigh(L, **{name: None}) == 1 and weigh(L, **{name: ODD}) == 4
    for decay in (-0.1, 1.5, math.nan, math.inf):
        assert weigh(L, decay=decay) == 2
    # 16 bits: no scales at all
    assert weigh(L, kscale=None, vscale=None, wsb=large - 1) == 7


def test_read_errors(L):
    for name in ("kc", "vc", "k", "v", "kscale", "vscale"):
        assert read(L, **{name: None}) == 1, name
        assert read(L, **{name: ODD}) == 4, name
    assert read(L, cu=ODD) == 4 and read(L, T=-1) == 2 and read(L, T=3) == 2
    assert read(L, desc(page_stride=64 * 2 * 128 + 8)) == 2
    assert read(L, T=0, cu=FAKE, k=None, v=None) == 0


def test_evict_errors(L):
    for name in ("w", "table", "lens", "wo", "freed", "cnt"):
        assert evict(L, **{name: None}) == 1, name
        assert evict(L, **{name: ODD}) == 4, name
    assert evict(L, first=-1) == 2 and evict(L, last=0) == 2 and evict(L, keep=1) == 2 and evict(L, keep=0, first=0) == 2
    assert evict(L, keep=2 ** 31 - 1, first=2 ** 31 - 1, last=2 ** 31 - 1) == 2
    need = L.vsa_paged_workspace_size(C.byref(desc()))
    assert evict(L, wsb=need - 1) == 7 and evict(L, ws=None) == 7 and evict(L, ws=C.c_void_p((1 << 20) + 128)) == 7


def cache(**kw):
    a = dict(layout="bshd", dtype=torch.bfloat16, B=2, Hq=4, Hkv=2, D=128, page=32, num_pages=5, max_pages=3,
             device="cpu", kv_dtype=E4M3)
    a.update(kw)
    return vsa.PagedCache(**a)


def test_cache_refuses_bad_tensors(L):
    good = torch.zeros(5, 32, 2, 128, dtype=E4M3)
    one = torch.ones(5, 2, 2)
    c = cache(k=good, v=good.clone(), k_scale=one, v_scale=one.clone())
    assert c.k_scale is one and c.kv_dtype == E4M3 and c.dtype == torch.bfloat16
    assert cache().k_scale.shape == (5, 2, 2) and cache(allocate=False).k is None
    half = torch.zeros(5, 32, 2, 128, dtype=torch.bfloat16)
    for kw in (dict(kv_dtype=torch.float8_e5m2), dict(kv_dtype=torch.float16), dict(k=good, v=good.clone()),
               dict(k=half, v=half.clone(), k_scale=one, v_scale=one.clone()),
               dict(k=good, v=good.clone(), k_scale=one), dict(k=good, v=good.clone(), k_scale=one.half(), v_scale=one),
               dict(k=good, v=good.clone(), k_scale=one[:, :1], v_scale=one.clone()),
               dict(k=good, v=good.clone(), k_scale=one.transpose(1, 2), v_scale=one.clone()),
               dict(k=good, v=good.clone(), k_scale=one, v_scale=one),           # shared
               dict(k=good, v=good.clone(), k_scale=good.view(-1).view(torch.float32)[:20].view(5, 2, 2), v_scale=one),
               dict(allocate=False, k_scale=one, v_scale=one.clone()),
               dict(kv_dtype=None, k_scale=one, v_scale=one.clone()), dict(kv_dtype=None, k=good, v=good.clone()),
               dict(k=torch.zeros(5, 32 * 2 * 128 + 8, dtype=E4M3)[:, :32 * 2 * 128].view(5, 32, 2, 128),
                    v=torch.zeros(5, 32 * 2 * 128 + 8, dtype=E4M3)[:, :32 * 2 * 128].view(5, 32, 2, 128),
                    k_scale=one, v_scale=one.clone())):                             # pages 8 bytes off
        with pytest.raises(ValueError):
            cache(**kw)


@pytest.mark.parametrize("kv", [E4M3, None])
def test_calls_refuse_bad_tensors(L, kv):
    c = cache(kv_dtype=kv, weigh=True)
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    k, q = torch.zeros(2, 2, 128, **bf), torch.zeros(2, 4, 128, **bf)
    w, w2 = torch.zeros(2, 2, 3), torch.zeros(2, 2, 3)
    idx, cnt = torch.zeros(2, 2, 2, **i32), torch.zeros(2, 2, **i32)
    kk, wide = torch.zeros(7, 2, 128, **bf), torch.zeros(13)
    out = (c.page_table.clone(), c.seq_lens.clone(), w2)
    for match, call in (
            ("page_weight", lambda: c.attend(q, page_weight=w[:1])),
            ("page_weight", lambda: c.attend(q, page_weight=w.double())),
            ("contiguous", lambda: c.attend(q, page_weight=torch.zeros(2, 3, 2).transpose(1, 2))),
            ("weight_out", lambda: c.attend(q, page_weight=w, weight_out=w2[:1])),
            ("belong to", lambda: c.attend(q, weight_out=w2)),
            ("belong to", lambda: c.attend(q, decay=0.5)),
            ("decay", lambda: c.attend(q, page_weight=w, decay=1.5)),
            ("decay", lambda: c.attend(q, page_weight=w, decay=math.nan)),
            ("no longer than the table", lambda: c.attend(q, (torch.zeros(2, 2, 4, **i32), cnt), page_weight=w)),
            ("weigh=True", lambda: cache(kv_dtype=kv).attend(q, page_weight=w)),
            ("with page_weight", lambda: c.attend(q, lse=w.view(-1)[2:10].view(2, 4), page_weight=w, weight_out=w2)),
            ("with weight_out", lambda: c.attend(q, lse=w.view(-1)[2:10].view(2, 4), page_weight=w)),
            ("with page_weight", lambda: c.attend(q, page_weight=wide[:12].view(2, 2, 3), weight_out=wide[1:].view(2, 2, 3))),
            ("gradient", lambda: c.attend(q, page_weight=w.clone().requires_grad_())),
            ("tokens", lambda: c.read(-1)),
            ("one token per sequence", lambda: c.read(3)),
            ("cu_seqlens", lambda: c.read(3, cu_seqlens=torch.zeros(2, **i32))),
            ("k_out", lambda: c.read(2, k_out=k[:1])),
            ("shares memory", lambda: c.read(2, k_out=kk[:2], v_out=kk[1:3])),
            ("shares memory", lambda: c.read(2, k_out=c.k.view(-1).view(torch.bfloat16)[:512].view(2, 2, 128))),
            ("no k and v", lambda: cache(kv_dtype=kv, allocate=False).read(2)),
            ("page_weight", lambda: c.evict(w[:1], 2)),
            ("keep", lambda: c.evict(w, 0)),
            ("keep", lambda: c.evict(w, 2, keep_first=2)),
            ("keep", lambda: c.evict(w, 2, keep_first=-1)),
            ("keep", lambda: c.evict(w, 2, keep_last=0)),
            ("freed", lambda: c.evict(w, 2, freed=torch.zeros(2, 2, **i32))),
            ("freed_cnt", lambda: c.evict(w, 2, freed_cnt=torch.zeros(3, **i32))),
            ("out: expected", lambda: c.evict(w, 2, out=out[:2])),
            ("out: page_table", lambda: c.evict(w, 2, out=(out[0][:, :2], out[1], out[2]))),
            ("out: seq_lens", lambda: c.evict(w, 2, out=(out[0], out[1].long(), out[2]))),
            ("shares memory", lambda: c.evict(w, 2, out=(out[0], c.page_table.view(-1)[:2], out[2]))),
            ("shares memory", lambda: c.evict(w, 2, freed=c.page_table.view(-1)[1:3].view(2, 1))),
            ("shares memory", lambda: c.evict(w, 2, freed_cnt=c.seq_lens)),
            ("shares memory", lambda: c.evict(c.workspace[:48].view(torch.float32).view(2, 2, 3), 2)),
            ("shares memory", lambda: c.evict(c.workspace[:48].view(torch.float32).view(2, 2, 3), 2, out=out)),
            ("shares memory", lambda: c.attend(q, page_weight=c.workspace[-48:].view(torch.float32).view(2, 2, 3),
                                               weight_out=w2)),
            ("gradient", lambda: c.evict(w.clone().requires_grad_(), 2))):
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: c.append(k, k), lambda: c.select(q, 2), lambda: c.attend(q),
                 lambda: c.attend(q, (idx, cnt), page_weight=w),
                 lambda: c.attend(q, page_weight=w, weight_out=w2, decay=0.5), lambda: c.read(2), lambda: c.evict(w, 2),
                 lambda: c.evict(w, 5, out=out), lambda: cache(kv_dtype=kv, allocate=False).evict(w, 2)):
        with pytest.raises(ValueError, match="GPU only"):
            call()
    with pytest.raises(ValueError, match="gradient"):
        c.append(k.clone().requires_grad_(), k)
    if kv:
        with pytest.raises(ValueError, match="with the cache's k_scale"):
            c.attend(q, lse=c.k_scale.view(-1)[:8].view(2, 4))
        with pytest.raises(ValueError, match="shares memory"):
            c.append(k, k, q, cos=c.v_scale.view(-1)[:16].view(2, 8), sin=torch.zeros(2, 8))


def test_workspaces_of_a_size_serve_both(L):
    c = cache(weigh=True)
    need, plain = (f(C.byref(c.desc)) for f in (L.vsa_paged_weigh_workspace_size, L.vsa_paged_workspace_size))
    assert c.workspace.numel() == need > plain == cache().workspace.numel()
    w, q = torch.zeros(2, 2, 3), torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU only"):
        cache(workspace=torch.zeros(need + 5, dtype=torch.uint8)).attend(q, page_weight=w)
    with pytest.raises(ValueError, match="too small"):
        cache(workspace=torch.zeros(need - 1, dtype=torch.uint8)).attend(q, page_weight=w)
    with pytest.raises(ValueError, match="workspace"):
        cache(workspace=torch.zeros(need - 1, dtype=torch.uint8), weigh=True)


def test_reference_scales():
    for top, want in ((448.0, 1.0), (448.1, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7),
                      (0.0, 2.0 ** -126),
                      (1e-40, 2.0 ** -126), (3.3e38, 2.0 ** 120), (57344.0, 128.0), (65504.0, 256.0)):
        assert ref8.scale_of(top) == want, top
    x = torch.tensor([65504.0, -61440.0, 65520.0, math.inf, math.nan])
    assert ref8.as_bytes(x, 256.0, torch.float16).tolist()[:2] == [240.0, -240.0]
    assert torch.isnan(ref8.as_bytes(x, 256.0, torch.float16)).tolist() == [False, False, True, True, True]
    assert torch.isnan(ref8.as_bytes(x, 256.0, torch.bfloat16)).tolist() == [False, False, False, True, True]


def test_reference_evict_on_a_case_by_hand():
    w = torch.tensor([[[5.0, 1.0, 3.0, 1.0, 9.0, 0.0, 7.0]], [[1.0] * 7]])
    table, lens, weight, freed, cnt = ref8.evict([[10, 11, 12, 13, 14, 15, -7], [20, 21, 22, 23, -7, -7, -7]], [16 * 5 + 1, 60],
                                                 w, 16, 4, 1, 1)
    assert table == [[10, 12, 14, 15, -7, -1, -1], [20, 21, 22, 23, -7, -7, -7]] and lens == [16 * 3 + 1, 60]
    assert weight[0, 0].tolist() == [5.0, 3.0, 9.0, 0.0, 7.0, 0.0, 0.0]
    assert freed.tolist() == [[11, 13, -1], [-1, -1, -1]] and cnt.tolist() == [2, 0]
    assert ref8.evict([[10, 11, 12]], [48], torch.ones(1, 1, 3), 16, 2, 0, 1)[0] == [[10, 12, -1]]  # equals: the lower stays
