"""Paged-cache calls on a machine without a GPU: every bad argument is
refused on the host, before any CUDA call, and the references' own logic."""
import ctypes as C

import pytest
import torch

from bwd_tile_mean_gb300 import build as libbuild
from bwd_tile_mean_gb300 import vsa
from tests import paged_ref as ref

# aligned and never dereferenced: every call fails host validation
FAKE = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return vsa.lib()


def desc(**kw):
    d = dict(layout=1, dtype=0, B=2, Hq=8, Hkv=2, D=128, page=64, num_pages=10, max_pages=4, page_stride=0,
             page_table=1 << 20, seq_lens=1 << 20, scale=0.0)
    d.update(kw)
    return vsa.PagedDesc(*[d[f] for f, _ in vsa.PagedDesc._fields_])


BAD_DESC = [(dict(layout=2), 4), (dict(layout=-1), 4), (dict(dtype=2), 3), (dict(B=0), 2), (dict(Hq=7), 2),
            (dict(Hkv=0), 2), (dict(Hq=65537, Hkv=65537), 5), (dict(D=64), 5), (dict(page=48), 5),
            (dict(page=8), 5), (dict(page=512), 5),
            (dict(num_pages=0), 2), (dict(max_pages=0), 2), (dict(max_pages=1 << 25), 5),
            (dict(page_stride=64 * 2 * 128 - 8), 2), (dict(page_stride=64 * 2 * 128 + 4), 2),
            (dict(scale=-1.0), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2)]
BAD_ARRAYS = [(dict(page_table=None), 1), (dict(seq_lens=None), 1), (dict(seq_lens=(1 << 20) + 2), 4)]


def append(L, d=None, **kw):
    a = dict(T=2, k=FAKE, ks=0, v=FAKE, vs=0, q=FAKE, qs=0, q_out=FAKE, cu=None, pos=None, cos=FAKE, sin=FAKE,
             rows=9, rot=128, inter=0, kc=FAKE, vc=FAKE, mean=FAKE)
    a.update(kw)
    return L.vsa_paged_append(C.byref(d or desc()), *a.values(), None)


def select(L, d=None, **kw):
    a = dict(q=FAKE, qs=0, mean=FAKE, topk=2, first=0, last=1, idx=FAKE, cnt=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.vsa_page_select(C.byref(d or desc()), *a.values(), None)


def attn(L, d=None, **kw):
    a = dict(q=FAKE, qs=0, kc=FAKE, vc=FAKE, idx=None, cnt=None, cap=0, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.vsa_paged_attn(C.byref(d or desc()), *a.values(), None)


@pytest.mark.parametrize("bad,code", BAD_DESC + BAD_ARRAYS, ids=lambda x: str(x))
def test_descriptor_errors(L, bad, code):
    assert append(L, desc(**bad)) == code
    assert select(L, desc(**bad)) == code
    assert attn(L, desc(**bad)) == code
    size = L.vsa_paged_workspace_size(C.byref(desc(**bad)))
    assert (size > 0) == ((bad, code) in BAD_ARRAYS)  # the size needs no arrays
    assert L.vsa_paged_attn(None, FAKE, 0, FAKE, FAKE, None, None, 0, FAKE, FAKE, FAKE, 1 << 40, None) == 1


def test_append_errors(L):
    for name in ("k", "v", "kc", "vc", "q", "q_out", "cos", "sin"):
        assert append(L, **{name: None}) == 1, name
    for name in ("k", "v", "q", "q_out", "kc", "vc", "mean", "cos", "sin", "cu", "pos"):
        assert append(L, **{name: ODD}) == 4, name
    assert append(L, T=-1) == 2
    assert append(L, T=3) == 2                       # T != B without offsets
    assert append(L, ks=2 * 128 - 8) == 2            # tokens that overlap
    assert append(L, vs=2 * 128 + 4) == 2            # not a multiple of 8
    assert append(L, qs=-1024) == 2
    assert append(L, rot=120) == 5
    assert append(L, rot=144) == 5
    assert append(L, rot=-16) == 5
    assert append(L, rows=0) == 2
    assert append(L, T=0, cu=FAKE) == 0              # nothing to do, nothing launched


def test_select_errors(L):
    for name in ("q", "mean", "idx", "cnt"):
        assert select(L, **{name: None}) == 1, name
        assert select(L, **{name: ODD}) == 4, name
    assert select(L, topk=0) == 2
    assert select(L, first=-1) == 2
    assert select(L, last=0) == 2
    assert select(L, topk=2, first=2) == 2
    assert select(L, topk=3, first=2, last=2) == 2
    assert select(L, first=2 ** 31 - 1, last=2 ** 31 - 1) == 2
    assert select(L, qs=8) == 2
    need = L.vsa_paged_workspace_size(C.byref(desc()))
    assert select(L, wsb=need - 1) == 7 and select(L, ws=None) == 7 and select(L, ws=C.c_void_p((1 << 20) + 128)) == 7


def test_attend_errors(L):
    for name in ("q", "kc", "vc", "out", "lse"):
        assert attn(L, **{name: None}) == 1, name
        assert attn(L, **{name: ODD}) == 4, name
    assert attn(L, idx=FAKE, cap=3) == 1 and attn(L, cnt=FAKE, cap=3) == 1
    assert attn(L, idx=FAKE, cnt=FAKE, cap=0) == 2
    assert attn(L, idx=FAKE, cnt=FAKE, cap=1 << 26) == 5
    assert attn(L, idx=ODD, cnt=FAKE, cap=3) == 4
    assert attn(L, qs=12) == 2
    need = L.vsa_paged_workspace_size(C.byref(desc()))
    assert attn(L, wsb=need - 1) == 7 and attn(L, ws=None) == 7 and attn(L, ws=C.c_void_p((1 << 20) + 128)) == 7


def test_workspace_grows_with_the_problem(L):
    size = lambda **kw: L.vsa_paged_workspace_size(C.byref(desc(**kw)))  # noqa: E731
    assert size(max_pages=4000) > size()
    assert size(Hq=32) > size()
    assert size(B=300) > size()


def cache(**kw):
    a = dict(layout="bshd", dtype=torch.bfloat16, B=2, Hq=4, Hkv=2, D=128, page=16, num_pages=5, max_pages=3,
             device="cpu")
    a.update(kw)
    return vsa.PagedCache(**a)


def test_cache_refuses_bad_tensors(L):
    good = torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)
    cache(k=good, v=good)
    for kw in (dict(layout="tnd"), dict(dtype=torch.float32), dict(D=64), dict(page=48), dict(Hq=3),
               dict(k=good), dict(v=good), dict(k=good.half(), v=good), dict(k=good[:4], v=good),
               dict(k=good.transpose(1, 2), v=good), dict(k=torch.zeros(5, 16, 4, 128, dtype=good.dtype)[:, :, ::2], v=good),
               dict(k=torch.zeros(5, 2, 16, 2, 128, dtype=good.dtype)[:, 0], v=good),  # strides differ
               dict(seq_lens=torch.zeros(2)), dict(seq_lens=torch.zeros(3, dtype=torch.int32)),
               dict(page_table=torch.zeros(2, 4, dtype=torch.int32)),
               dict(page_table=torch.zeros(2, 6, dtype=torch.int32)[:, ::2]),
               dict(k_mean=torch.zeros(5, 2, 128, dtype=torch.bfloat16)), dict(workspace=torch.zeros(16))):
        with pytest.raises(ValueError):
            cache(**kw)


def test_calls_refuse_bad_tensors(L):
    c = cache()
    with pytest.raises(AttributeError):
        c.k = c.v  # the calls pass on the address they were made with
    bf = dict(dtype=torch.bfloat16)
    k, q = torch.zeros(2, 2, 128, **bf), torch.zeros(2, 4, 128, **bf)
    t = torch.zeros(9, 64)
    i32 = dict(dtype=torch.int32)
    for args, kw in (((k, k[:1]), {}), ((k, k, q[:1]), {}), ((k.half(), k), {}), ((k, k[:, :1]), {}),
                     ((k, k.transpose(1, 2)), {}), ((torch.zeros(3, 2, 128, **bf),) * 2, {}),
                     ((k, k), dict(cos=t)), ((k, k), dict(cos=t, sin=t[:8])), ((k, k), dict(cos=t.double(), sin=t)),
                     ((k, k), dict(cos=t.t(), sin=t.t())), ((k, k), dict(q_out=q)),
                     ((k, k, q), dict(q_out=q[:1])), ((k, k, q), dict(q_out=q)),
                     ((k, k), dict(cu_seqlens=torch.zeros(2, **i32))), ((k, k), dict(cu_seqlens=torch.zeros(3))),
                     ((k, k), dict(positions=torch.zeros(2))), ((k, k), dict(positions=torch.zeros(3, **i32)))):
        with pytest.raises(ValueError):
            c.append(*args, **kw)
    idx, cnt = torch.zeros(2, 2, 2, **i32), torch.zeros(2, 2, **i32)
    for call in (lambda: c.select(q[:1], 2), lambda: c.select(q.half(), 2), lambda: c.select(q, 3, page_idx=idx),
                 lambda: c.attend(k), lambda: c.attend(q, (idx, cnt[:1])), lambda: c.attend(q, (idx.long(), cnt)),
                 lambda: c.attend(q, (idx[:, :, ::2], cnt)), lambda: c.attend(q, out=q.half()),
                 lambda: c.attend(q, lse=torch.zeros(2, 3)), lambda: cache(k_mean=False).select(q, 2),
                 lambda: cache(allocate=False).attend(q), lambda: cache(allocate=False).append(k, k)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.append(k, k), lambda: c.select(q, 2), lambda: c.attend(q)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


def test_broadcast_tensors_are_refused(L):
    """An expanded tensor has the stride 0, which the C calls take for dense:
    its storage ends before the rows they would then read."""
    bf = dict(dtype=torch.bfloat16)
    one, pages = torch.zeros(1, 16, 2, 128, **bf).expand(5, -1, -1, -1), torch.zeros(5, 16, 2, 128, **bf)
    for kw in (dict(k=one, v=one), dict(k=one, v=pages), dict(k=pages, v=one),
               dict(k=pages.as_strided(pages.shape, (8, 256, 128, 1)), v=pages),
               dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 28))):
        with pytest.raises(ValueError):
            cache(**kw)
    c = cache()
    k, q = torch.zeros(2, 2, 128, **bf), torch.zeros(2, 4, 128, **bf)
    k1, q1 = k[:1].expand(2, -1, -1), q[:1].expand(2, -1, -1)
    for call in (lambda: c.append(k1, k), lambda: c.append(k, k1), lambda: c.append(k, k, q1), lambda: c.select(q1, 2),
                 lambda: c.attend(q1), lambda: c.append(k.as_strided(k.shape, (128, 128, 1)), k)):
        with pytest.raises(ValueError, match="share memory"):
            call()
    with pytest.raises(ValueError, match="must not be q"):
        c.attend(q, out=q)


def test_reference_select_and_attend_on_a_case_by_hand():
    pool = ref.Pool("bshd", torch.bfloat16, 1, 1, 16, 6, 6, [16 * 4 + 3], seed=1)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    q[0, 0, 0] = 1.0
    for j, value in enumerate((1.0, 3.0, 2.0, 3.0)):
        pool.mean[pool.table[0][j]] = value
    idx, cnt = ref.select(pool, q, 3, 0, 1)
    assert idx.tolist() == [[[1, 3, 4]]] and cnt.tolist() == [[3]]
    idx, cnt = ref.select(pool, q, 2, 0, 1)
    assert idx.tolist() == [[[1, 4]]]                # of equal scores the lower page
    q.zero_()
    out, lse, _, _ = ref.attend(pool, q, (idx, cnt))
    keys = [pool.v[pool.table[0][1]][:, 0].double(), pool.v[pool.table[0][4]][:3, 0].double()]
    assert torch.allclose(out[0, 0], torch.cat(keys).mean(0))
    assert abs(float(lse[0, 0]) - torch.log(torch.tensor(19.0)).item()) < 1e-6


def test_select_refuses_more_entries_than_a_list_can_have(L):
    """topk entries are written in steps of a CTA's threads, counted in 32
    bits; vsa_paged_attn takes lists of the same lengths."""
    for page in (16, 256):
        most = (2 ** 31 - 1) // page
        need = L.vsa_paged_workspace_size(C.byref(desc(page=page)))
        assert select(L, desc(page=page), topk=most + 1) == 5
        assert select(L, desc(page=page), topk=2 ** 31 - 1) == 5
        assert select(L, desc(page=page), topk=most, wsb=need - 1) == 7  # gets as far as the workspace
        assert attn(L, desc(page=page), idx=FAKE, cnt=FAKE, cap=most + 1) == 5
        assert attn(L, desc(page=page), idx=FAKE, cnt=FAKE, cap=most, wsb=need - 1) == 7


def test_outputs_that_share_memory_are_refused(L):
    """What a call writes may be no memory that it reads: the kernel's CTAs
    read and write in no set order."""
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    good = torch.zeros(5, 16, 2, 128, **bf)
    ahead = torch.zeros(6, 16, 2, 128, **bf)
    arena = torch.zeros(1 << 23, dtype=torch.uint8)
    kk = torch.zeros(2, 2, 128, **bf)
    for kv in (dict(k=good, v=good), dict(k=ahead[:5], v=ahead[1:]),
               dict(k=ahead.view(-1)[:20480].view(good.shape), v=ahead.view(-1)[8:20488].view(good.shape))):
        with pytest.raises(ValueError, match="k and v share memory"):  # good to attend to
            cache(**kv).append(kk, kk)
    for kw in (dict(k=good, v=good.clone(), k_mean=good.view(torch.float32).view(-1)[:1280].view(5, 2, 128)),
               dict(k_mean=arena[:5120].view(torch.float32).view(5, 2, 128), workspace=arena),
               dict(seq_lens=arena[4096:4104].view(torch.int32), workspace=arena)):
        with pytest.raises(ValueError, match="shares memory"):
            cache(**kw)
    both = torch.zeros(5, 2, 16, 2, 128, **bf)       # halves of one buffer lie apart
    three = torch.zeros(5, 3, 16, 2, 128, **bf)
    for pair in ((both[:, 0], both[:, 1]), (both[:, 1], both[:, 0]), (three[:, 2], three[:, 0]), (three[:, 1], three[:, 2]),
                 (both.view(10, 16, 2, 128)[:5], both.view(10, 16, 2, 128)[5:])):
        c = cache(k=pair[0], v=pair[1])
        with pytest.raises(ValueError, match="GPU only"):
            c.append(kk, kk)
    need = L.vsa_paged_workspace_size(C.byref(c.desc))  # an arena's first bytes, whatever lies behind them
    big = torch.zeros(need + 64, dtype=torch.uint8)
    cache(workspace=big, seq_lens=big[need:need + 8].view(torch.int32))

    c = cache(k=both[:, 0], v=both[:, 1])
    qkv = torch.zeros(2 * 8 + 4, 128, **bf)           # room for two tokens and a shifted view
    rows = qkv[:16].view(2, 8, 128)
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    dense = torch.zeros(13, 128, **bf)
    dq = dense[:8].view(2, 4, 128)
    idx, cnt = torch.zeros(2, 2, 3, **i32), torch.zeros(2, 2, **i32)
    lists = torch.zeros(16, **i32)
    words = lambda t: t.view(-1).view(torch.int32)  # noqa: E731
    for call, why in ((lambda: c.append(k, v, q, q_out=qkv[4:12].view(2, 4, 128)), "shares memory with"),
                      (lambda: c.append(k, v, q, q_out=qkv[9:17].view(2, 4, 128)), "shares memory with"),
                      (lambda: c.append(kk, kk, dq, q_out=dense[4:12].view(2, 4, 128)), "with q"),
                      (lambda: c.append(kk, kk, dq, q_out=both[4, 1, 12:].view(2, 4, 128)), "with the cache's v"),
                      (lambda: c.append(both[3, 0, :2], kk), "with k"),
                      (lambda: c.append(kk, both[3, 1, 4:6]), "with v"),
                      (lambda: c.select(dq, 3, page_idx=lists[:12].view(2, 2, 3), page_cnt=lists[11:15].view(2, 2)),
                       "with page_cnt"),
                      (lambda: c.select(dq, 3, page_idx=words(dense)[:12].view(2, 2, 3)), "with q"),
                      (lambda: c.select(dq, 3, page_cnt=c.page_table.view(-1)[:4].view(2, 2)), "with page_table"),
                      (lambda: c.attend(dq, out=dense[1:9].view(2, 4, 128)), "with q"),
                      (lambda: c.attend(dq, out=both[0, 0, :4].view(2, 4, 128)), "with the cache's k"),
                      (lambda: c.attend(dq, (idx, cnt), lse=idx.view(-1)[2:10].view(torch.float32).view(2, 4)), "page_idx"),
                      (lambda: c.attend(dq, lse=c.workspace[64:96].view(torch.float32).view(2, 4)), "workspace"),
                      (lambda: c.attend(dq, lse=words(dense)[480:488].view(torch.float32).view(2, 4)), "with q")):
        with pytest.raises(ValueError, match=why):
            call()
    # apart: parts of one projection's output, neighbouring memory, a gap between rows
    wide = torch.zeros(2, 24, 128, **bf)
    for call in (lambda: c.append(k, v, q, q_out=torch.zeros(2, 4, 128, **bf)),
                 lambda: c.append(kk, kk, wide[:, :4], q_out=wide[0, 4:12].view(2, 4, 128)),
                 lambda: c.append(kk, kk, wide[:, 20:], q_out=wide[1, 12:20].view(2, 4, 128)),
                 lambda: c.attend(wide[:, 2:6], out=wide[0, 6:14].view(2, 4, 128)),
                 lambda: c.attend(dense[5:].view(2, 4, 128), lse=words(dense)[312:320].view(torch.float32).view(2, 4))):
        with pytest.raises(ValueError, match="GPU only"):
            call()


def test_inputs_that_want_a_gradient_are_refused(L):
    """The calls give none: outputs without a history would look trained."""
    c = cache()
    bf = dict(dtype=torch.bfloat16)
    k, q = torch.zeros(2, 2, 128, **bf), torch.zeros(2, 4, 128, **bf)
    gk, gq = (torch.zeros_like(t, requires_grad=True) for t in (k, q))
    calls = (lambda: c.append(gk, k), lambda: c.append(k, gk), lambda: c.append(k, k, gq), lambda: c.select(gq, 2),
             lambda: c.attend(gq))
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call()
        for off in (torch.no_grad, torch.inference_mode):
            with off(), pytest.raises(ValueError, match="GPU only"):
                call()
    with pytest.raises(ValueError, match="no gradient"):
        c.append(k, k, cos=torch.zeros(9, 64, requires_grad=True), sin=torch.zeros(9, 64))
    with pytest.raises(ValueError, match="no gradient"):
        c.attend(q, out=torch.zeros_like(q, requires_grad=True))
    with pytest.raises(ValueError, match="GPU only"):
        c.attend(gq.detach())
    pages = [torch.zeros(5, 16, 2, 128, **bf, requires_grad=True) for _ in range(2)]
    with pytest.raises(ValueError, match="no gradient"):
        cache(k=pages[0], v=pages[1])
    with torch.no_grad():
        cache(k=pages[0], v=pages[1])


def test_binding_belongs_to_this_python_and_torch(L, monkeypatch):
    """The binding unpacks torch's own C++ objects: another torch or another
    Python on the same tree has one of its own, whatever the files' dates."""
    import os
    here = libbuild.binding()
    assert os.path.exists(here) and os.path.samefile(vsa._paged_binding().__file__, here)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    other = libbuild.binding()
    assert other != here
    monkeypatch.setattr(vsa, "_binding", None)
    with pytest.raises(RuntimeError, match="not built"):
        vsa._paged_binding()
    monkeypatch.undo()
    assert libbuild.binding() == here
    import sysconfig
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-0" if n == "SOABI" else get(n))
    assert libbuild.binding() not in (here, other)


def test_cache_refuses_sizes_past_32_bits(L):
    """The C descriptor holds 32-bit sizes; ctypes would keep the low bits."""
    for name in ("B", "Hq", "Hkv", "D", "page", "num_pages", "max_pages"):
        for past in (2 ** 32, -2 ** 32):
            good = dict(B=2, Hq=4, Hkv=2, D=128, page=16, num_pages=5, max_pages=3)
            tables = dict(page_table=torch.zeros(2, 3, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32))
            with pytest.raises(ValueError, match=name):
                cache(allocate=False, **tables, **{**good, name: good[name] + past})
    with pytest.raises(ValueError, match="num_pages"):
        cache(allocate=False, num_pages=2 ** 32 + 5)


@pytest.mark.parametrize("scale,fine", [(2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_scale_whose_log2_multiple_overflows_is_refused(L, scale, fine):
    """Weights are powers of two: scale * log2(e) infinite times the largest
    score's distance 0 from itself would be NaN."""
    need = L.vsa_paged_workspace_size(C.byref(desc(scale=scale)))
    assert (need > 0) == fine
    assert attn(L, desc(scale=scale), wsb=0) == (7 if fine else 2)
