"""Rotary positions with several axes on a machine without a GPU: the
frequencies' fixed point, and the refusals of both layers."""
import ctypes as C
import math
from fractions import Fraction

import pytest
import torch

from bwd_tile_mean_gb300 import build as libbuild
from bwd_tile_mean_gb300 import vsa

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return vsa.lib()


def pi(bits=400):
    """pi as a fraction, by Machin's formula."""
    def arctan(n):
        x = total = (1 << bits) // n
        k = 1
        while x:
            x //= n * n
            k += 2
            total += -(x // k) if k % 4 == 3 else x // k
        return total
    return Fraction(4 * (4 * arctan(5) - arctan(239)), 1 << bits)


@pytest.mark.parametrize("f", [1.0, 0.5, 10000.0 ** (-2 / 44), 1e-4, 2e-9, 5e-324, 1e-300, 0.0, 3.0, 100.25, 1024.0, -1.0,
                               -0.37, math.pi, 2 * math.pi, 1 / 3])
def test_turns_are_the_rounded_fractions(L, f):
    rope = vsa.RopeDesc()
    assert L.vsa_rope_init(C.byref(rope), 1, 16, 0, (C.c_int32 * 8)(), (C.c_double * 8)(*([f] * 8))) == 0
    exact = Fraction(f) / (2 * pi()) * (1 << 64)
    size = math.floor(abs(exact) + Fraction(1, 2))  # halves do not occur: pi is irrational
    want = (size if f >= 0 else -size) % (1 << 64)
    assert [rope.turn[i] for i in range(8)] == [want] * 8


def rope(**kw):
    a = dict(dims=(44, 42, 42), interleaved=True)
    a.update(kw)
    return vsa.AxialRope(**a)


def test_dims_and_frequencies(L):
    r = rope(scale=(2.0, 1.0, 1.0))
    assert r.rot_dim == 128 and len(r.freqs) == 64 and r.axes == (0,) * 22 + (1,) * 21 + (2,) * 21
    assert r.freqs[0] == 2.0 and r.freqs[22] == 1.0 and r.freqs[23] == 10000.0 ** (-2 / 42)
    r = vsa.AxialRope((16, 24, 24), freqs=[0.1] * 32, axes=[2, 1, 0, 0] * 8)
    assert r.axes[:4] == (2, 1, 0, 0)
    for bad in (dict(dims=()), dict(dims=(16,) * 5), dict(dims=(15, 17)), dict(dims=(10, 10)), dict(dims=(128, 16)),
                dict(dims=(0,)), dict(base=0.0), dict(base=-1.0), dict(scale=(1.0, 2.0)), dict(freqs=[1.0]), dict(axes=[0]),
                dict(freqs=[2000.0] * 64), dict(freqs=[math.nan] * 64), dict(axes=[3] * 64), dict(axes=[-1] * 64),
                dict(freqs=[1.0] * 64, scale=2.0)):
        with pytest.raises(ValueError):
            rope(**bad)


def test_init_errors(L):
    d = vsa.RopeDesc()
    axis, freq = (C.c_int32 * 64)(), (C.c_double * 64)()
    init = lambda n=1, rot=16, a=axis, f=freq, r=C.byref(d): L.vsa_rope_init(r, n, rot, 0, a, f)  # noqa: E731
    assert init() == 0 and init(n=4, rot=128) == 0
    assert init(r=None) == 1 and init(a=None) == 1 and init(f=None) == 1
    assert init(n=0) == 2 and init(n=5) == 2
    assert init(rot=0) == 5 and init(rot=24) == 5 and init(rot=144) == 5
    assert init(a=(C.c_int32 * 64)(*([1] * 64))) == 2
    assert init(f=(C.c_double * 64)(*([math.inf] * 64))) == 2


def apply(L, r=None, dtype=0, B=1, S=3, D=128, n=1, pos=FAKE, pb=0, pt=1, heads=2, **kw):
    t = dict(x=FAKE, y=FAKE, heads=heads, x_batch=0, x_token=256, x_head=128, y_batch=0, y_token=256, y_head=128)
    t.update(kw)
    one = vsa.RopeTensor(*[t[f] for f, _ in vsa.RopeTensor._fields_])
    return L.vsa_rope_apply(C.byref(r or rope().desc), dtype, B, S, D, (vsa.RopeTensor * 2)(one, one), n, pos, pb, pt, 0, None)


def test_apply_errors(L):
    assert apply(L, S=0) == 0 and apply(L, B=0) == 0 and apply(L, S=0, pos=None, x=None, y=None) == 0  # nothing to do
    assert L.vsa_rope_apply(None, 0, 1, 3, 128, None, 1, FAKE, 0, 1, 0, None) == 1
    assert L.vsa_rope_apply(C.byref(rope().desc), 0, 1, 3, 128, None, 1, FAKE, 0, 1, 0, None) == 1
    assert apply(L, x=None) == 1 and apply(L, y=None) == 1 and apply(L, pos=None) == 1
    assert apply(L, dtype=2) == 3
    assert apply(L, D=64) == 5
    assert apply(L, B=-1) == 2 and apply(L, S=-1) == 2 and apply(L, n=0) == 2 and apply(L, n=3) == 2
    assert apply(L, heads=0) == 2
    for name in ("x_batch", "x_token", "x_head", "y_batch", "y_token", "y_head"):
        assert apply(L, **{name: 4}) == 2 and apply(L, **{name: -8}) == 2, name
    assert apply(L, x=FAKE + 8) == 4 and apply(L, y=FAKE + 2) == 4 and apply(L, pos=FAKE + 2) == 4
    assert apply(L, pb=-1) == 2 and apply(L, pt=-1) == 2
    assert apply(L, B=1 << 16, S=1 << 15) == 5
    assert apply(L, heads=2 ** 31 - 1, n=2) == 5
    bad = vsa.RopeDesc(3, 128, 0)
    bad.axis[5] = 3
    assert apply(L, r=bad) == 2


def test_table_errors(L):
    t = lambda T=3, pos=FAKE, pt=3, c=FAKE, s=FAKE: L.vsa_rope_table(  # noqa: E731
        C.byref(rope().desc), T, pos, pt, c, s, None)
    assert t(T=0) == 0 and t(T=-1) == 2 and t(pt=-1) == 2
    assert t(pos=None) == 1 and t(c=None) == 1 and t(s=None) == 1
    assert t(pos=FAKE + 2) == 4 and t(c=FAKE + 4) == 4 and t(s=FAKE + 8) == 4
    assert L.vsa_rope_table(None, 3, FAKE, 3, FAKE, FAKE, None) == 1


def test_tensor_refusals(L):
    r = rope()
    q, k = torch.zeros(2, 5, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 128, dtype=torch.bfloat16)
    pos = torch.zeros(5, 3, dtype=torch.int32)
    buf = torch.zeros(2, 5, 8, 128, dtype=torch.bfloat16)
    for match, call in (
            ("GPU only", lambda: r.forward(q, k, pos)),
            ("GPU only", lambda: r.backward(q, None, pos)),
            ("positions", lambda: r.forward(q, k)),
            ("positions", lambda: r.forward(q, k, pos.long())),
            ("positions", lambda: r.forward(q, k, pos[:4])),
            ("positions", lambda: r.forward(q, k, pos[:, :2])),
            ("positions", lambda: r.forward(q, k, pos[None].expand(3, 5, 3))),
            ("positions", lambda: r.forward(q, k, torch.zeros(3, 5, dtype=torch.int32).T)),
            ("layout", lambda: r.forward(q, k, pos, layout="bsd")),
            ("q: expected", lambda: r.forward(q.float(), None, pos)),
            ("q: expected", lambda: r.forward(q[0], None, pos)),
            ("k: expected", lambda: r.forward(q, k.half(), pos)),
            ("k: expected", lambda: r.forward(q, k[:, :4], pos)),
            ("dense", lambda: r.forward(torch.zeros(2, 5, 128, 4, dtype=torch.bfloat16).transpose(2, 3), None, pos)),
            ("multiples of 8", lambda: r.forward(torch.zeros(2, 5, 4, 132, dtype=torch.bfloat16)[..., :128], None, pos)),
            ("k_out without k", lambda: r.forward(q, None, pos, k_out=k)),
            ("q_out: expected", lambda: r.forward(q, k, pos, q_out=k)),
            ("its rows share", lambda: r.forward(q, k, pos, q_out=torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
                                                 .expand(2, 5, 4, 128))),
            ("shares memory with q", lambda: r.forward(buf[:, :, 1:5], None, pos, q_out=buf[:, :, :4])),
            ("shares memory with k", lambda: r.forward(q, buf[:, :, 3:5], pos, q_out=buf[:, :, :4])),
            ("shares memory with k_out", lambda: r.forward(q, k, pos, q_out=buf[:, :, :4], k_out=buf[:, :, 3:5])),
            ("shares memory with q", lambda: r.forward(q[..., :2, :], k, pos, k_out=q[..., :2, :])),
            ("gradient", lambda: r.forward(q.clone().requires_grad_(), k, pos))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(ValueError, match="GPU only"):  # parts of one buffer side by side are fine
        r.forward(buf[:, :, :4], buf[:, :, 4:6], pos, q_out=buf[:, :, :4], k_out=buf[:, :, 6:8])
    with pytest.raises(ValueError, match="GPU only"):
        with torch.no_grad():
            r.forward(q.clone().requires_grad_(), k, pos)
    with pytest.raises(ValueError, match="GPU only"):
        r.forward(q.transpose(1, 2), k.transpose(1, 2), pos, layout="bhsd")
    empty = r.forward(q[:, :0], k[:, :0], pos[:0])  # no token: nothing to launch
    assert empty[0].shape == (2, 0, 4, 128) and empty[1].shape == (2, 0, 2, 128)
    for match, call in (("GPU only", lambda: r.table(pos)),
                        ("positions", lambda: r.table(pos[:, :2])),
                        ("cos: expected", lambda: r.table(pos, cos=torch.zeros(5, 63))),
                        ("shares memory", lambda: r.table(pos, cos=(x := torch.zeros(5, 64)), sin=x))):
        with pytest.raises(ValueError, match=match):
            call()
