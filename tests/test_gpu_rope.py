"""Rotary positions with several axes against their definition in fp64."""
import math

import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
D, U = ref.D, ref.U


def vsa():
    from bwd_tile_mean_gb300 import vsa as m
    return m


def randn(*shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def angles(rope, pos):
    """[..., pairs] in fp64: an angle is off by 2^-53 of itself, 2^-21 at the
    farthest positions here: those are reduced by whole turns first."""
    f = torch.tensor(rope.freqs, dtype=torch.float64)
    return pos.double()[..., list(rope.axes)] * f


def turned(rope, x, pos, back=False):
    """x [B, S, H, D] rotated, and a bound on the call's error: c and s are off
    by 2^-22 at most, each product and sum rounds to fp32 and the result to
    dtype (half a step: U)."""
    a = angles(rope, pos).unsqueeze(-2)
    c, s = a.cos(), a.sin() * (-1 if back else 1)
    h = rope.rot_dim // 2
    i = torch.arange(h)
    i1, i2 = (2 * i, 2 * i + 1) if rope.interleaved else (i, i + h)
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    x1, x2 = x.double()[..., i1], x.double()[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    one = (2.0 ** -22 + 2.0 ** -23) * (x1.abs() + x2.abs())
    tol[..., i1], tol[..., i2] = one, one
    tol[..., :2 * h] += U[x.dtype] * (y[..., :2 * h].abs() + tol[..., :2 * h])
    if x.dtype == torch.float16:
        tol[..., :2 * h] += 2.0 ** -25
    return y, tol


def check(got, want):
    y, tol = want
    d = (got.double().cpu() - y).abs()
    assert (d <= tol).all(), f"off by {float((d - tol).max()):.3e} over the bound"


def place(x, layout):
    return x.transpose(1, 2).contiguous() if layout == "bhsd" else x[0] if layout == "tnd" else x


def back_to(x, layout):
    return x.transpose(1, 2) if layout == "bhsd" else x[None] if layout == "tnd" else x


CASES = [  # B, S, Hq, Hkv, dims, layout, dtype, interleaved
    (1, 1, 1, 1, (128,), "bshd", torch.bfloat16, True),
    (1, 1, 1, 1, (16,), "tnd", torch.float16, False),
    (2, 37, 12, 3, (16, 56, 56), "bshd", torch.float16, False),
    (3, 101, 5, 5, (44, 42, 42), "bhsd", torch.bfloat16, True),
    (1, 333, 40, 40, (44, 42, 42), "bshd", torch.bfloat16, False),
    (1, 57, 7, 1, (48, 48), "tnd", torch.float16, True),
    (2, 64, 8, 2, (24, 20, 20), "bhsd", torch.float16, False),
    (1, 2111, 3, 2, (32, 32, 32, 32), "tnd", torch.bfloat16, False),
    (2, 19, 4, 4, (8, 4, 4), "bshd", torch.bfloat16, True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_backward(case):
    B, S, Hq, Hkv, dims, layout, dtype, inter = case
    rope = vsa().AxialRope(dims, interleaved=inter, scale=[1.0] * (len(dims) - 1) + [0.75])
    g = torch.Generator().manual_seed(S)
    pos = torch.randint(-50, 4000, (S, len(dims)), generator=g).to(torch.int32)
    q, k = randn(B, S, Hq, D, dtype=dtype, seed=1), randn(B, S, Hkv, D, dtype=dtype, seed=2)
    gpu = [place(x, layout).cuda() for x in (q, k)]
    for call, back in ((rope.forward, False), (rope.backward, True)):
        yq, yk = call(*gpu, positions=pos.cuda(), layout=layout)
        assert yq.is_contiguous() and yq.shape == gpu[0].shape
        for y, x in ((yq, q), (yk, k)):
            check(back_to(y, layout), turned(rope, x, pos, back))
            assert torch.equal(back_to(y, layout)[..., rope.rot_dim:].cpu(), x[..., rope.rot_dim:])
        alone = call(gpu[0], positions=pos.cuda(), layout=layout)
        assert torch.equal(alone, yq)
    # its own positions for every batch entry
    if layout != "tnd":
        per = torch.randint(0, 999, (B, S, len(dims)), generator=g).to(torch.int32)
        yq, yk = rope.forward(*gpu, positions=per.cuda(), layout=layout)
        check(back_to(yq, layout), turned(rope, q, per))


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(inter):
    """The angle is exact wherever the position: compared with a position one
    turn of a frequency of 2 pi / 2^10 earlier, and with fp64 while that holds."""
    f = [2 * math.pi / 1024, 1.0, 1e-4, 0.3] * 2
    rope = vsa().AxialRope((16,), freqs=f, interleaved=inter)
    at = [0, 1, -1, 1023, 1 << 20, (1 << 31) - 1, -(1 << 31), 123456789, -98765432]
    pos = torch.tensor(at, dtype=torch.int64)[:, None]
    c, s = rope.table(pos.to(torch.int32).cuda())
    from fractions import Fraction
    two_pi = Fraction(2 * 314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    for r, p in enumerate(at):
        for i, x in enumerate(f):
            a = Fraction(x) * p
            a = float(a - two_pi * math.floor(a / two_pi))
            assert abs(float(c[r, i]) - math.cos(a)) <= 2.0 ** -22, (p, x)
            assert abs(float(s[r, i]) - math.sin(a)) <= 2.0 ** -22, (p, x)


@pytest.mark.parametrize("inter", [False, True])
def test_same_bits_as_the_table(inter):
    dtype = torch.bfloat16
    rope = vsa().AxialRope((44, 42, 42), interleaved=inter)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 900, (131, 4), generator=g).to(torch.int32)
    x = randn(131, 6, D, dtype=dtype, seed=3)
    c, s = rope.table(pos.cuda()[:, :3])  # a token's positions 4 apart
    want = torch.from_numpy(ref.rotate(x, c.cpu(), s.cpu(), inter)).to(dtype)
    got = rope.forward(x.cuda(), positions=pos.cuda()[:, :3], layout="tnd")
    assert torch.equal(got.cpu(), want)
    cache = vsa().PagedCache("bshd", dtype, 1, 6, 6, D, 16, 10, 10)
    cache.page_table.copy_(torch.arange(10, dtype=torch.int32)[None])
    cache.seq_lens.fill_(131)
    q = cache.append(x.cuda(), x.cuda(), x.cuda(), cu_seqlens=torch.tensor([0, 131], dtype=torch.int32).cuda(), cos=c, sin=s,
                     positions=torch.arange(131, dtype=torch.int32).cuda(), interleaved=inter)
    assert torch.equal(q, got) and torch.equal(cache.k.view(160, 6, D)[:131], got)


@pytest.mark.parametrize("layout", ["bshd", "bhsd", "tnd"])
def test_strides_and_in_place(layout):
    """Parts of one projection's output, outputs into strided buffers, in place,
    a broadcast input."""
    dtype, B, S, Hq, Hkv = torch.float16, 1 if layout == "tnd" else 2, 45, 6, 2
    rope = vsa().AxialRope((16, 56, 56))
    pos = torch.randint(0, 100, (S, 3), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    qkv = randn(B, S, Hq + 2 * Hkv, D, dtype=dtype, seed=4).cuda()

    def parts(buf):
        q, k = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv]
        return [x.transpose(1, 2) if layout == "bhsd" else x[0] if layout == "tnd" else x for x in (q, k)]

    q, k = parts(qkv)
    want = rope.forward(q.contiguous(), k.contiguous(), positions=pos, layout=layout)
    got = rope.forward(q, k, positions=pos, layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = torch.full_like(qkv, 7.0)
    oq, ok = parts(buf)
    rope.forward(q, k, positions=pos, layout=layout, q_out=oq, k_out=ok)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and (buf[:, :, Hq + Hkv:] == 7.0).all()
    same = qkv.clone()
    q, k = parts(same)
    rope.forward(q, k, positions=pos, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(same[:, :, Hq + Hkv:], qkv[:, :, Hq + Hkv:])
    one = parts(qkv)[1][:1] if layout != "tnd" else parts(qkv)[1][:, :1]  # shared by all batch entries, or heads
    wide = one.expand(B, -1, -1, -1) if layout != "tnd" else one.expand(-1, 5, -1)
    assert torch.equal(rope.forward(wide, positions=pos, layout=layout),
                       rope.forward(wide.contiguous(), positions=pos, layout=layout))


def test_gradient_is_the_formulas_and_the_differences():
    """<dy, J dx> from differences of forward (linear in x: exact but for
    roundings) against <backward(dy), dx>."""
    rope = vsa().AxialRope((44, 42, 42), interleaved=True)
    pos = torch.randint(0, 500, (77, 3), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    x, d, dy = (randn(1, 77, 3, D, dtype=torch.float16, seed=s).cuda() for s in (1, 2, 3))
    d = d * 0.125
    rise = (rope.forward(x + d, positions=pos).double() - rope.forward(x, positions=pos).double()) * dy.double()
    back = rope.backward(dy, positions=pos).double() * ((x + d).double() - x.double())
    # forward's values round by U each, twice per entry; backward's by U
    # (independent, but summed as if they were not); c and s by 2^-22
    n = 4 * x.abs().amax().double()
    bound = (dy.double().abs() * n * U[torch.float16] * 2).sum() * 1.01 + (back.abs() * U[torch.float16]).sum() * 1.01
    assert abs(rise.sum() - back.sum()) <= bound
    # far below the size of either sum's terms, and the same row by row
    diff = (rise.sum((0, 2, 3)) - back.sum((0, 2, 3))).abs()
    assert (diff <= (dy.double().abs() * n * U[torch.float16] * 2 + back.abs() * U[torch.float16]).sum((0, 2, 3)) * 1.01).all()
    # there and back: the input, to roundings
    y = rope.backward(rope.forward(x, positions=pos), positions=pos)
    tol = 2 * U[torch.float16] * n + 2.0 ** -20
    assert ((y.double() - x.double()).abs() <= tol).all()


def test_infinite_and_nan_rows_stay_in_their_pairs():
    rope = vsa().AxialRope((32, 32), interleaved=False)
    pos = torch.ones(3, 2, dtype=torch.int32).cuda()
    x = torch.zeros(3, 1, D, dtype=torch.bfloat16)
    x[0, 0, 5], x[1, 0, 100], x[2, 0, 40] = math.inf, math.nan, math.nan
    y = rope.forward(x.cuda(), positions=pos, layout="tnd").cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [5, 37]] = want[1, 0, 100] = want[2, 0, [8, 40]] = True
    assert torch.equal(bad, want)


def test_streams_and_graphs():
    m = vsa()
    rope = m.AxialRope((44, 42, 42))
    pos = torch.randint(0, 100, (300, 3)).to(torch.int32).cuda()
    x = torch.randn(1, 300, 8, D, device="cuda").bfloat16()
    want = rope.forward(x, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rope.forward(x, positions=pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.forward(x, positions=pos, q_out=out)
        rope.backward(out, positions=pos, q_out=out)
        rope.forward(out, positions=pos, q_out=out)
    x.copy_(torch.randn(1, 300, 8, D, device="cuda").bfloat16())
    graph.replay()
    step = rope.forward(x, positions=pos)
    step = rope.forward(rope.backward(step, positions=pos), positions=pos)
    assert torch.equal(out, step)


def test_with_tiles_and_block_sparse_attention():
    """A clipped latent's training step: tiles, positions in tile order,
    rotation, attention, and the gradients back through both, against fp64
    autograd over the same selection."""
    m = vsa()
    T, H, W, heads, dtype = 6, 9, 13, 2, torch.bfloat16
    rope = m.AxialRope((44, 42, 42), interleaved=True)
    lat = [torch.randn(1, T, H, W, heads, D, generator=torch.Generator().manual_seed(s)).to(dtype).cuda() for s in range(4)]
    tiled, var = zip(*(m.tile_3d(x) for x in lat))
    q, k, v, dO = tiled
    pos = m.tile_positions(T, H, W)
    n = var[0].numel()
    plan = m.Plan("bshd", dtype, 1, heads, heads, D, 256, 256, n, n, 256 * n, 256 * n, n, q_var=var[0], kv_var=var[0])
    rq, rk = rope.forward(q, k, positions=pos)
    pad = torch.arange(256, device="cuda")[None] >= var[0][:, None]
    assert (rq.view(n, 256, heads, D)[pad] == 0).all()  # padding stays zero
    grid = torch.stack(torch.meshgrid(*(torch.arange(e) for e in (T, H, W)), indexing="ij"), -1).view(-1, 3)
    assert torch.equal(pos.cpu().view(n, 256, 3)[~pad.cpu()].double().sum(0), grid.double().sum(0))
    plan.build_block_map(rq, rk, n)
    out, lse, osp = plan.forward(rq, rk, v)
    dq, dk, dv = plan.backward(dO, rq, rk, v, osp, lse)
    gq, gk = rope.backward(dq, dk, positions=pos, q_out=dq, k_out=dk)

    qq, kk, vv = (x.double().cpu().requires_grad_() for x in (q, k, v))
    a = angles(rope, pos.cpu())[:, None]
    turn = torch.polar(torch.ones_like(a), a)
    rot = lambda x: torch.view_as_real(torch.view_as_complex(x.reshape(1, -1, heads, 64, 2)) * turn).flatten(-2)  # noqa: E731
    s = torch.einsum("bqhd,bkhd->bhqk", rot(qq), rot(kk)) / math.sqrt(D)
    s = s.masked_fill(pad.flatten().cpu()[None, None, None], -math.inf)
    o = torch.einsum("bhqk,bkhd->bqhd", s.softmax(-1), vv)
    (o * dO.double().cpu()).sum().backward()
    for name, got, want in (("out", out, o), ("dq", gq, qq.grad), ("dk", gk, kk.grad), ("dv", dv, vv.grad)):
        want, got = want.detach(), got.double().cpu()
        # the rotation's inputs, outputs and gradients and the attention's P, dS and outputs each round to bf16 once
        rel = float((got - want).norm() / want.norm())
        assert rel <= 6 * U[dtype], (name, rel)


def test_offsets_past_32_bits():
    """Tokens 2^31 elements apart, and more heads than one unit takes."""
    rope = vsa().AxialRope((44, 42, 42))
    pos = torch.tensor([[3, 4, 5], [700, 8, 9], [11, 0, 77]], dtype=torch.int32).cuda()
    apart = (1 << 31) + 512
    buf = torch.empty(2 * apart + 128 * 24, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, 3, 24, D), (0, apart, D, 1))
    x.copy_(torch.randn(1, 3, 24, D, generator=torch.Generator().manual_seed(1)))
    want = rope.forward(x.contiguous(), positions=pos)
    assert torch.equal(rope.forward(x, positions=pos), want)
    rope.forward(x, positions=pos, q_out=x)
    assert torch.equal(x, want)


def test_tokens_without_heads_or_batch():
    rope = vsa().AxialRope((64, 64))
    pos = torch.zeros(3, 2, dtype=torch.int32).cuda()
    x = torch.randn(1, 3, 2, D, device="cuda").bfloat16()
    q, k = rope.forward(x, x[:, :, :0], positions=pos)
    assert k.shape == (1, 3, 0, D) and torch.equal(q, x)  # position 0: no turn
    assert rope.forward(x[:0], positions=pos).shape == (0, 3, 2, D)
    assert rope.table(pos[:0])[0].shape == (0, 64)
