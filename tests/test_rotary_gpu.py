"""GPU tests of rotary positions against the formulas in float64 and, for far positions, in more.

Bounds, with u = 2^-24: an angle within an eighth of a turn is off by u (its rounding to fp32) and 2^-30; sine and
cosine of fp32 inputs by 2 u of theirs, of bf16 by 2^-21 (the hardware's); their scaling, the two products
and the sum by a rounding each. So an output is off by at most 8 u (|x0| + |x1|) scale for fp32, 2^-20 (|x0| +
|x1|) scale for bf16, and then by half a step of its type."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from paged_reference import HALF, Problem
from paged_tree_reference import depths, trees
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu
ERR = {F32: 8 * 2.0 ** -24, BF: 2.0 ** -20}


def turned(x, spec, pos, backward=False):
    """(x [..., d] rotated by pos [...] in float64, the bound)."""
    x64, half, rot = x.double(), spec.rot // 2, spec.rot
    a = pos.double()[..., None] * torch.tensor(spec.freq, dtype=torch.float64)
    c, s = torch.cos(a) * spec.scale, torch.sin(a) * spec.scale * (-1 if backward else 1)
    i, j = (slice(0, half), slice(half, rot)) if spec.layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    y, tol = x64.clone(), torch.zeros_like(x64)
    y[..., i], y[..., j] = x64[..., i] * c - x64[..., j] * s, x64[..., i] * s + x64[..., j] * c
    tol[..., i] = tol[..., j] = ERR[x.dtype] * (x64[..., i].abs() + x64[..., j].abs()) * abs(spec.scale)
    return y, tol + HALF[x.dtype] * (y.abs() + tol) * (tol > 0)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype,d,rot", [(BF, 64, 64), (BF, 128, 128), (BF, 128, 96), (BF, 64, 18), (BF, 16, 2), (BF, 32, 12),
                                         (F32, 64, 64), (F32, 128, 32), (F32, 16, 6), (F32, 32, 20), (F32, 64, 30)])
@pytest.mark.parametrize("B,T,heads", [(1, 1, (1,)), (3, 37, (5, 2)), (2, 300, (8, 8, 8)), (1, 5, (0, 3)), (2, 2, (33, 1, 2))])
def test_rotation(lla, B, T, heads, dtype, d, rot, layout, backward):  # noqa: F811
    g = torch.Generator().manual_seed(d + rot + T)
    spec = lla.RotarySpec(rot, layout=layout, stretch=lla.STRETCH_WAVELENGTHS, factor=4.0, context=512)
    xs = [torch.randn(B, h, T, d, generator=g).to(dtype) for h in heads]
    for positions in (None, torch.randint(-5000, 5000, (B, T), generator=g).to(torch.int32)):
        pos = torch.arange(T).expand(B, T) if positions is None else positions
        dev = [x.cuda() for x in xs]
        got = lla.lla_rotary(dev, spec, positions=None if positions is None else positions.cuda(), backward=backward)
        for x, y, z in zip(xs, got, dev):
            check("y", y, *turned(x, spec, pos[:, None], backward))
            assert torch.equal(z.cpu(), x)
            assert torch.equal(y[..., rot:], z[..., rot:])
        into = lla.lla_rotary(dev, spec, positions=None if positions is None else positions.cuda(), backward=backward, out=dev)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(into, dev, got))
    assert lla.lla_stream_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_far_positions(lla, dtype):  # noqa: F811
    """Angles of positions to 2^31, whose product with a frequency has no bits left in fp32, and few in fp64."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    pos = [0, 1, 12345, 10 ** 6 + 3, 2 ** 24 + 1, 2 ** 30 - 7, 2 ** 31 - 1, -1, -2 ** 31]
    freq = [1.0, 0.1, 10000.0 ** -0.25, 1e-4, 3.0, -0.7, 1e-9, 1e5]
    spec = lla.RotarySpec(16, freq=freq, scale=1.0)
    x = torch.randn(1, 1, len(pos), 16, generator=torch.Generator().manual_seed(1)).to(dtype)
    angle = torch.tensor([[float((Decimal(p) * Decimal(f)) % two_pi) for f in freq] for p in pos], dtype=torch.float64)
    a, b = x[0, 0, :, :8].double(), x[0, 0, :, 8:].double()
    want = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)
    tol = ERR[dtype] * (a.abs() + b.abs()).repeat(1, 2)
    # (a frequency in turns is exact to 2^-65 and more of its doubles' product: 2^-100 of it)
    got = lla.lla_rotary(x.cuda(), spec, positions=torch.tensor([pos], dtype=torch.int32, device="cuda"))
    check("far", got[0, 0], want, tol + HALF[dtype] * (want.abs() + tol))


def test_values_that_are_not_finite_stay_in_their_pair(lla):  # noqa: F811
    for layout in (0, 1):
        spec = lla.RotarySpec(10, layout=layout)
        x = torch.randn(1, 1, 3, 16, dtype=F32)
        x[0, 0, 1, 1], x[0, 0, 1, 12] = math.inf, math.nan
        y = lla.lla_rotary(x.cuda(), spec).cpu()
        pair = [1, 6] if layout == 0 else [0, 1]
        bad = ~y.isfinite()
        assert bad[0, 0, 1, pair].all() and bad[0, 0, 1, 12] and bad.sum() == 3
        x[0, 0, 1, 12] = math.inf
        assert lla.lla_rotary(x.cuda(), spec)[0, 0, 1, 12] == math.inf


@pytest.mark.parametrize("dtype", [F32, BF])
def test_the_gradient_is_the_transpose(lla, dtype):  # noqa: F811
    """The rotation is linear: L(x + v) - L(x) = <gradient, v> for L = <g, rotated>, to the roundings of both."""
    gen = torch.Generator().manual_seed(3)
    spec = lla.RotarySpec(24, layout=1, scale=1.25, freq=[0.9 ** i for i in range(12)])
    x, v, g = (torch.randn(2, 3, 50, 32, generator=gen).to(dtype) for _ in range(3))
    fwd = lambda z: lla.lla_rotary(z.to(dtype).cuda(), spec).double().cpu()  # noqa: E731
    y, z = fwd(x), fwd(v)
    grad = lla.lla_rotary(g.cuda(), spec, backward=True).double().cpu()
    slack = 4 * (HALF[dtype] + ERR[dtype]) * 1.25 * 1.5
    terms = (g.double() * z).abs().sum() + (grad * v.double()).abs().sum()
    assert abs((g.double() * z).sum() - (grad * v.double()).sum()) <= slack * terms
    both = fwd(x.double() + v.double())
    step = (g.double() * (both - y)).sum()
    assert abs(step - (grad * v.double()).sum()) <= slack * ((g.double() * both).abs() + (g.double() * y).abs()).sum() + slack * terms


def test_a_training_step_of_rotated_parallax(lla):  # noqa: F811
    """lla_rotary, lla_parallax_forward, lla_parallax_backward and lla_rotary back, against autograd in float64.
    fp32: a logit of |s| up to 5 over d = 16 and sums over 40 keys are off by some (16 + 40) 10 u = 3e-5."""
    g = torch.Generator().manual_seed(5)
    B, H, T, d = 2, 3, 40, 16
    q, k, v, r, dout = (torch.randn(B, H, T, d, generator=g) for _ in range(5))
    r = r / 4
    spec = lla.RotarySpec(12, layout=1, base=100.0)
    pos = torch.randint(0, 9000, (B, T), generator=g).sort(-1).values.to(torch.int32)
    leaves = [x.double().requires_grad_() for x in (q, k, v, r)]
    a = pos.double()[:, None, :, None] * torch.tensor(spec.freq, dtype=torch.float64)
    z = torch.polar(torch.ones_like(a), a)

    def rot(x):
        w = torch.view_as_complex(x[..., :12].reshape(B, H, T, 6, 2)) * z
        return torch.cat([torch.view_as_real(w).reshape(B, H, T, 12), x[..., 12:]], -1)
    Q, K, R = rot(leaves[0]), rot(leaves[1]), rot(leaves[3])
    s = (Q @ K.transpose(-1, -2) / 4).masked_fill(~torch.ones(T, T, dtype=torch.bool).tril(), -math.inf)
    p = torch.softmax(s, -1)
    t = R @ K.transpose(-1, -2)
    out = (p * (1 + (p * t).sum(-1, keepdim=True) - t)) @ leaves[2]
    grads = torch.autograd.grad(out, leaves, dout.double())
    gq, gk, gv, gr = (x.cuda() for x in (q, k, v, r))
    fq, fk, fr = lla.lla_rotary([gq, gk, gr], spec, positions=pos.cuda())
    got = lla.lla_parallax_forward(fq, fk, gv, fr, 4.0)
    dq, dk, dv, dr = lla.lla_parallax_backward(fq, fk, gv, fr, dout.cuda(), 4.0)
    dq, dk, dr = lla.lla_rotary([dq, dk, dr], spec, positions=pos.cuda(), backward=True, out=[dq, dk, dr])
    rel = lambda x, y: float((x.double().cpu() - y.detach()).norm() / y.detach().norm())  # noqa: E731
    assert rel(got, out) <= 1e-4
    for x, y in zip((dq, dk, dv, dr), grads):
        assert rel(x, y) <= 1e-4


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("probe,offsets", [(False, False), (True, True)])
@pytest.mark.parametrize("dtype,d,dv,Hq,Hkv,page,rot", [(BF, 64, 64, 8, 2, 16, 64), (BF, 128, 128, 40, 8, 64, 96),
                                                        (F32, 64, 32, 6, 2, 16, 30), (BF, 16, 128, 3, 3, 32, 2), (F32, 32, 16, 1, 1, 16, 32)])
@pytest.mark.parametrize("lens,news", [([1], [1]), ([40, 0, 77, 300], [1, 0, 12, 200]), ([5000] * 3, [900] * 3)])
def test_append(lla, lens, news, dtype, d, dv, Hq, Hkv, page, rot, probe, offsets, layout):  # noqa: F811
    P = Problem(lens, news, Hq, Hkv, d, dv, page, dtype, probe, seed=d + rot)
    g = torch.Generator().manual_seed(2)
    N = sum(news)
    k, v = torch.randn(N, Hkv, d, generator=g).to(dtype), torch.randn(N, Hkv, dv, generator=g).to(dtype)
    spec = lla.RotarySpec(rot, layout=layout, base=500.0, scale=1.5)
    cache, q, r, starts = P.cuda(lla)
    where = [(b, n - t, i) for b, (n, t) in enumerate(zip(lens, news)) for i in range(t)]
    off = None
    if offsets:
        off = torch.tensor([x + 10 ** 6 for tree in trees(news, 2) for x in depths(tree)], dtype=torch.int32)
    pos = torch.tensor([first + (i if off is None else int(off[at])) for at, (_, first, i) in enumerate(where)])
    got_q, got_r = lla.lla_paged_append_rotary(k.cuda(), v.cuda(), cache, starts, spec, q, r=r,
                                               offsets=None if off is None else off.cuda())
    assert lla.lla_stream_status() == 0
    check("q", got_q, *turned(P.q, spec, pos[:, None]))
    assert (got_r is None) == (r is None)
    if probe:
        check("r", got_r, *turned(P.r, spec, pos[:, None]))
    at = [(int(P.table[b, (f + i) // page]), (f + i) % page) for b, f, i in where]
    pg, slot = torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])
    check("k", cache.k_pages.cpu()[pg, :, slot], *turned(k, spec, pos[:, None]))
    assert torch.equal(cache.v_pages.cpu()[pg, :, slot], v) and (cache.mass.cpu()[pg, :, slot] == 0).all()
    rest = torch.ones(P.num_pages, page, dtype=torch.bool)
    rest[pg, slot] = False
    for x, y in ((cache.k_pages, P.k), (cache.v_pages, P.v), (cache.mass, P.mass)):
        assert torch.equal(x.cpu().transpose(1, 2)[rest], y.transpose(1, 2)[rest])
    # in place, alone, and without queries
    cache2, q2, r2, _ = P.cuda(lla)
    lla.lla_paged_append_rotary(k.cuda(), v.cuda(), cache2, starts, spec, q2, r=r2, q_out=q2, r_out=r2,
                                offsets=None if off is None else off.cuda())
    assert torch.equal(q2, got_q) and torch.equal(cache2.k_pages, cache.k_pages) and (r is None or torch.equal(r2, got_r))
    cache3 = P.cuda(lla)[0]
    assert lla.lla_paged_append_rotary(k.cuda(), v.cuda(), cache3, starts, spec,
                                       offsets=None if off is None else off.cuda()) == (None, None)
    assert torch.equal(cache3.k_pages, cache.k_pages) and torch.equal(cache3.v_pages, cache.v_pages)


def test_append_leaves_what_no_sequence_covers(lla):  # noqa: F811
    """Rows around the sequences, an impossible length, a bad page number, more new tokens than positions."""
    P = Problem([30, 40, 50], [4, 5, 6], 2, 1, 32, 32, 16, F32, False, seed=1)
    spec = lla.RotarySpec(32)
    cache, q, _, starts = P.cuda(lla)
    k = v = torch.randn(18, 1, 32, device="cuda")
    q = torch.cat([q, q[:3]])
    out = torch.full_like(q, 7.0)
    cache.lens[0] = 10000
    cache.page_table[1, 2] = 99
    lla.lla_paged_append_rotary(k, v, cache, starts, spec, q, q_out=out)
    assert lla.lla_stream_status() == 1
    assert (out[:4] == 7).all() and (out[15:] == 7).all() and not (out[9:15] == 7).any()
    pg, off = P.slots(0)
    assert torch.equal(cache.k_pages.cpu()[pg, :, off], P.k[pg, :, off])
    cache, q, _, starts = P.cuda(lla)
    cache.lens[2] = 4  # six new tokens: the first two have no slot
    lla.lla_paged_append_rotary(k[:15], v[:15], cache, starts, spec)
    assert lla.lla_stream_status() == 0
    pg, off = P.slots(2)
    assert torch.equal(cache.v_pages[pg[:4], :, off[:4]], v[11:15])
    assert torch.equal(cache.v_pages.cpu()[pg[4:], :, off[4:]], P.v[pg[4:], :, off[4:]])


def test_streams_and_capture(lla):  # noqa: F811
    x = torch.randn(2, 4, 100, 64, device="cuda", dtype=BF)
    spec = lla.RotarySpec(64)
    want = lla.lla_rotary(x, spec)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        got = lla.lla_rotary(x, spec, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        lla.lla_rotary(x, spec, out=out)
    x.mul_(2)
    graph.replay()
    assert torch.equal(out, lla.lla_rotary(x, spec))


def test_binding_refusals(lla):  # noqa: F811
    x = torch.randn(2, 4, 10, 64, device="cuda", dtype=BF)
    spec = lla.RotarySpec(64)
    for bad in (x.cpu(), x[0], x.half(), x.transpose(1, 2), [x] * 4, [], [x, x[:, :, :5].contiguous()], [x, x.float()]):
        with pytest.raises(ValueError):
            lla.lla_rotary(bad, spec)
    for kw in (dict(positions=torch.zeros(2, 10, device="cuda")), dict(positions=torch.zeros(2, 9, dtype=torch.int32, device="cuda")),
               dict(positions=torch.zeros(2, 10, dtype=torch.int32)), dict(out=x[:1]), dict(out=[x, x])):
        with pytest.raises(ValueError):
            lla.lla_rotary(x, spec, **kw)
    with pytest.raises(lla.LlaError):
        lla.lla_rotary(x[..., :32].contiguous(), spec)
    with pytest.raises(lla.LlaError):
        lla.lla_rotary([x, x.clone()], spec, out=[x, x])


def test_more_heads_than_a_grid_has_rows(lla):  # noqa: F811
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 600000, 1, 16, generator=g).to(BF)
    spec = lla.RotarySpec(16)
    pos = torch.tensor([[7]], dtype=torch.int32)
    check("y", lla.lla_rotary(x.cuda(), spec, positions=pos.cuda()), *turned(x, spec, pos[:, None]))
    P = Problem([20], [1], 600000, 1, 16, 16, 16, BF, False, seed=1)
    cache, q, _, starts = P.cuda(lla)
    k = torch.zeros(1, 1, 16, dtype=BF, device="cuda")
    got, _ = lla.lla_paged_append_rotary(k, k, cache, starts, spec, q)
    check("q", got, *turned(P.q, spec, torch.tensor([[19]])))
    assert lla.lla_stream_status() == 0
