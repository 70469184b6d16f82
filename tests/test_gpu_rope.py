"""Rotary positions on several axes against the formula in 64 bits.

Tolerance of an element y = a cos - b sin (or a sin + b cos), per element:
  |got - y| <= eps/2 |y| + 2^-21 (|a| + |b|)
  - the result is rounded once to its type: half a step, torch.finfo(t).eps / 2 relative to the value;
  - cos and sin carry at most two ulp of fp32 (2^-23), and the two products and their sum three roundings of 2^-24:
    less than 2^-21 of |a| + |b|; the angle itself is reduced in fp64 (under 2^-30 for these positions).
Elements that no axis covers are copies.
"""
import pytest
import torch

from tests.gpu_util import expect_status, sd

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = (torch.bfloat16, torch.float16, torch.float32)


def pairs(axes, halves):
    lo, hi, axis, rel, at = [], [], [], [], 0
    for a, s in enumerate(axes):
        for m in range(s // 2):
            lo.append(at + (m if halves else 2 * m))
            hi.append(at + (m + s // 2 if halves else 2 * m + 1))
            axis.append(a)
            rel.append(-2.0 * m / s)
        at += s
    return lo, hi, axis, rel


def reference(x, pos, axes, thetas, halves, inverse):
    """(rotated, |a| + |b| per element) in fp64; x [B,H,n,d], pos [B or 1,n,A]."""
    lo, hi, axis, rel = pairs(axes, halves)
    x = x.double().cpu()
    pos = pos.double().cpu().expand(x.shape[0], -1, -1)
    base = torch.tensor([thetas[a] for a in axis], dtype=torch.float64)
    ang = pos[..., axis] * base ** torch.tensor(rel, dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    if inverse:
        s = -s
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return y, mag


def close(got, ref, mag, what=""):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double().cpu() - ref).abs()
    bound = half * ref.abs() + 2.0 ** -21 * mag
    # below the smallest normal a type's step no longer shrinks
    bound = bound + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    assert bool((err <= bound).all()), f"{what}: {float((err - bound).max()):.3e} over the bound"


def rows(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def positions(shape, dtype, seed, top=4096):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, top, shape, generator=g)
    return (p.float() * 0.37).to(DEV) if dtype == torch.float32 else p.to(torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("halves, d, axes", [
    (False, 8, (8,)), (False, 64, (64,)), (False, 96, (32, 32, 32)), (False, 96, (18, 22)), (False, 128, (16, 56, 56)),
    (False, 72, (2, 2, 2, 4)), (False, 256, (64, 96, 96)), (True, 64, (64,)), (True, 96, (8, 24, 56)),
    (True, 128, (16, 56, 56)), (True, 104, (8, 40)), (True, 256, (256,))])
@pytest.mark.parametrize("inverse", (False, True))
def test_widths_axes_types(dtype, halves, d, axes, inverse):
    thetas = (1e4, 1e6, 500.0, 1.0)[: len(axes)]
    layout = sd().ROPE_HALVES if halves else sd().ROPE_INTERLEAVED
    spec = sd().rope_spec(axes, thetas, layout, inverse)
    for n, pt in ((1, torch.int32), (37, torch.float32)):
        x = [rows((2, h, n, d), dtype, 3 + h) for h in (5, 1)]
        pos = positions((2, n, len(axes)), pt, 9)
        y = [torch.empty_like(v) for v in x]
        sd().safedit_rope_rows(x, y, pos, spec)
        expect_status(0)
        for a, b in zip(x, y):
            close(b, *reference(a, pos, axes, thetas, halves, inverse), what=f"n={n}")
            rest = sum(axes)
            assert torch.equal(a[..., rest:], b[..., rest:])


def test_far_positions_keep_their_angle():
    """Positions near 2^31 (i32) and 2^23 (f32): the reduction is in fp64."""
    spec = sd().rope_spec((32, 32), (1e4, 10.0))
    x = rows((1, 2, 64, 64), torch.float32, 1)
    for pos in (torch.arange(64, dtype=torch.int32)[None, :, None].expand(1, 64, 2) + (2 ** 31 - 70),
                (torch.arange(64).float()[None, :, None].expand(1, 64, 2) + 2 ** 23), -positions((1, 64, 2), torch.int32, 4).cpu()):
        y = torch.empty_like(x)
        sd().safedit_rope_rows([x], [y], pos.to(DEV), spec)
        expect_status(0)
        ref, mag = reference(x, pos, (32, 32), (1e4, 10.0), False, False)
        # a frequency's fp64 rounding is multiplied by the position: 2^31 * 2^-50 radians
        close(y, ref, mag * (1 + 2.0 ** 3))


@pytest.mark.parametrize("si, di", [(False, False), (True, False), (False, True), (True, True)])
def test_indexed_sides(si, di):
    B, H, N, n, d, axes = 2, 3, 50, 17, 96, (32, 32, 32)
    thetas = (1e4,) * 3
    g = torch.Generator().manual_seed(5)
    idx = torch.randperm(N, generator=g)[:n].to(torch.int32).to(DEV)
    tok = idx.long().cpu()
    x = rows((B, H, N if si else n, d), torch.bfloat16, 6)
    y = rows((B, H, N if di else n, d), torch.bfloat16, 7)
    before = y.clone()
    pos = positions((1, N, 3), torch.int32, 8)
    sd().safedit_rope_rows([x], [y], pos, sd().rope_spec(axes, thetas), idx, n, si, di)
    expect_status(0)
    ref, mag = reference(x[:, :, tok] if si else x, pos[:, tok], axes, thetas, False, False)
    close(y[:, :, tok] if di else y, ref, mag)
    if di:
        keep = torch.ones(N, dtype=torch.bool)
        keep[tok] = False
        assert torch.equal(y[:, :, keep], before[:, :, keep])


def test_bad_indices_are_reported_and_skipped():
    n, N, d = 6, 20, 64
    idx = torch.tensor([3, -1, 19, 20, 2 ** 31 - 1, 0], dtype=torch.int32, device=DEV)
    x, y = rows((1, 2, n, d), torch.float16, 1), rows((1, 2, N, d), torch.float16, 2)
    before = y.clone()
    pos = positions((1, N, 1), torch.int32, 3)
    sd().safedit_rope_rows([x], [y], pos, sd().rope_spec((64,), (1e4,)), idx, n, False, True)
    expect_status(sd().ERR_INDEX)
    good, at = [0, 2, 5], [3, 19, 0]
    ref, mag = reference(x[:, :, good], pos[:, at], (64,), (1e4,), False, False)
    close(y[:, :, at], ref, mag)
    keep = [i for i in range(N) if i not in at]
    assert torch.equal(y[:, :, keep], before[:, :, keep])
    # the index check finds a token named twice
    old = sd().safedit_debug_set_index_check(True)
    try:
        twice = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
        sd().safedit_rope_rows([x[:, :, :2].contiguous()], [y], pos, sd().rope_spec((64,), (1e4,)), twice, 2, False, True)
        expect_status(sd().ERR_INDEX)
    finally:
        sd().safedit_debug_set_index_check(old)


def test_strided_views_and_in_place():
    """Q and K as views of a fused projection [B, n, 3, H, d] and broadcast positions, rotated in place; V stays."""
    B, H, n, d, axes, thetas = 2, 4, 33, 96, (32, 32, 32), (1e4,) * 3
    x = rows((B, n, 3, H, d), torch.bfloat16, 1)
    before = x.clone()
    q, k = (x[:, :, t].transpose(1, 2) for t in range(2))
    pos = positions((1, n, 3), torch.float32, 2).expand(B, n, 3)
    sd().safedit_rope_rows([q, k], [q, k], pos, sd().rope_spec(axes, thetas))
    expect_status(0)
    for t, got in ((0, q), (1, k)):
        close(got, *reference(before[:, :, t].transpose(1, 2), pos, axes, thetas, False, False))
    assert torch.equal(x[:, :, 2], before[:, :, 2])


def test_inverse_is_the_transpose_and_the_gradient():
    """<R x, y> = <x, R' y>, and R' y is the slope of <R x, y>: differences of a linear function are exact up to
    rounding, so each is held to the fp32 sums' 2^-18 of sum |x| |y|."""
    d, axes, thetas = 64, (24, 24), (1e4, 100.0)
    x, y = rows((1, 2, 19, d), torch.float32, 1), rows((1, 2, 19, d), torch.float32, 2)
    pos = positions((1, 19, 2), torch.int32, 3)
    for layout in (sd().ROPE_INTERLEAVED, sd().ROPE_HALVES):
        fwd = sd().rope_spec(axes, thetas, layout)
        back = sd().rope_spec(axes, thetas, layout, inverse=True)

        def turn(v, spec):
            o = torch.empty_like(v)
            sd().safedit_rope_rows([v], [o], pos, spec)
            return o
        rx, grad = turn(x, fwd), turn(y, back)
        scale = float((x.double().abs() * y.double().abs()).sum() + (rx.double().abs() * y.double().abs()).sum())
        assert abs(float((rx.double() * y.double()).sum() - (x.double() * grad.double()).sum())) <= 2.0 ** -18 * scale
        close(turn(rx, back), x.double().cpu(), 16 * torch.ones_like(x).double().cpu())
        for at in ((0, 1, 3, 5), (0, 0, 18, 47), (0, 1, 7, 60)):
            up, dn = x.clone(), x.clone()
            up[at] += 0.5
            dn[at] -= 0.5
            slope = ((turn(up, fwd).double() - turn(dn, fwd).double()) * y.double()).sum()
            assert abs(float(slope - grad[at].double())) <= 2.0 ** -18 * (8 + scale / 100)
        expect_status(0)


def test_streams_and_graph():
    B, H, n, d, axes, thetas = 1, 3, 40, 64, (32, 32), (1e4,) * 2
    x, pos = rows((B, H, n, d), torch.bfloat16, 1), positions((1, n, 2), torch.int32, 2)
    spec = sd().rope_spec(axes, thetas)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sd().safedit_rope_rows([x], [y], pos, spec, stream=side)
    side.synchronize()
    close(y, *reference(x, pos, axes, thetas, False, False))
    z = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd().safedit_rope_rows([x], [z], pos, spec)
    for seed in (3, 4):
        x.copy_(rows((B, H, n, d), torch.bfloat16, seed))
        pos.copy_(positions((1, n, 2), torch.int32, seed))
        graph.replay()
        torch.cuda.synchronize()
        close(z, *reference(x, pos, axes, thetas, False, False))
    expect_status(0)


def test_refusals_of_the_binding():
    x, pos, spec = rows((1, 1, 4, 64), torch.bfloat16, 1), positions((1, 4, 1), torch.int32, 1), sd().rope_spec((64,), (1e4,))
    for bad in (dict(src=[x.cpu()]), dict(pos=pos.cpu()), dict(dst=[x, x])):
        a = dict(src=[x], dst=[x.clone()], pos=pos, rope=spec)
        a.update(bad)
        with pytest.raises(sd().SafeditError):
            sd().safedit_rope_rows(**a)
    with pytest.raises(sd().SafeditError):  # an index of 64 bits
        sd().safedit_rope_rows([x], [x.clone()], pos, spec, torch.arange(4, device=DEV), 4, False, True)
    with pytest.raises(sd().SafeditError):  # shorter than it says
        sd().safedit_rope_rows([x], [x.clone()], pos, spec, torch.arange(3, device=DEV, dtype=torch.int32), 4, False, True)
    expect_status(0)


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart."""
    n, d = 3, 64
    step = (2 ** 31 + 2 ** 20) // d * d
    buf = torch.zeros(2 * step + n * d, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((1, 3, n, d), (0, step, d, 1))
    x.copy_(rows((1, 3, n, d), torch.bfloat16, 1))
    y = torch.empty((1, 3, n, d), dtype=torch.bfloat16, device=DEV)
    pos = positions((1, n, 1), torch.int32, 2)
    sd().safedit_rope_rows([x], [y], pos, sd().rope_spec((d,), (1e4,)))
    expect_status(0)
    close(y, *reference(x, pos, (d,), (1e4,), False, False))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("halves, axes", [(False, (20, 10)), (True, (24, 16))])
def test_elements_behind_the_last_axis_are_copies(dtype, halves, axes):
    """Infinities, NaN, the type's ends and zeros of both signs there stay where they are and reach no neighbour, wherever
    the rows lie and whatever their position."""
    d, n, end = 64, 32, sum(axes)
    f = torch.finfo(dtype)
    x = rows((1, 2, n, d), dtype, 3)
    special = torch.tensor([float("inf"), -0.0, float("nan"), 0.0, -float("inf"), f.max, f.tiny], dtype=dtype)
    take = torch.randint(0, 7, (1, 2, n, d - end), generator=torch.Generator().manual_seed(4))
    x[..., end:] = special[take].to(DEV)
    pos = positions((1, n, len(axes)), torch.float32, 5)
    pos[0, 3, 0] = float("inf")  # no position reaches them either
    y = torch.empty_like(x)
    sd().safedit_rope_rows([x], [y], pos, sd().rope_spec(axes, (1e4, 100.0), int(halves)))
    expect_status(0)
    got, want = y[..., end:].float().cpu(), x[..., end:].float().cpu()
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan].view(torch.int32), want[~nan].view(torch.int32))
    keep = [r for r in range(n) if r != 3]
    ref, mag = reference(x[:, :, keep, :end], pos[:, keep], axes, (1e4, 100.0), halves, False)
    close(y[:, :, keep, :end], ref, mag)
