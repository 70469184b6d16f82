"""The 8-bit state's store against its definition in 64 bits.

Rows of 16-bit types, not rotated: codes and scales are equal to the definition's, bit for bit (x qmax / m is rounded
once, and its product is exact).  Rotated rows and fp32 rows: the stored value code * scale is within half a step of the
row's value, where a step is 2^-3 of the value's binade for e4m3 (half of it: 2^-4 relative, 2^-10 scales for the
subnormal codes) and one scale for int8, plus 2^-19 of the block's largest magnitude for the fp32 arithmetic before the
rounding (rotation under 2^-21 (|a| + |b|), quotient and scale 2^-22 each).
"""
import pytest
import torch

from tests.gpu_util import expect_status, sd
from tests.test_gpu_rope import positions, reference, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


def e4m3_nearest(y):
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp(-6, 8) - 3)
    return torch.round(y / step) * step


def definition(x, kind, block):
    """x [B,H,n,d] fp64 -> (codes as numbers [B,H,nb*block,d], scales [B,H,nb]) in fp64."""
    top = CODES[kind][1]
    B, H, n, d = x.shape
    nb = -(-n // block)
    p = torch.zeros(B, H, nb * block, d, dtype=torch.float64)
    p[:, :, :n] = x
    p = p.view(B, H, nb, block, d)
    m = p.abs().amax((-1, -2))
    m = torch.where(m == 0, torch.full_like(m, top), m.clamp_min(2.0 ** -100))
    y = p * top / m[..., None, None]
    y = e4m3_nearest(y) if kind == "e4m3" else torch.round(y)
    return y.view(B, H, nb * block, d), m / top


def new_state(B, H, N, d, kind, block, fill=0x55):
    ty = CODES[kind][0]
    c = torch.full((B, H, N, d), fill, dtype=torch.uint8, device=DEV).view(ty)
    return c, torch.full((B, H, -(-N // block)), 3.5, device=DEV)


def raw(c):
    return c.view(torch.uint8).cpu()


def check_exact(c, f, x, kind, block, row0, before_c, before_f):
    N, n = c.shape[2], x.shape[2]
    y, sc = definition(x.double().cpu(), kind, block)
    nb = sc.shape[2]
    end = min(N, row0 + nb * block)
    assert torch.equal(c[:, :, row0:end].float().double().cpu(), y[:, :, : end - row0])
    assert torch.equal(f[:, :, row0 // block: row0 // block + nb].cpu(), sc.float())
    # everything else is as it was
    keep = torch.ones(N, dtype=torch.bool)
    keep[row0:end] = False
    assert torch.equal(raw(c)[:, :, keep], raw(before_c)[:, :, keep])
    kf = torch.ones(f.shape[2], dtype=torch.bool)
    kf[row0 // block: row0 // block + nb] = False
    assert torch.equal(f[:, :, kf].cpu(), before_f[:, :, kf].cpu())
    assert n <= nb * block


@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("block", (16, 32, 64, 128))
@pytest.mark.parametrize("d", (64, 96, 128))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float16))
def test_codes_and_scales_are_the_definitions(kind, block, d, dtype):
    for n, N, row0 in ((1, 1, 0), (1, 300, 128), (block, block, 0), (block + 1, 2 * block + 5, 0), (129, 400, 256),
                       (144, 400, 256)):
        x = [rows((2, h, n, d), dtype, n + h) for h in (3, 1)]
        st = [new_state(2, h, N, d, kind, block) for h in (3, 1)]
        old = [(c.clone(), f.clone()) for c, f in st]
        sd().safedit_state8_store(x, [c for c, _ in st], [f for _, f in st], block, row0)
        expect_status(0)
        for v, (c, f), (oc, of) in zip(x, st, old):
            check_exact(c, f, v, kind, block, row0, oc, of)


@pytest.mark.parametrize("kind", CODES)
def test_magnitudes(kind):
    """Zero blocks (scale 1), the smallest and largest magnitudes, wide blocks, ties between codes."""
    block, d, n = 16, 64, 16 * 8
    x = torch.zeros(1, 1, n, d)
    g = torch.Generator().manual_seed(1)
    for k, scale in enumerate((0.0, 1e-38, 1e-30, 1e-10, 1.0, 1e30, 3e38)):
        x[:, :, 16 * k: 16 * k + 16] = (torch.rand(16, d, generator=g) * 2 - 1) * scale
    # ties: multiples of half a step of int8 and of e4m3 when the largest magnitude is qmax
    top = CODES[kind][1]
    x[0, 0, 112:] = (torch.arange(16 * d).view(16, d) % 128 - 64) * 0.5
    x[0, 0, 112, 0] = top
    x = x.to(torch.bfloat16).to(DEV)
    c, f = new_state(1, 1, n, d, kind, block)
    oc, of = c.clone(), f.clone()
    sd().safedit_state8_store([x], [c], [f], block)
    expect_status(0)
    check_exact(c, f, x, kind, block, 0, oc, of)
    assert float(f[0, 0, 0]) == 1.0


@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("halves, d, axes", [(False, 96, (32, 32, 32)), (False, 64, (20, 30)), (True, 128, (16, 56, 56)),
                                             (True, 64, (8, 24)), (False, 128, (128,))])
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_rotated_rows(kind, halves, d, axes, dtype):
    thetas = (1e6, 1e4, 1e4)[: len(axes)]
    spec = sd().rope_spec(axes, thetas, sd().ROPE_HALVES if halves else sd().ROPE_INTERLEAVED)
    for block, n, N, row0 in ((16, 37, 100, 16), (64, 200, 200, 0), (128, 130, 300, 0), (32, 1, 33, 32)):
        k, v = rows((2, 2, n, d), dtype, 1), rows((2, 2, n, d), dtype, 2)
        pos = positions((2, n, len(axes)), torch.int32, 3)
        (kc, kf), (vc, vf) = new_state(2, 2, N, d, kind, block), new_state(2, 2, N, d, kind, block)
        sd().safedit_state8_store([k, v], [kc, vc], [kf, vf], block, row0, rotate=(True, False), pos=pos, rope=spec)
        expect_status(0)
        turned, _ = reference(k, pos, axes, thetas, halves, False)
        for want, c, f in ((turned, kc, kf), (v.double().cpu(), vc, vf)):
            sc = f.double().cpu().repeat_interleave(block, 2)[:, :, row0: row0 + n, None]
            got = c.float().double().cpu()[:, :, row0: row0 + n] * sc
            top = CODES[kind][1]
            half = torch.maximum(want.abs() * 2.0 ** -4, sc * 2.0 ** -10) if kind == "e4m3" else sc / 2
            assert bool(((got - want).abs() <= half * (1 + 2.0 ** -18) + 2.0 ** -19 * top * sc).all())
            _, def_sc = definition(want, kind, block)
            nb = def_sc.shape[2]
            have = f.double().cpu()[:, :, row0 // block: row0 // block + nb]
            assert bool(((have - def_sc).abs() <= 2.0 ** -20 * def_sc).all())
            end = min(N, row0 + nb * block)
            assert int(raw(c)[:, :, row0 + n: end].ne(0).sum()) == 0


def test_gathered_rows_strided_views_and_rotation_by_token():
    """Rows gathered from a fused projection's views by token, rotated at those tokens, blocks elsewhere untouched."""
    B, H, N, n, d, block = 2, 3, 90, 41, 96, 32
    x = rows((B, N, 2, H, d), torch.bfloat16, 1)
    k, v = (x[:, :, t].transpose(1, 2) for t in range(2))
    idx = torch.randperm(N, generator=torch.Generator().manual_seed(2))[:n].to(torch.int32).to(DEV)
    tok = idx.long().cpu()
    (kc, kf), (vc, vf) = new_state(B, H, 150, d, "int8", block), new_state(B, H, 150, d, "int8", block)
    oc, of = vc.clone(), vf.clone()
    pos = positions((1, N, 3), torch.float32, 3)
    axes, thetas = (32, 32, 32), (1e4,) * 3
    sd().safedit_state8_store([k, v], [kc, vc], [kf, vf], block, 64, idx, n, True, (True, False), pos,
                              sd().rope_spec(axes, thetas))
    expect_status(0)
    check_exact(vc, vf, v.cpu()[:, :, tok], "int8", block, 64, oc, of)
    turned, _ = reference(k.cpu()[:, :, tok], pos.cpu()[:, tok], axes, thetas, False, False)
    sc = kf.double().cpu().repeat_interleave(block, 2)[:, :, 64: 64 + n, None]
    got = kc.double().cpu()[:, :, 64: 64 + n] * sc
    assert bool(((got - turned).abs() <= sc / 2 * (1 + 2.0 ** -18) + 2.0 ** -19 * 127 * sc).all())


@pytest.mark.parametrize("kind", CODES)
def test_values_that_are_not_finite(kind):
    """Reported; NaN is stored as 0 and infinities as the largest codes, the finite elements as if they were alone."""
    x = rows((1, 1, 40, 64), torch.bfloat16, 1)
    x[0, 0, 3, 5], x[0, 0, 3, 6], x[0, 0, 4, 0] = float("nan"), float("inf"), -float("inf")
    x[0, 0, 32:, :] = float("inf")
    clean = x.clone()
    clean[0, 0, 3, 5] = clean[0, 0, 3, 6] = clean[0, 0, 4, 0] = 0
    c, f = new_state(1, 1, 40, 64, kind, 16)
    sd().safedit_state8_store([x], [c], [f], 16)
    expect_status(sd().ERR_INVALID_ARG)
    y, sc = definition(clean[:, :, :32].double().cpu(), kind, 16)
    top = CODES[kind][1]
    y[0, 0, 3, 6], y[0, 0, 4, 0] = top, -top
    assert torch.equal(c[:, :, :32].float().double().cpu(), y)
    assert torch.equal(f[:, :, :2].cpu(), sc.float())
    assert bool((c[:, :, 32:].float() == top).all()) and float(f[0, 0, 2]) == 1.0


def test_bad_indices_store_zero_rows():
    x = rows((1, 2, 30, 64), torch.bfloat16, 1)
    idx = torch.tensor([2, 30, -5, 7], dtype=torch.int32, device=DEV)
    c, f = new_state(1, 2, 32, 64, "e4m3", 16)
    oc, of = c.clone(), f.clone()
    sd().safedit_state8_store([x], [c], [f], 16, 0, idx, 4, True)
    expect_status(sd().ERR_INDEX)
    want = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    want[:, :, 0], want[:, :, 3] = x.cpu()[:, :, 2], x.cpu()[:, :, 7]
    check_exact(c, f, want, "e4m3", 16, 0, oc, of)


def test_streams_and_graph():
    x = rows((1, 2, 50, 96), torch.float16, 1)
    c, f = new_state(1, 2, 64, 96, "int8", 32)
    oc, of = c.clone(), f.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sd().safedit_state8_store([x], [c], [f], 32, stream=side)
    side.synchronize()
    check_exact(c, f, x, "int8", 32, 0, oc, of)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd().safedit_state8_store([x], [c], [f], 32)
    for seed in (5, 6):
        x.copy_(rows((1, 2, 50, 96), torch.float16, seed))
        graph.replay()
        torch.cuda.synchronize()
        check_exact(c, f, x, "int8", 32, 0, oc, of)
    expect_status(0)


def test_offsets_past_32_bits():
    """State rows of heads more than 2^32 bytes apart."""
    n, d = 20, 64
    step = (2 ** 32 + 2 ** 20) // d * d
    buf = torch.zeros(step + 32 * d, dtype=torch.int8, device=DEV)
    c = buf.as_strided((1, 2, 32, d), (0, step, d, 1))
    f = torch.zeros(1, 2, 2, device=DEV)
    oc, of = c.clone(), f.clone()
    x = rows((1, 2, n, d), torch.bfloat16, 1)
    sd().safedit_state8_store([x], [c], [f], 16)
    expect_status(0)
    check_exact(c.contiguous(), f, x, "int8", 16, 0, oc, of)


def test_a_value_that_is_not_finite_stays_alone():
    """An infinity behind the last axis is reported and saturates; its neighbours' codes are what they are without it."""
    B, H, n, d, axes = 1, 2, 64, 64, (20, 10)
    x = rows((B, H, n, d), torch.bfloat16, 8)
    pos, spec = positions((1, n, 2), torch.int32, 9), sd().rope_spec(axes, (1e4, 1e4))
    x[0, 0, 5, 40] = 50.0  # the block's largest
    x[0, 0, 7, 31] = x[0, 1, 9, 60] = 0.0
    at = torch.zeros(B, H, n, d, dtype=torch.bool)
    at[0, 0, 7, 31] = at[0, 1, 9, 60] = True
    out = []
    for value, status in ((0.0, 0), (float("inf"), sd().ERR_INVALID_ARG)):
        x[at.to(DEV)] = value
        c, f = new_state(B, H, n, d, "int8", 64)
        sd().safedit_state8_store([x], [c], [f], 64, rotate=[True], pos=pos, rope=spec)
        expect_status(status)
        out.append((raw(c), f.cpu()))
    assert torch.equal(out[0][1], out[1][1])
    assert torch.equal(out[0][0][~at], out[1][0][~at])
    assert bool((out[1][0][at] == 127).all())


def test_an_index_that_nothing_reads():
    """Compact rows that are not rotated: only the index' length counts."""
    x = rows((1, 2, 40, 64), torch.float16, 3)
    c, f = new_state(1, 2, 64, 64, "e4m3", 16)
    c0, f0 = c.clone(), f.clone()
    sd().safedit_state8_store([x], [c], [f], 16, idx=torch.full((40,), -5, dtype=torch.int32, device=DEV), n_idx=40)
    expect_status(0)
    check_exact(c, f, x, "e4m3", 16, 0, c0, f0)
