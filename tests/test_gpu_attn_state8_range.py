"""Attention over the 8-bit state where the scales of V, the pads and the codes are of every size the interface admits.

Tolerance, per element, with A = sum_j p_j |v_j| and S = max_j(p_j) sum_j |v_j| in fp64:
  |got - out| <= 2^-8 |out| + (2^-11 + 2^-12) A + 2^-23 S
  - the result is rounded once to bf16: half a step, 2^-8 of the value;
  - every weight is rounded to f16 or finer (half a step, 2^-11 relative): at most 2^-11 A;
  - f16's steps stop shrinking at 2^-14, where half a step is 2^-25.  The row's largest weight is 2^6 or more and an f16
    weight belongs to a scale no further than 2^8 below the largest: 2^-25 2^-6 2^8 max(p) of each |v|;
  - scores of N(0,1) rows: under 2^-12 A (as in the tests of the ordinary range).
Every term goes by the element's own values, so a row or a channel that lost its share of the sum is seen whatever
the others hold.
"""
import math

import pytest
import torch

from tests.gpu_util import expect_status, sd
from tests.test_gpu_attn_state8 import BF, CODES, DEV, dense, padded, run, state
from tests.test_gpu_rope import rows

pytestmark = pytest.mark.gpu
# rows of a call: one, two tiles of the kernel for few rows, both query tiles on the same rows, units of 256
COUNTS = (1, 12, 40, 300)


def attended(q, st, block, pad=None, scale=None):
    """(out, A, S) in fp64."""
    (k8, ks), (v8, vs) = st
    k, v = dense(k8, ks, block), dense(v8, vs, block)
    t = q.double().cpu() @ k.transpose(2, 3) * (q.shape[-1] ** -0.5 if scale is None else scale)
    if pad is not None:
        dead = pad.cpu() == -math.inf
        t = t + pad.double().cpu()[:, None, None, :]
        t = torch.where(dead[:, None, None, :], torch.full_like(t, -math.inf), t)
        v = torch.where(dead[:, None, :, None], torch.zeros_like(v), v)
    p = torch.softmax(t, -1)
    return p @ v, p @ v.abs(), p.amax(-1, keepdim=True) * v.abs().sum(2, keepdim=True)


def bound(out, A, S):
    return 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -12) * A + 2.0 ** -23 * S


def close(got, out, A, S):
    err, most = (got.double().cpu() - out).abs(), bound(out, A, S)
    assert bool((err <= most).all()), f"worst error/bound {float((err / most.clamp_min(1e-300)).max()):.3g}"


def scaled(B, H, N, d, kind, block, seed, power):
    """Codes and scales of N(0, 4^power) rows."""
    codes, scales = state(B, H, N, d, kind, block, seed)
    return codes, scales * 2.0 ** power


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("live, masked", ((-30.0, 2.0 ** 30), (30.0, 2.0 ** -40), (0.0, 2.0 ** 31)))
def test_masked_blocks_beside_scales_of_another_size(n, kind, live, masked):
    """A masked block's scales count for nothing whatever they are: ordinary values too, in tiles with live keys."""
    B, H, N, d, block = 1, 2, 600, 64, 16
    st = state(B, H, N, d, kind, block, 1), scaled(B, H, N, d, kind, block, 2, live)
    q = rows((B, H, n, d), BF, 3)
    pad = padded(B, N)
    dead = [0, 3, 4, 17, 24, 25, 26, 27, 28, 29, 30, 31, 37]
    for i in dead:
        pad[:, i * block: (i + 1) * block] = -math.inf
    want = attended(q, st, block, pad)
    for _, f in st:
        f[:, :, dead] = masked
    close(run(q, st, block, pad=pad), *want)


# (rows, heads, keys): whole, over a cluster's blocks, in parts; both query tiles on the same rows whole and in parts;
# units of 256 rows whole and with the last ones in parts
PLANS = ((1, 2, 300), (12, 2, 300), (1, 3, 4000), (9, 40, 3000), (1, 1, 30000), (20, 1, 30000), (40, 2, 200),
         (100, 2, 6000), (300, 2, 600), (300, 2, 9000))


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("masked", (False, True))
def test_a_query_row_of_nan(n, H, N, kind, masked):
    """It comes out as NaN with no status in every plan, and the other rows as if it were not there."""
    d, block = 96, 64
    st = state(1, H, N, d, kind, block, 1), state(1, H, N, d, kind, block, 2)
    q = rows((1, H, n, d), BF, 3)
    pad = None
    if masked:
        pad = padded(1, N)
        pad[:, N // 5: N // 3] = -math.inf
        pad[:, N - N // 4:] = -math.inf
    want = attended(q, st, block, pad)
    bad = n // 2
    q[:, :, bad, 5] = math.nan
    got = run(q, st, block, pad=pad)
    assert bool(got[:, :, bad].isnan().all())
    keep = [r for r in range(n) if r != bad]
    close(got[:, :, keep], *(x[:, :, keep] if x.shape[2] == n else x for x in want))


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("where", ("k", "v", "k beside pads", "v beside pads", "pad", "pad of inf"))
def test_nan_codes_and_pads_are_reported(n, H, N, where):
    """One NaN code of a key that is not masked, or one pad that is no number, in every plan; under -inf it is nothing."""
    d, block = 96, 64
    st = state(1, H, N, d, "e4m3", block, 1), state(1, H, N, d, "e4m3", block, 2)
    q = rows((1, H, n, d), BF, 3)
    pad = None
    if "pad" in where:
        pad = padded(1, N)
        pad[:, N // 5: N // 3] = -math.inf
    at = N // 2
    if where.startswith("pad"):
        pad[0, at] = math.inf if "inf" in where else math.nan
    else:
        st["kv".index(where[0])][0].view(torch.uint8)[0, 0, at, 11] = 0xFF
    run(q, st, block, pad=pad, status=sd().ERR_INVALID_ARG)
    if pad is not None:
        pad[0, at] = -math.inf
        clean = [(c.float().nan_to_num(0.0), f) for c, f in st]
        close(run(q, st, block, pad=pad), *attended(q, clean, block, pad))


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("power", (-60, -24, 40))
@pytest.mark.parametrize("far", (-1e9, 1e9, torch.finfo(torch.float32).min))
def test_far_pads_on_every_key_and_v_of_another_size(n, kind, power, far):
    """Pads that absorb the scores absorb no scale of V: the row is the mean of V, whatever its size."""
    B, H, N, d, block = 1, 2, 700, 64, 16
    st = state(B, H, N, d, kind, block, 1), scaled(B, H, N, d, kind, block, 2, power)
    q = rows((B, H, n, d), BF, 3)
    pad = padded(B, N)
    pad[:] = far
    v = dense(*st[1], block)
    # scores under 2^6 against a step of 2^7 of the pad in log2 units: nothing of them is left
    want = [x.mean(2, keepdim=True).expand(B, H, n, d) for x in (v, v.abs(), v.abs())]
    close(run(q, st, block, pad=pad), *want)


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("power", (-117, -100, 100, 120))
@pytest.mark.parametrize("masked", (False, True))
def test_v_near_the_ends_of_fp32(n, H, N, kind, power, masked):
    """The row sums neither overflow nor vanish where every scale of V is tiny or huge."""
    d, block = 96, 64
    st = state(1, H, N, d, kind, block, 1), scaled(1, H, N, d, kind, block, 2, power)
    q = rows((1, H, n, d), BF, 3)
    pad = None
    if masked:
        pad = padded(1, N)
        pad[:, N // 5: N // 3] = -math.inf
    close(run(q, st, block, pad=pad), *attended(q, st, block, pad))


def stored(x, kind, block):
    """Codes and scales of x [B,H,N,d] as the store writes them."""
    B, H, N, d = x.shape
    codes = torch.zeros(B, H, N, d, dtype=torch.uint8, device=DEV).view(CODES[kind][0])
    scales = torch.zeros(B, H, -(-N // block), device=DEV)
    sd().safedit_state8_store([x], [codes], [scales], block)
    expect_status(0)
    return codes, scales


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("kind, d, block", (("e4m3", 96, 32), ("int8", 64, 16), ("e4m3", 128, 64), ("int8", 96, 128)))
@pytest.mark.parametrize("size", (1e-3, 1e-5, 3e-7, 1e-12, 1e-22))
@pytest.mark.parametrize("zeros", ((0,), (3,), (0, 5)))
@pytest.mark.parametrize("masked", (False, True))
def test_small_rows_beside_blocks_of_zeros(n, kind, d, block, size, zeros, masked):
    """Stored and attended: a block of zeros has the scale 1, which takes nothing from rows of 1e-3 to 1e-22 (nor does
    the bound: a result of zeros is outside it nearly everywhere)."""
    B, H, N = 1, 2, 1000
    q, k = rows((B, H, n, d), BF, 1), rows((B, H, N, d), BF, 2)
    v = (rows((B, H, N, d), BF, 3).float() * size).to(BF)
    for i in zeros:
        v[:, :, i * block: (i + 1) * block] = 0.0
    st = stored(k, kind, block), stored(v, kind, block)
    assert bool((st[1][1][:, :, list(zeros)] == 1.0).all())
    pad = None
    if masked:
        pad = padded(B, N)
        pad[:, 100:900:3] = -math.inf
        pad[:, 2 * block: 3 * block] = -math.inf
    want = attended(q, st, block, pad)
    assert float((want[0].abs() > bound(*want)).double().mean()) > 0.95
    close(run(q, st, block, pad=pad), *want)


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("power", (17, 20, 40))
def test_one_outlier_of_v(n, H, N, kind, power):
    """One element of 2^17 and more lifts its block's scale: the other channels keep what the other blocks hold there."""
    d, block = 96, 32
    q, k, v = (rows((1, H, m, d), BF, s) for s, m in enumerate((n, N, N)))
    v[:, :, N // 3, 7] = 2.0 ** power
    st = stored(k, kind, block), stored(v, kind, block)
    want = attended(q, st, block)
    others = [c for c in range(d) if c != 7]
    # A result of zeros is seen.  Weights of N(0,1) scores have sum p^2 = e / N, so an element has the deviation
    # (e / N)^(1/2), 9.5e-3 at 30000 keys, and A = 0.8: the bound's 6e-4 hides 2 * 0.4 * 6e-4 / 9.5e-3 = 5% of them
    # there and less elsewhere.
    assert float((want[0].abs() > bound(*want))[..., others].double().mean()) > 0.9
    close(run(q, st, block), *want)


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind, d, block", (("e4m3", 96, 16), ("int8", 128, 32), ("e4m3", 64, 128), ("int8", 64, 64),
                                            ("e4m3", 128, 16)))
@pytest.mark.parametrize("order", ("random", "rising", "falling"))
@pytest.mark.parametrize("masked", (False, True))
def test_scales_over_the_whole_range(n, H, N, kind, d, block, order, masked):
    """Blocks of V from 2^-30 to 2^30, in any order, each channel in use by one size of block alone, so that it shows
    whether the small ones' shares are kept beside the large ones'."""
    st = state(1, H, N, d, kind, block, 1), state(1, H, N, d, kind, block, 2)
    (_, _), (v8, vs) = st
    nb = vs.shape[2]
    power = torch.linspace(-30.0, 30.0, nb) if nb > 1 else torch.zeros(1)
    if order == "random":
        power = power[torch.randperm(nb, generator=torch.Generator().manual_seed(nb))]
    elif order == "falling":
        power = power.flip(0)
    vs *= torch.exp2(power.round()).to(DEV)
    mine = ((power + 30.0) / 60.0 * d).long().clamp(0, d - 1)  # the channel from which on a block holds zeros
    keep = torch.arange(d)[None, :] <= mine[:, None]
    keep &= torch.arange(d)[None, :] > mine[:, None] - max(2, d // 8)
    codes = v8.view(torch.uint8)
    codes *= keep.to(DEV).repeat_interleave(block, 0)[:N].to(torch.uint8)
    q = rows((1, H, n, d), BF, 3)
    pad = None
    if masked:
        pad = padded(1, N)
        pad.copy_(-torch.rand(1, N, generator=torch.Generator().manual_seed(3)))
        pad[:, N // 5: N // 3] = -math.inf
        pad[:, 1::5] = -math.inf
    close(run(q, st, block, pad=pad), *attended(q, st, block, pad))


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("order", ("rising", "falling"))
def test_far_pads_and_scales_over_the_whole_range(n, kind, order):
    """Where pads absorb every score the weights are the scales alone: the row is the mean of V still."""
    B, H, N, d, block = 1, 2, 700, 64, 16
    st = state(B, H, N, d, kind, block, 1), state(B, H, N, d, kind, block, 2)
    vs = st[1][1]
    power = torch.linspace(-30.0, 30.0, vs.shape[2]).round()
    vs *= torch.exp2(power if order == "rising" else power.flip(0)).to(DEV)
    q = rows((B, H, n, d), BF, 3)
    pad = padded(B, N)
    pad[:] = -1e9
    v = dense(*st[1], block)
    close(run(q, st, block, pad=pad), *(x.mean(2, keepdim=True).expand(B, H, n, d) for x in (v, v.abs(), v.abs())))


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("power", (-40, 0, 40))
def test_far_pads_and_parts_that_start_at_different_scales(n, H, N, kind, power):
    """Sums of a row that begin at scales of another size are joined as exactly under a far pad as without one."""
    d, block = 96, 16
    st = state(1, H, N, d, kind, block, 1), state(1, H, N, d, kind, block, 2)
    vs = st[1][1]
    vs *= torch.exp2(torch.randint(-3, 4, vs.shape, generator=torch.Generator().manual_seed(3)).float() + power).to(DEV)
    q = rows((1, H, n, d), BF, 3)
    pad = padded(1, N)
    pad[:] = -1e9
    v = dense(*st[1], block)
    close(run(q, st, block, pad=pad), *(x.mean(2, keepdim=True).expand(1, H, n, d) for x in (v, v.abs(), v.abs())))


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("size", (1e3, 1e5, 1e7, 1e9))
@pytest.mark.parametrize("masked", (False, True))
def test_scores_far_beyond_the_exponents_steps(n, H, N, kind, size, masked):
    """Scores of 1e3 to 1e9: a key that leads the others of its row by more than fp32 leaves uncertain has all of the
    weight (no weight leaves f16's range on the way), and every row stays within what V holds."""
    d, block = 96, 64
    st = state(1, H, N, d, kind, block, 1), state(1, H, N, d, kind, block, 2)
    q = (rows((1, H, n, d), BF, 3).float() * size).to(BF)
    pad = None
    if masked:
        pad = padded(1, N)
        pad[:, N // 5: N // 3] = -math.inf
    got = run(q, st, block, pad=pad).double().cpu()
    k, v = dense(*st[0], block), dense(*st[1], block)
    t = q.double().cpu() @ k.transpose(2, 3) * d ** -0.5
    if pad is not None:
        t = t.masked_fill(pad.cpu()[:, None, None, :] == -math.inf, -math.inf)
    two, at = t.topk(2, -1)
    # a score's products and their sum in fp32: 96 terms of 4 size each, 2^-24 of their absolute sum, twice over; and the
    # exponent's sum, 2^-24 of the score.  40 beyond that leaves e^-40 N.
    sure = two[..., 0] - two[..., 1] > 40.0 + 2.0 ** -22 * (96 * 4 * size * d ** -0.5 + two[..., 0].abs())
    assert bool(sure.any()) or size < 1e5
    best = v.gather(2, at[..., :1].expand(1, H, n, d))
    # the key's weight is rounded to f16 where the row's sum has it in fp32: 2^-11, then the result to bf16
    assert bool(((got - best).abs() <= (2.0 ** -8 + 2.0 ** -11 * (1 + 2.0 ** -8)) * best.abs() + 1e-12)[sure].all())
    assert bool((got.abs() <= 1.01 * v.abs().amax(2, keepdim=True)).all())


@pytest.mark.parametrize("n", COUNTS)
def test_k_scales_of_zero_beside_v_scales_of_every_size(n):
    """K of zeros (k_scale 0 too): every key counts alike, whatever the scales of V."""
    B, H, N, d, block = 1, 2, 700, 64, 16
    st = state(B, H, N, d, "e4m3", block, 1), state(B, H, N, d, "e4m3", block, 2)
    st[0][1].zero_()
    vs = st[1][1]
    vs *= torch.exp2(torch.linspace(-30.0, 30.0, vs.shape[2]).flip(0).round()).to(DEV)
    q = rows((B, H, n, d), BF, 3)
    q[:, :, 0] = 0.0
    close(run(q, st, block), *attended(q, st, block))


@pytest.mark.parametrize("n, H, N", ((1, 300, 2000), (12, 44, 6000), (40, 3, 2000), (100, 3, 2000), (300, 3, 2000)))
@pytest.mark.parametrize("kind", ("e4m3", "int8"))
@pytest.mark.parametrize("masked", (False, True))
def test_waits_that_run_out_among_wide_keys(n, H, N, kind, masked):
    """With no time to wait every role gives up on tiles of small V scales too: reported, and the next call gives the
    first one's bits."""
    d, block = 96, 64
    st = state(1, H, N, d, kind, block, 1), state(1, H, N, d, kind, block, 2)
    st[1][1][:, :, ::3] *= 2.0 ** 20
    q = rows((1, H, n, d), BF, 3)
    pad = None
    if masked:
        pad = padded(1, N)
        pad[:, 5::7] = -math.inf
    first = run(q, st, block, pad=pad)
    old = sd().safedit_debug_set_wait_limit_ns(0)
    try:
        run(q, st, block, pad=pad, status=sd().ERR_TIMEOUT)
    finally:
        sd().safedit_debug_set_wait_limit_ns(old)
    again = run(q, st, block, pad=pad)
    assert torch.equal(first, again)
    close(again, *attended(q, st, block, pad))


@pytest.mark.parametrize("n", COUNTS)
def test_wide_keys_in_two_graphs_with_workspaces_of_their_own(n):
    """Captured and replayed in turn on new inputs, wide and ordinary slices beside each other."""
    B, H, N, d, block = 1, 3, 3000, 64, 32
    sets = []
    for s in (1, 2):
        st = state(B, H, N, d, "e4m3", block, s), state(B, H, N, d, "e4m3", block, s + 5)
        st[1][1][:, s, 7::9] *= 2.0 ** 18
        q = rows((B, H, n, d), BF, s)
        out = torch.zeros(B, H, n, d, dtype=BF, device=DEV)
        size = sd().safedit_attn_subset_state8_workspace_size(B, H, n, N, d)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
        (k8, ks), (v8, vs) = st
        call = lambda q=q, k8=k8, ks=ks, v8=v8, vs=vs, out=out, ws=ws: sd().safedit_attn_subset_state8(  # noqa: E731
            q, k8, ks, v8, vs, block, None, 0, None, 0.0, out, 0, ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((q, st, out, graph))
    for q, st, out, graph in sets:
        q.copy_(q.flip(2) * 0.5)
        st[1][1].copy_(st[1][1].flip(2))
        out.zero_()
    for _ in range(2):
        for *_, graph in sets:
            graph.replay()
    torch.cuda.synchronize()
    expect_status(0)
    for q, st, out, _ in sets:
        close(out, *attended(q, st, block))


@pytest.mark.parametrize("n, H, N", PLANS)
@pytest.mark.parametrize("power, status", ((-78, 0), (-88, 1), (88, 0), (100, 1)))
def test_how_far_a_scale_of_one_may_lie_off(n, H, N, power, status):
    """A block of zeros (scale 1) within 2^88 of the others takes nothing from them; farther off it is reported."""
    d, block = 96, 64
    st = state(1, H, N, d, "e4m3", block, 1), scaled(1, H, N, d, "e4m3", block, 2, power)
    codes, scales = st[1]
    codes.view(torch.uint8)[:, :, block: 2 * block] = 0
    scales[:, :, 1] = 1.0
    q = rows((1, H, n, d), BF, 3)
    if status:
        run(q, st, block, status=sd().ERR_INVALID_ARG)
    else:
        close(run(q, st, block), *attended(q, st, block))
