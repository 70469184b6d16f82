"""Attention over the 8-bit state against its definition in 64 bits on the stored codes and scales.

Tolerance, per element, with A = sum_j p_j |v_j| (the weights' mean of |v|) in fp64:
  |got - out| <= 2^-8 |out| + (2^-11 + 2^-12) A + 2^-25 M
  - the result is rounded once to bf16: half a step, 2^-8 of the value;
  - every weight is rounded once to f16 (half a step, 2^-11 relative): at most 2^-11 A;
  - f16's steps stop shrinking at 2^-14: there half a step is 2^-25.  A weight is p_j vs_j over the row's largest (or a
    smaller reference), so each may be off by 2^-25 max_j(p_j vs_j), times |code_j|: M = max_j(p_j vs_j) sum_j |code_j|.
    It shows where one key has nearly all the weight and its code is 0 (a row of 16 keys with p = 0.99997 and the
    others at 1e-6 did);
  - scores of N(0,1) rows: fp32 products and sums leave under 2^-14 of a log2 unit, exp2 (hardware or a polynomial of
    7.5e-5 relative error) under 2^-13: together under 2^-12 A.
"""
import math

import pytest
import torch

from tests.gpu_util import expect_status, sd
from tests.test_gpu_rope import positions, reference as turn_reference, rows
from tests.test_gpu_state8 import CODES, definition

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def state(B, H, N, d, kind, block, seed, spread=0.0):
    """Codes and scales of N(0,1) rows; spread: log2 of how far the blocks' magnitudes vary."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, N, d, generator=g).double()
    nb = -(-N // block)
    if spread:
        f = torch.exp2((torch.rand(B, H, nb, generator=g).double() - 0.5) * spread)
        x = x * f.repeat_interleave(block, 2)[:, :, :N, None]
    y, sc = definition(x, kind, block)
    return y[:, :, :N].float().to(CODES[kind][0]).to(DEV), sc.float().to(DEV)


def dense(c, f, block):
    return c.float().double().cpu() * f.double().cpu().repeat_interleave(block, 2)[:, :, : c.shape[2], None]


def attend(q, st, block, idx, pad, scale=None):
    """(out, A with the term of the f16 weights' smallest step) in fp64; rows without a key are zeros."""
    (k8, ks), (v8, vs) = st
    k, v = dense(k8, ks, block), dense(v8, vs, block)
    vf = vs.double().cpu().repeat_interleave(block, 2)[:, :, : v.shape[2]]
    code = v8.float().double().cpu().abs()
    q = q.double().cpu()
    if idx is not None:
        q = q[:, :, idx.long().cpu()]
    t = q @ k.transpose(2, 3) * (q.shape[-1] ** -0.5 if scale is None else scale)
    if pad is not None:
        dead = pad.cpu() == -math.inf
        t = t + pad.double().cpu()[:, None, None, :]
        t = torch.where(dead[:, None, None, :], torch.full_like(t, -math.inf), t)
        v, code = (torch.where(dead[:, None, :, None], torch.zeros_like(x), x) for x in (v, code))
        vf = torch.where(dead[:, None, :], torch.zeros_like(vf), vf)
    p = torch.softmax(t, -1).nan_to_num(0.0)
    M = (p * vf[:, :, None, :]).amax(-1, keepdim=True) * code.sum(2, keepdim=True)
    return p @ v, p @ v.abs() + M * 2.0 ** -25 / (2.0 ** -11 + 2.0 ** -12)


def workspace(B, H, n, N, d):
    size = sd().safedit_attn_subset_state8_workspace_size(B, H, n, N, d)
    return torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if size else None


def close(got, out, A, what=""):
    err = (got.double().cpu() - out).abs()
    bound = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -12) * A
    assert bool((err <= bound).all()), f"{what}: worst error/bound {float((err / bound.clamp_min(1e-300)).max()):.2f}"


def padded(B, N, seed=0):
    """A [B, N] view whose rows start at 16 bytes."""
    return torch.zeros(B, -(-N // 4) * 4, device=DEV)[:, :N]


def run(q, st, block, idx=None, pad=None, scale=0.0, scattered=False, out=None, status=0):
    (k8, ks), (v8, vs) = st
    B, H, N, d = k8.shape
    n = q.shape[2] if idx is None else idx.numel()
    if out is None:
        out = torch.full((B, H, q.shape[2] if scattered else n, d), 7.0, dtype=BF, device=DEV)
    sd().safedit_attn_subset_state8(q, k8, ks, v8, vs, block, idx, n, pad, scale, out, int(scattered),
                                    workspace(B, H, n, N, d))
    expect_status(status)
    return out


@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("d", (64, 96, 128))
@pytest.mark.parametrize("block", (16, 32, 64, 128))
def test_rows_and_keys(kind, d, block):
    """Row counts around the tiles' edges against key counts around theirs."""
    B, H = 2, 2
    for N in (1, 15, 16, 17, 127, 128, 129, 700):
        st = state(B, H, N, d, kind, block, N), state(B, H, N, d, kind, block, N + 1)
        for n in (1, 2, 16, 17, 33, 128, 129, 257):
            q = rows((B, H, n, d), BF, n)
            close(run(q, st, block), *attend(q, st, block, None, None), what=f"N={N} n={n}")


@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("n", (1, 13, 100, 300))
def test_long_keys(kind, n):
    B, H, N, d, block = 1, 2, 9001, 96, 64
    st = state(B, H, N, d, kind, block, 1), state(B, H, N, d, kind, block, 2)
    q = rows((B, H, 400, d), BF, 3)
    idx = torch.randperm(400, generator=torch.Generator().manual_seed(4))[:n].to(torch.int32).to(DEV)
    close(run(q, st, block, idx), *attend(q, st, block, idx, None))


@pytest.mark.parametrize("n", (1, 9, 130, 270))
@pytest.mark.parametrize("scale", (0.0, 0.03, 0.5))
def test_scattered_rows_scale_and_views(n, scale):
    """Unsorted rows scattered into a state whose other rows stay; Q a view of a fused projection, K and V codes of one
    buffer."""
    B, H, N, Nq, d, block = 2, 3, 333, 300, 64, 32
    x = rows((B, Nq, 3, H, d), BF, 1)
    q = x[:, :, 1].transpose(1, 2)
    both = torch.empty(B, N, 2, H, d, dtype=torch.int8, device=DEV)
    k8, v8 = (both[:, :, t].transpose(1, 2) for t in range(2))
    (kc, ks), (vc, vs) = state(B, H, N, d, "int8", block, 1), state(B, H, N, d, "int8", block, 2)
    k8.copy_(kc)
    v8.copy_(vc)
    idx = torch.randperm(Nq, generator=torch.Generator().manual_seed(4))[:n].to(torch.int32).to(DEV)
    out = rows((B, H, Nq, d), BF, 9)
    before = out.clone()
    run(q, ((k8, ks), (v8, vs)), block, idx, None, scale, True, out)
    want, A = attend(q, ((kc, ks), (vc, vs)), block, idx, None, scale or None)
    # a larger scale stretches the scores' error with it: 2^-14 units at 1/sqrt(d) = 1/8
    close(out[:, :, idx.long()], want, A * (4 if scale == 0.5 else 1))
    keep = torch.ones(Nq, dtype=torch.bool, device=DEV)
    keep[idx.long()] = False
    assert torch.equal(out[:, :, keep], before[:, :, keep])


@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("n", (1, 20, 150, 260))
@pytest.mark.parametrize("N", (5, 130, 1000))
def test_key_pad(kind, n, N):
    """Soft pads, -inf tails and holes, the type's lowest value beside ordinary ones; NaN codes and NaN scales under
    -inf do not show."""
    B, H, d, block = 3, 2, 96, 16
    st = state(B, H, N, d, kind, block, 1), state(B, H, N, d, kind, block, 2)
    pad = padded(B, N)
    pad.copy_(-torch.rand(B, N, generator=torch.Generator().manual_seed(3)))
    pad[0, N - N // 3:] = -math.inf
    pad[1, : N // 2] = -math.inf
    pad[2, 1::2] = torch.finfo(torch.float32).min
    q = rows((B, H, n, d), BF, 4)
    want, A = attend(q, st, block, None, pad)
    close(run(q, st, block, pad=pad), want, A)
    # whatever masked keys hold
    for c, f in st:
        off = (pad == -math.inf)
        c.view(torch.uint8).masked_fill_(off[:, None, :, None], 0x7F if kind == "e4m3" else 0x80)
        nb = f.shape[2]
        dead = torch.nn.functional.pad(off, (0, nb * block - N), value=True).view(B, nb, block).all(-1)
        f.masked_fill_(dead[:, None, :], float("nan"))
    close(run(q, st, block, pad=pad), want, A, "masked garbage")


@pytest.mark.parametrize("n", (1, 40, 260))
def test_rows_without_a_key(n):
    """A batch whose every key is masked: reported, zeros there; the other batch is untouched by it."""
    B, H, N, d, block = 2, 2, 300, 64, 64
    st = state(B, H, N, d, "e4m3", block, 1), state(B, H, N, d, "e4m3", block, 2)
    pad = padded(B, N)
    pad[1] = -math.inf
    q = rows((B, H, n, d), BF, 3)
    out = run(q, st, block, pad=pad, status=sd().ERR_MASKED_ROW)
    want, A = attend(q, st, block, None, pad)
    close(out[:1], want[:1], A[:1])
    assert int(out[1].view(torch.int16).ne(0).sum()) == 0


@pytest.mark.parametrize("n", (1, 40, 260))
def test_keys_that_all_carry_the_lowest_value(n):
    """Adding the lowest fp32 value to every score absorbs them: the row is the mean of V, not empty (scales differ)."""
    B, H, N, d, block = 1, 2, 333, 64, 16
    st = state(B, H, N, d, "int8", block, 1), state(B, H, N, d, "int8", block, 2, spread=6.0)
    pad = padded(B, N)
    pad[:] = torch.finfo(torch.float32).min
    q = rows((B, H, n, d), BF, 3)
    v = dense(*st[1], block)
    mean, A = v.mean(2, keepdim=True).expand(B, H, n, d), v.abs().mean(2, keepdim=True).expand(B, H, n, d)
    # the weights are 2^log2(vs) here, down to 2^-10: f16 subnormal from 2^-14 on, so 2^-11 of each still
    close(run(q, st, block, pad=pad), mean, A)


@pytest.mark.parametrize("n", (1, 40, 260))
def test_scales_of_different_size(n):
    """Blocks of V whose magnitudes vary by 2^30, blocks of K by 2^6, zero blocks (scale 1) among them."""
    B, H, N, d, block = 1, 2, 1000, 96, 32
    st = state(B, H, N, d, "e4m3", block, 1, spread=6.0), state(B, H, N, d, "e4m3", block, 2, spread=30.0)
    for c, f in st:
        c.view(torch.uint8)[:, :, 64:96] = 0
        f[:, :, 2] = 1.0
    q = rows((B, H, n, d), BF, 3)
    # scores grow with K's magnitudes: 2^3 times the error of N(0,1) rows
    want, A = attend(q, st, block, None, None)
    err = (run(q, st, block).double().cpu() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -9) * A).all())


@pytest.mark.parametrize("n", (1, 260))
@pytest.mark.parametrize("value", (float("nan"), float("inf"), 0.0, -1.0, 2.0 ** 70))
def test_bad_scales_are_reported(n, value):
    st = state(1, 1, 600, 64, "int8", 64, 1), state(1, 1, 600, 64, "int8", 64, 2)
    st[1][1][0, 0, 3] = value
    run(rows((1, 1, n, 64), BF, 1), st, 64, status=sd().ERR_INVALID_ARG)


@pytest.mark.parametrize("n", (1, 16, 129))
def test_magnitudes_of_queries(n):
    """Rows whose elements span many binades, zero rows, tiny and large ones (the factor to f16 is exact)."""
    B, H, N, d, block = 1, 2, 500, 128, 64
    st = state(B, H, N, d, "e4m3", block, 1), state(B, H, N, d, "e4m3", block, 2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(B, H, n, d, generator=g) * torch.exp2(torch.randint(-24, 1, (B, H, n, d), generator=g).float())
    q[:, :, 0] = 0.0
    if n > 2:
        q[:, :, 1] *= 1e-30
        q[:, :, 2] = 1e-38
    q = q.to(BF).to(DEV)
    close(run(q, st, block), *attend(q, st, block, None, None))
    # large rows with a small scale
    big = (q.float() * 1e25).to(BF)
    close(run(big, st, block, scale=1e-26), *attend(big, st, block, None, None, 1e-26))


def test_bad_indices_are_skipped():
    B, H, N, d, block = 1, 2, 200, 64, 64
    st = state(B, H, N, d, "int8", block, 1), state(B, H, N, d, "int8", block, 2)
    q = rows((B, H, 50, d), BF, 3)
    for n in (5, 200):
        idx = (torch.arange(n) % 50).to(torch.int32)
        idx[1], idx[3] = 50, -1
        out = torch.full((B, H, n, d), 7.0, dtype=BF, device=DEV)
        run(q, st, block, idx.to(DEV), out=out, status=sd().ERR_INDEX)
        good = [i for i in range(n) if i not in (1, 3)]
        want, A = attend(q, st, block, idx[good], None)
        close(out[:, :, good], want, A)
        assert bool((out[:, :, [1, 3]] == 7.0).all())


@pytest.mark.parametrize("n", (1, 300))
def test_two_streams_two_graphs_and_repeats(n):
    """The same call twice gives the same bits; calls on two streams with their own workspaces do not mix; a graph
    replays on new inputs."""
    B, H, N, d, block = 1, 3, 3000, 64, 64
    sets = []
    for s in (1, 2):
        st = state(B, H, N, d, "e4m3", block, s), state(B, H, N, d, "e4m3", block, s + 5)
        q = rows((B, H, n, d), BF, s)
        sets.append((q, st, torch.zeros(B, H, n, d, dtype=BF, device=DEV), workspace(B, H, n, N, d), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def call(q, st, out, ws, stream=None):
        (k8, ks), (v8, vs) = st
        sd().safedit_attn_subset_state8(q, k8, ks, v8, vs, block, None, 0, None, 0.0, out, 0, ws, stream=stream)
    for _ in range(5):
        for q, st, out, ws, stream in sets:
            call(q, st, out, ws, stream)
    torch.cuda.synchronize()
    refs = []
    for q, st, out, ws, _ in sets:
        refs.append(attend(q, st, block, None, None))
        close(out, *refs[-1])
        again = torch.zeros_like(out)
        call(q, st, again, ws)
        assert torch.equal(out, again)
    graphs = []
    for q, st, out, ws, _ in sets:
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(q, st, out, ws)
        graphs.append(graph)
    for graph in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    for (q, st, out, ws, _), ref in zip(sets, refs):
        close(out, *ref)
    sets[0][0].copy_(sets[1][0])
    graphs[0].replay()
    torch.cuda.synchronize()
    close(sets[0][2], *attend(sets[1][0], sets[0][1], block, None, None))
    expect_status(0)


def test_offsets_past_32_bits():
    """Codes of heads more than 2^32 bytes apart."""
    N, d, block = 150, 64, 64
    step = (2 ** 32 + 2 ** 20) // d * d
    buf = torch.zeros(step + N * d, dtype=torch.int8, device=DEV)
    far = buf.as_strided((1, 2, N, d), (0, step, d, 1))
    (kc, ks), vst = state(1, 2, N, d, "int8", block, 1), state(1, 2, N, d, "int8", block, 2)
    far.copy_(kc)
    for n in (1, 140):
        q = rows((1, 2, n, d), BF, 3)
        close(run(q, ((far, ks), vst), block), *attend(q, ((kc, ks), vst), block, None, None))


@pytest.mark.parametrize("kind", CODES)
def test_a_step_of_the_trajectory(kind):
    """Rows projected, rotated, stored and attended as a trajectory does it: an anchor writes S and C rows into blocks of
    their own, an SRSU step rewrites the S blocks alone and attends from the rotated S queries over everything, the
    output scattered into the cached output.  Against the same steps in 64 bits on the stored codes."""
    B, H, N, n, d, block = 2, 3, 400, 90, 96, 32
    axes, thetas = (32, 32, 32), (1e6, 1e4, 1e4)
    spec = sd().rope_spec(axes, thetas)
    pos = positions((1, N, 3), torch.int32, 1, top=64)
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(2))
    idx_s, idx_c = (p.sort().values.to(torch.int32).to(DEV) for p in (perm[:n], perm[n:]))
    first_c = -(-n // block) * block
    total = first_c + N - n
    x = rows((B, N, 3, H, d), BF, 3)
    q, k, v = (x[:, :, t].transpose(1, 2) for t in range(3))
    ty = CODES[kind][0]
    k8, v8 = (torch.full((B, H, total, d), 0x7F, dtype=torch.uint8, device=DEV).view(ty) for _ in range(2))
    ks, vs = (torch.full((B, H, -(-total // block)), float("nan"), device=DEV) for _ in range(2))
    pad = padded(B, total)
    pad[:, n:first_c] = -math.inf
    for idx, row0 in ((idx_s, 0), (idx_c, first_c)):  # the anchor
        sd().safedit_state8_store([k, v], [k8, v8], [ks, vs], block, row0, idx, idx.numel(), True, (True, False), pos, spec)
    # the step: fresh S rows, compact
    y = rows((B, n, 3, H, d), BF, 4)
    qs, kn, vn = (y[:, :, t].transpose(1, 2) for t in range(3))
    sd().safedit_state8_store([kn, vn], [k8, v8], [ks, vs], block, 0, idx_s, n, False, (True, False), pos, spec)
    qt = torch.zeros(B, H, N, d, dtype=BF, device=DEV)
    sd().safedit_rope_rows([qs], [qt], pos, spec, idx_s, n, False, True)
    out = rows((B, H, N, d), BF, 5)
    before = out.clone()
    run(qt, ((k8, ks), (v8, vs)), block, idx_s, pad, 0.0, True, out)
    want, A = attend(qt, ((k8, ks), (v8, vs)), block, idx_s, pad)
    close(out[:, :, idx_s.long()], want, A)
    assert torch.equal(out[:, :, idx_c.long()], before[:, :, idx_c.long()])
    # and against rows that never went through 8 bits: the mean over keys of quantisation errors (at most half a step,
    # 2^-4 relative for e4m3 and 1/254 of the block's largest for int8) leaves the output within a few hundredths
    at = idx_s.long().cpu()
    kk, vv = k.double().cpu().clone(), v.double().cpu().clone()
    kk[:, :, at], vv[:, :, at] = kn.double().cpu(), vn.double().cpu()
    kt, _ = turn_reference(kk, pos, axes, thetas, False, False)
    qq, _ = turn_reference(qs, pos.cpu()[:, at], axes, thetas, False, False)
    ref = torch.softmax(qq @ kt.transpose(2, 3) * d ** -0.5, -1) @ vv
    got = out[:, :, idx_s.long()].double().cpu()
    assert float((got - ref).norm() / ref.norm()) <= 2.0 ** -4 * 1.5


@pytest.mark.parametrize("n, H, N", ((1, 300, 2000), (12, 300, 2000), (1, 44, 6000), (12, 44, 6000), (40, 3, 2000),
                                     (100, 3, 2000), (300, 3, 2000)))
@pytest.mark.parametrize("kind", CODES)
@pytest.mark.parametrize("masked", (False, True))
def test_waits_that_run_out_end_the_call(n, H, N, kind, masked):
    """With no time to wait every role gives up: reported, the device stays usable, and the next call is right.
    (With few rows a block has more keys than its copies in flight hold, so that one waits: 300 heads whole, or the
    keys of 44 heads over eight blocks each.)"""
    B, d, block = 1, 96, 64
    st = state(B, H, N, d, kind, block, 1), state(B, H, N, d, kind, block, 2)
    q = rows((B, H, n, d), BF, 3)
    pad = None
    if masked:
        pad = padded(B, N)
        pad[:, 5::7] = -math.inf
        pad[:, N - 500:] = -math.inf
    first = run(q, st, block, pad=pad)
    old = sd().safedit_debug_set_wait_limit_ns(0)
    try:
        run(q, st, block, pad=pad, status=sd().ERR_TIMEOUT)
    finally:
        sd().safedit_debug_set_wait_limit_ns(old)
    again = run(q, st, block, pad=pad)
    assert torch.equal(first, again)
    close(again, *attend(q, st, block, None, pad))


@pytest.mark.parametrize("n", (1, 20, 100, 300))
def test_heads_that_share_a_state(n):
    """Codes and scales of one head broadcast to all (stride 0), pads of one batch to both."""
    B, H, N, d, block = 2, 4, 700, 64, 32
    (kc, ks), (vc, vs) = state(B, 1, N, d, "e4m3", block, 1), state(B, 1, N, d, "e4m3", block, 2)
    k8, v8 = (c.expand(B, H, N, d) for c in (kc, vc))
    kf, vf = (f.expand(B, H, f.shape[2]) for f in (ks, vs))
    pad = padded(1, N)
    pad[:, 600:] = -math.inf
    pad = pad.expand(B, N)
    q = rows((B, H, n, d), BF, 3)
    close(run(q, ((k8, kf), (v8, vf)), block, pad=pad), *attend(q, ((k8, kf), (v8, vf)), block, None, pad))


@pytest.mark.parametrize("n", (1, 40, 260))
@pytest.mark.parametrize("what", ("hole", "head", "all far", "far apart", "mixed"))
def test_pads_of_every_size(n, what):
    """Live tiles apart from one another, masked keys in front, pads far from 0 in both directions and beside each
    other; scales that differ."""
    B, H, N, d, block = 2, 2, 1500, 128, 16
    st = state(B, H, N, d, "e4m3", block, 1), state(B, H, N, d, "e4m3", block, 2, spread=4.0)
    q = rows((B, H, n, d), BF, 3)
    pad = padded(B, N)
    pad.copy_(torch.randn(B, N, generator=torch.Generator().manual_seed(4)))
    if what == "hole":
        pad[0, 128:512] = pad[0, 700:1290] = -math.inf
        pad[1, 3:1400:2] = -math.inf
    elif what == "head":
        pad[:, :1111] = -math.inf
    elif what == "all far":
        pad += 20000.0 * torch.tensor([[1.0], [-1.0]], device=DEV)
    elif what == "far apart":
        pad[:, ::3] -= 10000.0
        pad[1, 1::3] -= 1e30
    else:
        pad[0, :] -= 1e9
        pad[0, 777] = -math.inf
        pad[1, 500:] = torch.finfo(torch.float32).min
    # the sums score + pad in fp32, as the kernel (and a plain fp32 sum) has them: what the pad absorbs is gone
    qq, k = q.double().cpu(), dense(*st[0], block)
    t = (qq @ k.transpose(2, 3) * d ** -0.5 * math.log2(math.e)).float()
    p2 = (pad.cpu().double() * math.log2(math.e)).clamp(-3.0e38, 3.0e38).float()
    p2 = torch.where(pad.cpu() == -math.inf, pad.cpu(), p2)
    t = (t + p2[:, None, None, :]).double()
    p = torch.softmax(t * math.log(2.0), -1)
    v = dense(*st[1], block)
    out = run(q, st, block, pad=pad)
    A = p @ v.abs()
    vf = st[1][1].double().cpu().repeat_interleave(block, 2)[:, :, :N]
    M = (p * vf[:, :, None, :]).amax(-1, keepdim=True) * st[1][0].float().double().cpu().abs().sum(2, keepdim=True)
    # a pad of size P leaves the fp32 sums 2^-24 P of a log2 unit, on both sides (20000: 2^-9; beyond 2^24 the sums are
    # the pads' own multiples and agree), so the weights 2^-8 there; the rest as above
    extra = 2.0 ** -8 if what == "all far" else 0.0
    err = (out.double().cpu() - p @ v).abs()
    assert bool((err <= 2.0 ** -8 * (p @ v).abs() + (2.0 ** -11 + 2.0 ** -12 + extra) * A + 2.0 ** -25 * M).all()), \
        float((err / (2.0 ** -8 * (p @ v).abs() + (2.0 ** -11 + 2.0 ** -12 + extra) * A + 2.0 ** -25 * M)).max())


@pytest.mark.parametrize("n", (1, 40, 300))
@pytest.mark.parametrize("value", (1e-42, 1e-30, 1e30, 3e38, float("inf"), float("nan"), -1.0, 0.0))
@pytest.mark.parametrize("kind", CODES)
def test_scales_of_masked_blocks_count_for_nothing(n, value, kind):
    """Whatever they are, beside blocks in use in the same tile and in tiles of their own."""
    B, H, N, d, block = 1, 2, 600, 64, 16
    st = state(B, H, N, d, kind, block, 1), state(B, H, N, d, kind, block, 2)
    (k8, ks), (v8, vs) = st
    q = rows((B, H, n, d), BF, 3)
    pad = padded(B, N)
    dead = [0, 3, 4, 17, 24, 25, 26, 27, 28, 29, 30, 31, 37]
    for i in dead:
        pad[:, i * block: (i + 1) * block] = -math.inf
    out, A = attend(q, st, block, None, pad)
    ks[:, :, dead], vs[:, :, dead] = value, value
    close(run(q, st, block, pad=pad), out, A)


@pytest.mark.parametrize("n", (1, 9, 32))
@pytest.mark.parametrize("H, N", ((3, 300), (3, 511), (3, 520), (1, 9000), (44, 700), (60, 1500), (110, 1030), (230, 600)))
def test_few_rows_whole_in_clusters_and_in_parts(n, H, N):
    """Short and long states, few slices and many: keys whole, over two to eight blocks that join them, and in parts; a
    row without a key in one batch, a bad index, masked keys over whole parts."""
    d, block = (64, 96, 128)[(n + N) % 3], 16
    kind = "int8" if n % 2 else "e4m3"
    st = state(2, H, N, d, kind, block, 1), state(2, H, N, d, kind, block, 2)
    pad = padded(2, N)
    pad[0, N // 3:] = -math.inf
    pad[1, : N // 2] = -math.inf
    idx = torch.randperm(40, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).to(DEV)
    q = rows((2, H, 40, d), BF, 3)
    close(run(q, st, block, idx=idx, pad=pad), *attend(q, st, block, idx, pad))
    out = run(q, st, block, idx=idx)
    close(out, *attend(q, st, block, idx, None))
    assert torch.equal(out, run(q, st, block, idx=idx))
    pad[1] = -math.inf
    idx[n // 2] = 40
    got = torch.full((2, H, n, d), 7.0, dtype=BF, device=DEV)
    sd().safedit_attn_subset_state8(q, st[0][0], st[0][1], st[1][0], st[1][1], block, idx, n, pad, 0.0, got, 0,
                                    workspace(2, H, n, N, d))
    expect_status(sd().ERR_INDEX)
    keep = [r for r in range(n) if r != n // 2]
    assert bool((got[:, :, n // 2] == 7.0).all())
    assert bool((got[1, :, keep] == 0.0).all())
    ref, A = attend(q, st, block, idx[keep], pad)
    close(got[:1, :, keep], ref[:1], A[:1])
