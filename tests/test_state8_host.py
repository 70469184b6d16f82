"""Host-side checks of the rotary positions, the 8-bit state and the attention over it: every refusal comes before any
launch, from shapes, types, strides and pointers alone (fake device pointers, nothing is launched), and the quotient
that the state's codes are rounded from is checked in exact arithmetic."""
import ctypes

import numpy as np
import pytest

R = ctypes.byref


@pytest.fixture(scope="module")
def sd():
    from spatially_adaptive_dit_b200 import build
    build.build()
    from spatially_adaptive_dit_b200 import safedit
    return safedit


def desc(sd, dims, dtype, ptr=0x10000, strides=None):
    t = sd.SafeditTensor()
    t.data, t.dtype, t.ndim = ptr, dtype, len(dims)
    if strides is None:
        strides, acc = [], 1
        for n in reversed(dims):
            strides.insert(0, acc)
            acc *= n
    for i, (a, b) in enumerate(zip(dims, strides)):
        t.dims[i], t.strides[i] = a, b
    return t


def arr(sd, *ts):
    return (sd.SafeditTensor * len(ts))(*ts)


IDX = ctypes.c_void_p(0x20000)


# ---------------------------------------------------------------- rotary rows
def rope_call(sd, src, dst, pos, rope, idx=None, n_idx=0, si=0, di=0, n=None):
    return sd.raw_call("safedit_rope_rows", src, dst, len(src) if n is None else n, R(pos), R(rope), idx, n_idx, si, di,
                       None)


def test_rope_refusals(sd):
    B, H, N, D = 2, 3, 64, 96
    x = desc(sd, (B, H, N, D), sd.BF16)
    pos = desc(sd, (1, N, 3), sd.I32)
    spec = sd.rope_spec((32, 32, 32), (1e4, 1e4, 1e4))
    go = lambda s=x, d=x, p=pos, r=spec, **k: rope_call(sd, arr(sd, s), arr(sd, d), p, r, **k)  # noqa: E731
    mk = lambda dims=(B, H, N, D), dt=sd.BF16, **k: desc(sd, dims, dt, **k)  # noqa: E731
    assert go(n=0) == sd.ERR_INVALID_ARG and go(n=5) == sd.ERR_INVALID_ARG
    assert go(s=mk(dt=sd.F64), d=mk(dt=sd.F64)) == sd.ERR_DTYPE
    assert go(d=mk(dt=sd.F16)) == sd.ERR_DTYPE
    assert go(s=mk(dt=sd.E4M3), d=mk(dt=sd.E4M3)) == sd.ERR_DTYPE
    assert go(d=mk((B, H, N + 1, D))) == sd.ERR_SHAPE
    assert go(d=mk((B, H + 1, N, D))) == sd.ERR_SHAPE
    assert go(s=mk(ptr=0x10008)) == sd.ERR_ALIGNMENT
    assert go(s=mk(strides=(H * N * 100, N * 100, 100, 1))) == sd.ERR_ALIGNMENT
    assert go(s=mk(strides=(H * N * D * 2, N * D * 2, D * 2, 2))) == sd.ERR_ALIGNMENT
    # widths: a multiple of 8 up to 256
    for d in (4, 12, 264):
        y = mk((B, H, N, d))
        assert go(s=y, d=y, r=sd.rope_spec((2,), (1e4,)), p=desc(sd, (1, N, 1), sd.I32)) == sd.ERR_UNSUPPORTED
    # axes: even (multiples of 8 for halves), no wider than the row, one position each, finite positive bases
    assert go(r=sd.rope_spec((31, 32, 32), (1e4,) * 3)) == sd.ERR_UNSUPPORTED
    assert go(r=sd.rope_spec((20, 32, 32), (1e4,) * 3, sd.ROPE_HALVES)) == sd.ERR_UNSUPPORTED
    assert go(r=sd.rope_spec((34, 32, 32), (1e4,) * 3)) == sd.ERR_SHAPE
    assert go(r=sd.rope_spec((32, 0, 32), (1e4,) * 3)) == sd.ERR_INVALID_ARG
    assert go(r=sd.rope_spec((32, 32), (1e4,) * 2)) == sd.ERR_SHAPE
    for theta in (0.0, -1.0, float("inf"), float("nan"), 1e-300, 0.5):
        assert go(r=sd.rope_spec((32, 32, 32), (1e4, theta, 1e4))) == sd.ERR_INVALID_ARG
    bad = sd.rope_spec((32, 32, 32), (1e4,) * 3)
    bad.halves = 2
    assert go(r=bad) == sd.ERR_INVALID_ARG
    bad.halves, bad.n_axes = 0, 5
    assert go(r=bad) == sd.ERR_INVALID_ARG
    # positions: i32 or f32, of one or every batch, one for each token
    assert go(p=desc(sd, (1, N, 3), sd.F64)) == sd.ERR_DTYPE
    assert go(p=desc(sd, (3, N, 3), sd.I32)) == sd.ERR_SHAPE
    assert go(p=desc(sd, (1, N - 1, 3), sd.I32)) == sd.ERR_SHAPE
    assert go(p=desc(sd, (N, 3), sd.I32)) == sd.ERR_SHAPE
    # indexed sides need an index; a compact side has n_idx rows
    assert go(si=1) == sd.ERR_INVALID_ARG and go(di=1) == sd.ERR_INVALID_ARG and go(di=2) == sd.ERR_INVALID_ARG
    assert go(idx=IDX, n_idx=-1, di=1) == sd.ERR_INVALID_ARG
    assert go(idx=IDX, n_idx=10, di=1) == sd.ERR_SHAPE
    # nothing to do: checked, then nothing is launched
    n0 = sd.safedit_kernel_launch_count()
    e = mk((B, H, 0, D), ptr=None)
    assert go(s=e, d=e) == sd.OK
    assert go(s=mk((B, H, 0, D), ptr=None), idx=IDX, n_idx=0, di=1) == sd.OK
    assert sd.safedit_kernel_launch_count() == n0


def test_rope_spec_refusals(sd):
    for dims, thetas in (((), ()), ((8,) * 5, (1e4,) * 5), ((8, 8), (1e4,))):
        with pytest.raises(sd.SafeditError) as e:
            sd.rope_spec(dims, thetas)
        assert e.value.code == sd.ERR_INVALID_ARG


# ---------------------------------------------------------------- 8-bit state
def store_call(sd, src, codes, scales, block=64, row0=0, idx=None, n_idx=0, si=0, rot=None, pos=None, rope=None, n=None):
    flags = None if rot is None else (ctypes.c_int32 * len(rot))(*rot)
    return sd.raw_call("safedit_state8_store", src, codes, scales, len(src) if n is None else n, block, row0, idx, n_idx,
                       si, flags, None if pos is None else R(pos), None if rope is None else R(rope), None)


def test_store_refusals(sd):
    B, H, n, N, D = 2, 3, 64, 256, 96
    x, c, f = desc(sd, (B, H, n, D), sd.BF16), desc(sd, (B, H, N, D), sd.I8), desc(sd, (B, H, 4), sd.F32)
    go = lambda s=x, k=c, v=f, **kw: store_call(sd, arr(sd, s), arr(sd, k), arr(sd, v), **kw)  # noqa: E731
    assert go(n=0) == sd.ERR_INVALID_ARG and go(n=5) == sd.ERR_INVALID_ARG
    assert go(k=desc(sd, (B, H, N, D), sd.U8)) == sd.ERR_DTYPE
    assert go(k=desc(sd, (B, H, N, D), sd.BF16)) == sd.ERR_DTYPE
    assert go(s=desc(sd, (B, H, n, D), sd.I8)) == sd.ERR_DTYPE
    assert go(v=desc(sd, (B, H, 4), sd.F64)) == sd.ERR_DTYPE
    for block in (0, 8, 48, 256, -64):
        assert go(block=block) == sd.ERR_UNSUPPORTED
    assert go(row0=32) == sd.ERR_ALIGNMENT and go(row0=-64) == sd.ERR_INVALID_ARG
    assert go(row0=256) == sd.ERR_SHAPE and go(row0=1 << 62) == sd.ERR_SHAPE
    assert go(v=desc(sd, (B, H, 3), sd.F32)) == sd.ERR_SHAPE
    assert go(v=desc(sd, (B, H, 4), sd.F32, strides=(24, 8, 2))) == sd.ERR_ALIGNMENT
    assert go(k=desc(sd, (B, H, N, D), sd.I8, ptr=0x10004)) == sd.ERR_ALIGNMENT
    assert go(k=desc(sd, (B, H, N, D), sd.I8, strides=(H * N * 104, N * 104, 104, 1))) == sd.ERR_ALIGNMENT
    assert go(s=desc(sd, (B, H, n, D), sd.BF16, ptr=0x10002)) == sd.ERR_ALIGNMENT
    assert go(s=desc(sd, (B, H + 1, n, D), sd.BF16)) == sd.ERR_SHAPE
    y = desc(sd, (B, H, n, 80), sd.BF16)
    assert go(s=y, k=desc(sd, (B, H, N, 80), sd.I8)) == sd.ERR_UNSUPPORTED
    assert go(si=1) == sd.ERR_INVALID_ARG and go(idx=IDX, n_idx=-1) == sd.ERR_INVALID_ARG
    assert go(idx=IDX, n_idx=10) == sd.ERR_SHAPE  # a compact source has n_idx rows
    # two tensors of different code types
    assert store_call(sd, arr(sd, x, x), arr(sd, c, desc(sd, (B, H, N, D), sd.E4M3)), arr(sd, f, f)) == sd.ERR_DTYPE
    # rotation: flags of 0 or 1, positions and axes where one is set, no inverse
    pos, rope = desc(sd, (1, n, 3), sd.I32), sd.rope_spec((32, 32, 32), (1e4,) * 3)
    assert go(rot=(2,)) == sd.ERR_INVALID_ARG
    assert go(rot=(1,)) == sd.ERR_INVALID_ARG
    assert go(rot=(1,), pos=pos) == sd.ERR_INVALID_ARG
    assert go(rot=(1,), pos=desc(sd, (1, n - 1, 3), sd.I32), rope=rope) == sd.ERR_SHAPE
    assert go(rot=(1,), pos=pos, rope=sd.rope_spec((32,) * 3, (1e4,) * 3, inverse=True)) == sd.ERR_INVALID_ARG
    n0 = sd.safedit_kernel_launch_count()
    assert go(s=desc(sd, (B, H, 0, D), sd.BF16, ptr=None), row0=256) == sd.OK
    assert sd.safedit_kernel_launch_count() == n0


def test_attention_refusals(sd):
    B, H, Nq, N, D = 1, 2, 100, 3000, 64
    q, o = desc(sd, (B, H, Nq, D), sd.BF16), desc(sd, (B, H, Nq, D), sd.BF16)
    k, f = desc(sd, (B, H, N, D), sd.E4M3), desc(sd, (B, H, 47), sd.F32)
    big = 1 << 30

    def go(q=q, k=k, ks=f, v=k, vs=f, block=64, idx=None, n_idx=0, pad=None, o=o, scat=0, ws=0x40000, nb=big):
        return sd.raw_call("safedit_attn_subset_state8", R(q), R(k), R(ks), R(v), R(vs), block, idx, n_idx,
                           None if pad is None else R(pad), 0.0, R(o), scat, ctypes.c_void_p(ws), nb, None)

    codes = lambda dims=(B, H, N, D), dt=sd.E4M3, **kw: desc(sd, dims, dt, **kw)  # noqa: E731
    assert go(q=desc(sd, (B, H, Nq, D), sd.F16)) == sd.ERR_DTYPE
    assert go(k=codes(dt=sd.BF16)) == sd.ERR_DTYPE and go(v=codes(dt=sd.I8)) == sd.ERR_DTYPE
    assert go(o=desc(sd, (B, H, Nq, D), sd.F32)) == sd.ERR_DTYPE
    assert go(block=24) == sd.ERR_UNSUPPORTED
    assert go(block=32) == sd.ERR_SHAPE  # scales of another block
    assert go(v=codes((B, H, N - 1, D))) == sd.ERR_SHAPE
    assert go(q=desc(sd, (B, 3, Nq, D), sd.BF16)) == sd.ERR_SHAPE
    assert go(o=desc(sd, (B, H, Nq - 1, D), sd.BF16)) == sd.ERR_SHAPE
    assert go(scat=2) == sd.ERR_INVALID_ARG and go(idx=IDX, n_idx=-1) == sd.ERR_INVALID_ARG
    assert go(k=codes(ptr=0x10008)) == sd.ERR_ALIGNMENT
    assert go(v=codes(strides=(H * N * 72, N * 72, 72, 1))) == sd.ERR_ALIGNMENT
    assert go(q=desc(sd, (B, H, Nq, D), sd.BF16, ptr=0x10004)) == sd.ERR_ALIGNMENT
    assert go(k=codes((B, H, 0, D)), v=codes((B, H, 0, D)), ks=desc(sd, (B, H, 0), sd.F32),
              vs=desc(sd, (B, H, 0), sd.F32)) == sd.ERR_SHAPE
    w = desc(sd, (B, H, Nq, 80), sd.BF16)
    assert go(q=w, o=w, k=codes((B, H, N, 80)), v=codes((B, H, N, 80))) == sd.ERR_UNSUPPORTED
    assert go(pad=desc(sd, (B, N), sd.BF16)) == sd.ERR_DTYPE
    assert go(pad=desc(sd, (B, N + 1), sd.F32)) == sd.ERR_SHAPE
    assert go(pad=desc(sd, (B, N), sd.F32, ptr=0x10004)) == sd.ERR_ALIGNMENT
    assert go(pad=desc(sd, (B, N), sd.F32, strides=(3001, 1))) == sd.ERR_ALIGNMENT
    # the workspace: large enough, aligned, given
    need = sd.safedit_attn_subset_state8_workspace_size(B, H, Nq, N, D)
    assert need > 0
    assert go(nb=need - 1) == sd.ERR_INVALID_ARG and go(ws=None) == sd.ERR_INVALID_ARG
    assert go(ws=0x40008) == sd.ERR_ALIGNMENT
    n0 = sd.safedit_kernel_launch_count()
    none = desc(sd, (B, H, 0, D), sd.BF16, ptr=None)
    assert go(idx=IDX, n_idx=0, o=none) == sd.OK
    assert sd.safedit_kernel_launch_count() == n0


def test_attention_workspace_size(sd):
    ws = sd.safedit_attn_subset_state8_workspace_size
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, 0, 64), (1, 1, 1, 1, 80),
                (1 << 40, 1 << 40, 1, 1, 64), (1, 1, 1 << 40, 1, 64), (1, 1, 1, 1 << 40, 64), (-1, 1, 1, 1, 64)):
        assert ws(*bad) == 0
    assert ws(1, 1, 1, 1, 64) == 0      # one key: nothing to split
    assert ws(1, 1, 1, 25600, 96) > 0   # one row of one slice: the keys go over the SMs


def test_other_calls_refuse_code_types(sd):
    """The 8-bit code types belong to the state: every other entry point refuses them as it refuses unknown types."""
    t8 = desc(sd, (1, 2, 64, 64), sd.I8)
    tb = desc(sd, (1, 2, 64, 64), sd.BF16)
    assert sd.raw_call("safedit_attn_subset", R(t8), R(tb), R(tb), None, 0, None, None, 0.0, R(tb), 0, None) == sd.ERR_DTYPE
    a = arr(sd, t8)
    assert sd.raw_call("safedit_scatter_state", a, a, 1, IDX, 64, None) == sd.ERR_DTYPE
    m = desc(sd, (8, 8), sd.E4M3)
    assert sd.raw_call("safedit_mask_is_row_constant", R(m), ctypes.c_void_p(0x70000), None, None) == sd.ERR_DTYPE


# ---------------------------------------------------------------- the codes' quotient
def _markstein(x, most, qmax):
    """The store kernel's arithmetic in numpy: fp32 products, fp32 fused multiply-adds (their exact value fits 64 bits'
    extended product here: both factors have 24 bits, so the product is exact in fp64 and the sum is rounded once by
    going through np.longdouble)."""
    f32, ld = np.float32, np.longdouble
    ex = np.floor(np.log2(most.astype(ld))).astype(int)
    m1 = (most / np.exp2(ex.astype(ld)).astype(ld)).astype(f32)
    up = (np.exp2((-ex).astype(ld)) * qmax).astype(f32)
    inv = (f32(1.0) / m1).astype(f32)
    a = (x * up).astype(f32)
    q = (a * inv).astype(f32)
    r = (-(q.astype(ld) * m1.astype(ld)) + a.astype(ld)).astype(f32)
    return (r.astype(ld) * inv.astype(ld) + q.astype(ld)).astype(f32)


@pytest.mark.parametrize("mantissa, qmax", [(7, 448.0), (7, 127.0), (10, 448.0), (10, 127.0)])
def test_quotient_rounds_to_the_right_code(mantissa, qmax):
    """For every pair of significands of a 16-bit type the corrected quotient lands on the same code as the exact one,
    ties included."""
    sig = (1.0 + np.arange(2 ** mantissa) / 2 ** mantissa).astype(np.float32)
    rng = np.random.RandomState(0)
    tops = sig if mantissa == 7 else sig[rng.choice(sig.size, 96, replace=False)]
    for top in tops:
        most = np.float32(top * 4.0)
        x = np.concatenate([sig * np.float32(2.0 ** e) for e in range(-5, 3)])
        x = x[x <= most]
        y = _markstein(x, np.full_like(x, most), qmax)
        exact = x.astype(np.float64) * qmax / np.float64(most)
        if qmax == 127.0:
            step = np.ones_like(exact)
        else:
            step = np.exp2(np.clip(np.floor(np.log2(exact)), -6, 8) - 3)
        # rint of the exact quotient: a tie is met exactly, since x qmax / most differs from a tie by at least
        # 2^-19 of it or not at all (significands of at most 11 bits), and fp64 keeps 2^-53
        assert np.array_equal(np.rint(y.astype(np.float64) / step), np.rint(exact / step))
