"""The rotary positions, the 8-bit state and the attention that reads it: what is timed, on what inputs.

Three operators of a spatially adaptive transformer step:

  rope   rows of Q and K rotated at their tokens' positions on several axes (time or text, height, width);
  store  rows of K and V written into an 8-bit state with a scale for each block of rows and head, K rotated first
         where the case says so;
  attn   query rows attending over such a state.

`run` computes them in elementary torch operations where `own` is false, and calls the library where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
# the base of each axis' frequencies: a slow one for time or text, the usual one for height and width
BASES = (1.0e6, 1.0e4, 1.0e4)
# blocks whose largest magnitude is below this are scaled as if it were this (nothing overflows on the way)
LEAST = 2.0 ** -100


# ------------------------------------------------------------------ cases
def _rope(name, **kw):
    c = {"op": "rope", "B": 1, "H": 1, "n": 1, "N": 1, "d": 64, "axes": "64", "halves": False, "dtype": "bf16",
         "pos": "i32", "tensors": 2, "indexed": False, "fused": False, "inverse": False}
    c.update(kw)
    return dict(c, name=name) if name else c


def _store(name, **kw):
    c = {"op": "store", "B": 1, "H": 1, "n": 1, "N": 1, "d": 64, "codes": "e4m3", "block": 64, "dtype": "bf16",
         "axes": "", "halves": False, "indexed": False, "fused": False, "row0": 0}
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, **kw):
    c = {"op": "attn", "B": 1, "H": 1, "n": 1, "N": 1, "Nq": 1, "d": 64, "codes": "e4m3", "block": 64, "pad": False,
         "indexed": False}
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a step: latency
        _rope("rope_one_token", B=2, H=24, n=1, N=4096, d=96, axes="32,32,32", indexed=True),
        # Q and K of a dense step of a 1024 x 1024 image, read out of the fused projection, at fractional positions
        # (a grid stretched to another resolution)
        _rope("rope_image_1024", B=2, H=24, n=4096, N=4096, d=96, axes="32,32,32", pos="f32", fused=True),
        # the sensitive rows of a video-like grid, rotated straight into the cached state
        _rope("rope_rows_into_state", B=1, H=32, n=4915, N=16384, d=128, axes="16,56,56", halves=True, dtype="f16",
              indexed=True),
        # the transpose (what a gradient needs) in fp32, an odd number of rows, part of the width left unrotated
        _rope("rope_transpose_f32", B=1, H=8, n=16383, N=16383, d=64, axes="24,24", dtype="f32", inverse=True,
              tensors=1),
        # a handful of rows into the state: latency
        _store("store_few_rows", B=1, H=2, n=37, N=256, d=64, codes="int8", block=16, row0=16),
        # the sensitive rows of a 1024 x 1024 step, already rotated, gathered from the dense projection
        _store("store_rows_1024", B=2, H=24, n=1229, N=4096, d=96, codes="int8", block=32, indexed=True),
        # every row of a 2560 x 2560 dense step out of the fused projection, K rotated on the way
        _store("store_anchor_2560", B=2, H=24, n=25600, N=25600, d=96, codes="e4m3", block=64, axes="32,32,32",
               fused=True),
        # one query row over a long state: read the state once
        _attn("attn_one_row", B=2, H=24, n=1, N=25600, Nq=25600, d=96, indexed=True),
        # a few rows, an odd key count, padding
        _attn("attn_few_rows", B=3, H=8, n=13, N=4999, Nq=4999, d=64, codes="int8", block=16, pad=True, indexed=True),
        # the sensitive rows of a 1024 x 1024 step
        _attn("attn_rows_1024", B=2, H=24, n=1229, N=4096, Nq=4096, d=96, codes="int8", block=32, indexed=True),
        # wide heads, the last eighth of the keys padding
        _attn("attn_rows_16k_pad", B=1, H=32, n=4915, N=16384, Nq=16384, d=128, block=128, pad=True, indexed=True),
        # the sensitive rows of a 2560 x 2560 step
        _attn("attn_rows_2560", B=2, H=24, n=7680, N=25600, Nq=25600, d=96, indexed=True),
    ]


# what a drawn case holds at most: the largest listed ones' scores and values
MOST_SCORES = 2 * 24 * 7680 * 25600
MOST_VALUES = 2 * 24 * 25600 * 96


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _axes(rng, d, halves):
    """Segments that rotate (part of) a row of d: one to three axes."""
    step = 8 if halves else 2
    left = d if rng.random() < 0.7 else d - 8 * rng.randint(1, d // 16)
    k = min(rng.randint(1, 3), left // step)
    got = []
    for a in range(k):
        most = left - step * (k - 1 - a)
        s = most if a == k - 1 else step * rng.randint(1, max(1, most // step // (k - a)))
        got.append(s // step * step)
        left -= got[-1]
    return ",".join(str(s) for s in got)


def draw(rng):
    op = rng.choice(("rope", "store", "attn"))
    B, H = rng.randint(1, 3), _log(rng, 1, 32)
    if op == "rope":
        d = 8 * rng.randint(4, 16)
        N = min(_log(rng, 1, 25600), MOST_VALUES // (B * H * d))
        indexed = rng.random() < 0.5
        n = _log(rng, 1, N) if indexed else N
        halves = rng.random() < 0.5
        return _rope("", B=B, H=H, n=n, N=N, d=d, axes=_axes(rng, d, halves), halves=halves,
                     dtype=rng.choice(("bf16", "f16", "f32")), pos=rng.choice(("i32", "f32")), tensors=rng.randint(1, 2),
                     indexed=indexed, fused=rng.random() < 0.5, inverse=rng.random() < 0.3)
    d = rng.choice((64, 96, 128))
    codes, block = rng.choice(("e4m3", "int8")), rng.choice((16, 32, 64, 128))
    if op == "store":
        N = min(_log(rng, 1, 25600), MOST_VALUES // (B * H * d))
        indexed = rng.random() < 0.5
        row0 = block * rng.randint(0, max(0, N // block - 1)) if rng.random() < 0.5 else 0
        n = _log(rng, 1, N - row0)
        halves = rng.random() < 0.5
        # rotated rows in int8 meet rounding borders that 32 bits cannot tell apart: they go to e4m3 here
        rotated = codes == "e4m3" and rng.random() < 0.6
        return _store("", B=B, H=H, n=n, N=N, d=d, codes=codes, block=block, dtype=rng.choice(("bf16", "f16")),
                      axes=_axes(rng, d, halves) if rotated else "", halves=halves and rotated, indexed=indexed,
                      fused=rng.random() < 0.5, row0=row0)
    N = _log(rng, 1, 25600)
    n = _log(rng, 1, N)
    while B * H * n * N * d > MOST_SCORES * 96 or B * H * n * N > MOST_SCORES:
        n = max(1, n // 2)
    indexed = rng.random() < 0.7
    return _attn("", B=B, H=H, n=n, N=N, Nq=N if indexed else n, d=d, codes=codes, block=block,
                 pad=rng.random() < 0.4, indexed=indexed)


# ------------------------------------------------------------------ inputs
def _positions(c, g):
    """[1, N, axes]: tokens of a grid in row order behind a seeded origin; fractional ones are stretched."""
    axes = [int(s) for s in c["axes"].split(",")]
    side = max(1, math.isqrt(max(1, c["N"] // (2 if len(axes) == 3 else 1))))
    i = torch.arange(c["N"], device=DEV)
    cols = [i // (side * side), i // side % side, i % side][3 - len(axes):] if len(axes) > 1 else [i]
    origin = torch.randint(0, 2048, (len(axes),), generator=g, device=DEV)
    p = torch.stack(cols, -1) + origin
    if c.get("pos", "i32") == "f32":
        return (p.double() * 0.4140625).float()[None]
    return p.to(torch.int32)[None].contiguous()


def _rows(c, g, dtype, rows):
    """A [B, H, rows, d] tensor; out of a fused projection [B, rows, 2, H, d] it is a strided view."""
    def one():
        return torch.randn(c["B"], c["H"], rows, c["d"], generator=g, device=DEV).to(dtype)
    count = c.get("tensors", 2)
    if not c["fused"]:
        return [one() for _ in range(count)]
    x = torch.randn(c["B"], rows, count, c["H"], c["d"], generator=g, device=DEV).to(dtype)
    return [x[:, :, t].transpose(1, 2) for t in range(count)]


def _index(c, g, size):
    return torch.randperm(size, generator=g, device=DEV)[: c["n"]].sort().values.to(torch.int32)


def _pairs(axes, d, halves):
    """Positions in a row of each pair's two elements, each pair's axis and its frequency (64 bits)."""
    lo, hi, axis, freq, at = [], [], [], [], 0
    for a, s in enumerate(axes):
        lo += [at + (m if halves else 2 * m) for m in range(s // 2)]
        hi += [at + (m + s // 2 if halves else 2 * m + 1) for m in range(s // 2)]
        axis += [a] * (s // 2)
        freq += [BASES[a] ** (-2.0 * m / s) for m in range(s // 2)]
        at += s
    t = lambda v, ty: torch.tensor(v, dtype=ty, device=DEV)  # noqa: E731
    return t(lo, torch.long), t(hi, torch.long), t(axis, torch.long), t(freq, torch.float64)


def _spec(c, inverse=False):
    from spatially_adaptive_dit_b200 import safedit as sd
    axes = [int(s) for s in c["axes"].split(",")]
    return sd.rope_spec(axes, BASES[: len(axes)], sd.ROPE_HALVES if c["halves"] else sd.ROPE_INTERLEAVED, inverse)


def _random_codes(c, g, shape):
    ty, _ = CODES[c["codes"]]
    x = torch.randint(0, 120, shape, generator=g, device=DEV, dtype=torch.uint8)  # no NaN among the e4m3 codes
    return x.view(ty)


def _quantised(c, g):
    """A state in 8 bits: codes [B, H, N, d], scales [B, H, blocks]."""
    ty, top = CODES[c["codes"]]
    B, H, N, d, block = c["B"], c["H"], c["N"], c["d"], c["block"]
    nb = -(-N // block)
    x = torch.zeros(B, H, nb * block, d, device=DEV)
    x[:, :, :N] = torch.randn(B, H, N, d, generator=g, device=DEV)
    x = x.view(B, H, nb, block, d)
    scale = x.abs().amax((-1, -2)) / top
    y = x / scale[..., None, None]
    y = y.to(ty) if c["codes"] == "e4m3" else y.round().clamp(-top, top).to(ty)
    return y.view(B, H, nb * block, d)[:, :, :N].contiguous(), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c, "idx": None}
    if c["op"] == "rope":
        dtype = DTYPES[c["dtype"]]
        s["src"] = _rows(c, g, dtype, c["n"])
        s["pos"] = _positions(c, g)
        rows = c["N"] if c["indexed"] else c["n"]
        if c["indexed"]:
            s["idx"] = _index(c, g, c["N"])
        s["dst"] = [torch.randn(c["B"], c["H"], rows, c["d"], generator=g, device=DEV).to(dtype) for _ in s["src"]]
        s["pairs"] = _pairs([int(v) for v in c["axes"].split(",")], c["d"], c["halves"])
        s["spec"] = _spec(c, c["inverse"]) if own else None
    elif c["op"] == "store":
        s["src"] = _rows(c, g, DTYPES[c["dtype"]], c["N"] if c["indexed"] else c["n"])
        if c["indexed"]:
            s["idx"] = _index(c, g, c["N"])
        nb = -(-c["N"] // c["block"])
        s["codes"] = [_random_codes(c, g, (c["B"], c["H"], c["N"], c["d"])) for _ in s["src"]]
        s["scales"] = [torch.rand(c["B"], c["H"], nb, generator=g, device=DEV) + 0.5 for _ in s["src"]]
        s["pos"] = s["pairs"] = s["spec"] = None
        if c["axes"]:
            s["pos"] = _positions(c, g)
            s["pairs"] = _pairs([int(v) for v in c["axes"].split(",")], c["d"], c["halves"])
            s["spec"] = _spec(c) if own else None
    else:
        B, H = c["B"], c["H"]
        s["q"] = torch.randn(B, H, c["Nq"], c["d"], generator=g, device=DEV).to(torch.bfloat16)
        s["k8"], s["ks"] = _quantised(c, g)
        s["v8"], s["vs"] = _quantised(c, g)
        if c["indexed"]:
            s["idx"] = _index(c, g, c["Nq"])
        s["pad"] = None
        if c["pad"]:  # soft weights, and no weight at all for the last eighth; rows of 16 bytes
            p = torch.zeros(B, -(-c["N"] // 4) * 4, device=DEV)
            p[:, : c["N"]] = -2.0 * torch.rand(B, c["N"], generator=g, device=DEV)
            p[:, c["N"] - c["N"] // 8: c["N"]] = -math.inf
            s["pad"] = p[:, : c["N"]]
        s["out"] = torch.zeros(B, H, c["n"], c["d"], device=DEV, dtype=torch.bfloat16)
        s["ws"] = None
        if own:
            from spatially_adaptive_dit_b200 import safedit as sd
            size = sd.safedit_attn_subset_state8_workspace_size(B, H, c["n"], c["N"], c["d"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
    return s


# ------------------------------------------------------------------ one pass
def _turned(x, s, tokens, inverse):
    """x [B, H, rows, d] in 32 bits, rotated at the positions of `tokens` (None: row r is token r)."""
    lo, hi, axis, freq = s["pairs"]
    pos = s["pos"] if tokens is None else s["pos"][:, tokens]
    angle = pos[:, : x.shape[2]].double()[..., axis] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    a, b = x[..., lo], x[..., hi]
    y = x.clone()
    y[..., lo] = a * cos - b * sin
    y[..., hi] = a * sin + b * cos
    return y


def _run_rope(s):
    c = s["case"]
    if own:
        from spatially_adaptive_dit_b200 import safedit as sd
        sd.safedit_rope_rows(s["src"], s["dst"], s["pos"], s["spec"], s["idx"], c["n"], False, c["indexed"])
        return s["dst"]
    at = s["idx"].long() if c["indexed"] else None
    y = _turned(torch.stack([x.float() for x in s["src"]]).flatten(0, 1), s, at, c["inverse"])
    y = y.to(s["dst"][0].dtype).unflatten(0, (len(s["src"]), c["B"])).unbind(0)
    if not c["indexed"]:
        return list(y)
    return [t.index_copy(2, at, x) for t, x in zip(s["dst"], y)]


def _stored(x, codes, scales, c):
    """x [B, H, n, d] in 32 bits into a copy of the state."""
    ty, top = CODES[c["codes"]]
    n, block, row0, N = c["n"], c["block"], c["row0"], c["N"]
    nb = -(-n // block)
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * block - n)).unflatten(2, (nb, block))
    most = x.abs().amax((-1, -2))
    most = torch.where(most == 0, torch.full_like(most, top), most.clamp_min(LEAST))
    # one rounding in the quotient: with 16-bit rows the product is exact and ties between codes are met exactly
    y = x * top / most[..., None, None]
    y = y.clamp(-top, top).to(ty) if c["codes"] == "e4m3" else y.round().clamp(-top, top).to(ty)
    rows = min(N, row0 + nb * block) - row0
    codes, scales = codes.clone(), scales.clone()
    codes[:, :, row0: row0 + rows] = y.flatten(2, 3)[:, :, :rows]
    scales[:, :, row0 // block: row0 // block + nb] = most / top
    return codes, scales


def _run_store(s):
    c = s["case"]
    if own:
        from spatially_adaptive_dit_b200 import safedit as sd
        sd.safedit_state8_store(s["src"], s["codes"], s["scales"], c["block"], c["row0"], s["idx"], c["n"], c["indexed"],
                                (True, False) if c["axes"] else None, s["pos"], s["spec"])
        return s["codes"] + s["scales"]
    at = s["idx"].long() if c["indexed"] else None
    k, v = (x.float() if at is None else x[:, :, at].float() for x in s["src"])
    if c["axes"]:
        k = _turned(k, s, at, False)
    k8, ks = _stored(k, s["codes"][0], s["scales"][0], c)
    v8, vs = _stored(v, s["codes"][1], s["scales"][1], c)
    return [k8, v8, ks, vs]


def _run_attn(s):
    c = s["case"]
    if own:
        from spatially_adaptive_dit_b200 import safedit as sd
        sd.safedit_attn_subset_state8(s["q"], s["k8"], s["ks"], s["v8"], s["vs"], c["block"], s["idx"], c["n"], s["pad"],
                                      0.0, s["out"], 0, s["ws"])
        return s["out"]
    q = (s["q"][:, :, s["idx"].long()] if c["indexed"] else s["q"][:, :, : c["n"]]).float()
    k = s["k8"].float() * s["ks"].repeat_interleave(c["block"], 2)[:, :, : c["N"], None]
    v = s["v8"].float() * s["vs"].repeat_interleave(c["block"], 2)[:, :, : c["N"], None]
    w = (q / math.sqrt(c["d"])) @ k.transpose(2, 3)
    if s["pad"] is not None:
        w += s["pad"][:, None, None, :]
    w -= w.amax(-1, keepdim=True)
    w.exp_()
    total = w.sum(-1, keepdim=True)
    return ((w @ v) / total).to(torch.bfloat16)


def run(state):
    return {"rope": _run_rope, "store": _run_store, "attn": _run_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    rows = c["B"] * c["H"] * c["n"]
    if c["op"] == "rope":
        es, axes = DTYPES[c["dtype"]].itemsize, c["axes"].count(",") + 1
        size = rows * c["d"] * c["tensors"]
        return {"bytes": 2 * es * size + 4 * c["n"] * (axes + c["indexed"]), "flops": 3 * size}
    if c["op"] == "store":
        size, blocks = 2 * rows * c["d"], 2 * c["B"] * c["H"] * -(-c["n"] // c["block"])
        axes = c["axes"].count(",") + 1 if c["axes"] else 0
        return {"bytes": 3 * size + 4 * blocks + 4 * c["n"] * (axes + c["indexed"]), "flops": 2 * size}
    keys = c["B"] * c["H"] * c["N"]
    return {"bytes": 4 * rows * c["d"] + 2 * keys * c["d"] + 8 * c["B"] * c["H"] * -(-c["N"] // c["block"])
            + (4 * c["B"] * c["N"] if c["pad"] else 0) + 4 * c["n"] * c["indexed"], "flops": 4 * rows * c["N"] * c["d"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_turn(x, c, pos, inverse):
    """x [B, H, rows, d] in 64 bits times exp(i angle), axis by axis, as complex numbers."""
    parts, at = [], 0
    for a, size in enumerate(int(v) for v in c["axes"].split(",")):
        seg = x[..., at: at + size]
        m = torch.arange(size // 2, device=DEV, dtype=torch.float64)
        angle = pos[:, :, a, None].double() * torch.exp(-(2.0 * m / size) * math.log(BASES[a]))
        turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None]
        z = torch.complex(*seg.chunk(2, -1)) if c["halves"] else torch.view_as_complex(seg.unflatten(-1, (-1, 2)).contiguous())
        z = z * turn
        parts.append(torch.cat([z.real, z.imag], -1) if c["halves"] else torch.view_as_real(z).flatten(-2))
        at += size
    return torch.cat(parts + [x[..., at:]], -1)


def _exact_e4m3(y):
    """The e4m3 value nearest to y, ties to the even one."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    tokens = s["idx"].long() if s["idx"] is not None else torch.arange(c["n"], device=DEV)
    if c["op"] == "rope":
        got = []
        for x, t in zip(s["src"], s["dst"]):
            y = torch.cat([_exact_turn(x[b: b + 1].double(), c, s["pos"][:, tokens], c["inverse"]) for b in range(c["B"])])
            t = t.double()
            t[:, :, tokens] = y
            got.append(t)
        return got
    if c["op"] == "store":
        codes, scales = [], []
        _, top = CODES[c["codes"]]
        for k, x in enumerate(s["src"]):
            if c["indexed"]:
                x = x.index_select(2, tokens)
            x = x.double()
            if c["axes"] and k == 0:
                x = torch.cat([_exact_turn(x[b: b + 1], c, s["pos"][:, tokens], False) for b in range(c["B"])])
            sc, cd = s["scales"][k].double(), s["codes"][k].float().double()
            for at in range(0, c["n"], c["block"]):
                part = x[:, :, at: at + c["block"]]
                most = part.abs().flatten(2).max(-1).values
                most = torch.where(most > 0, torch.maximum(most, torch.full_like(most, LEAST)), torch.full_like(most, top))
                sc[:, :, (c["row0"] + at) // c["block"]] = most / top
                first = c["row0"] + at
                cd[:, :, first: first + c["block"]] = 0.0
                cd[:, :, first: first + part.shape[2]] = _exact_e4m3(part * top / most[:, :, None, None])
            codes.append(cd if c["codes"] == "e4m3" else None)
            scales.append(sc)
        return codes + scales
    out = torch.empty(c["B"], c["H"], c["n"], c["d"], dtype=torch.float64, device=DEV)
    block_of = torch.arange(c["N"], device=DEV) // c["block"]
    for b in range(c["B"]):
        for h in range(c["H"]):
            k = s["k8"][b, h].float().double() * s["ks"][b, h].double()[block_of][:, None]
            v = s["v8"][b, h].float().double() * s["vs"][b, h].double()[block_of][:, None]
            for at in range(0, c["n"], 4096):
                rows = tokens[at: at + 4096]
                z = torch.mm(s["q"][b, h, rows].double(), k.t()).mul_(c["d"] ** -0.5)
                if s["pad"] is not None:
                    z += s["pad"][b].double()
                out[b, h, at: at + rows.numel()] = torch.softmax(z, -1) @ v
    return out
