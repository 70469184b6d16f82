"""Rotary positions far out, in segments of many pairs whose frequencies fall slowly.

Tolerance per element, as for the ordinary positions but for the angle:
  |got - y| <= 2^-24 |y| + (2^-21 + 2^-19.9) (|a| + |b|)
  - a frequency rounded to fp64 is off by 2^-53 of itself, and so is its product with the position, on either side: four
    times 2^31 * 2^-53 radians at the farthest, 2^-20, and the position in turns another 2^28.4 * 2^-54 * 2 pi;
  - nothing more, however many pairs a segment has.
"""
import pytest
import torch

from tests.gpu_util import expect_status, sd
from tests.test_gpu_rope import reference, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("halves", (False, True))
@pytest.mark.parametrize("axes, thetas", (((256,), (1.5,)), ((256,), (10.0,)), ((128, 128), (1e4, 2.0)), ((96,), (500.0,))))
def test_wide_segments_at_far_positions(halves, axes, thetas):
    d, n = max(sum(axes), 96), 64
    spec = sd().rope_spec(axes, thetas, sd().ROPE_HALVES if halves else sd().ROPE_INTERLEAVED)
    x = rows((1, 2, n, d), torch.float32, 1)
    at = (2 ** 31 - 1 - 37 * torch.arange(n)).to(torch.int32)
    pos = at[None, :, None].expand(1, n, len(axes)).to(x.device)
    y = torch.empty_like(x)
    sd().safedit_rope_rows([x], [y], pos, spec)
    expect_status(0)
    ref, mag = reference(x, pos, axes, thetas, halves, False)
    err = (y.double().cpu() - ref).abs()
    most = 2.0 ** -24 * ref.abs() + (2.0 ** -21 + 2.0 ** -19.9) * mag
    assert bool((err <= most).all()), f"worst error/bound {float((err / most.clamp_min(1e-300)).max()):.2f}"
