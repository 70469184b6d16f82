"""A tensor that is missing is refused by the calls around the 8-bit state as by every other call of the binding."""
import pytest
import torch

from tests.gpu_util import expect_status, sd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attn_args():
    x = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(1, 1, 64, 64, dtype=torch.int8, device=DEV)
    f = torch.ones(1, 1, 1, device=DEV)
    return [x, c, f, c.clone(), f.clone(), 64, None, 0, None, 0.0, torch.zeros_like(x), 0]


@pytest.mark.parametrize("at", (0, 1, 2, 3, 4, 10))
def test_attention_without_a_tensor(at):
    args = attn_args()
    sd().safedit_attn_subset_state8(*args)  # key_pad and the index may be missing
    expect_status(0)
    args[at] = None
    with pytest.raises(sd().SafeditError) as e:
        sd().safedit_attn_subset_state8(*args)
    assert e.value.code == sd().ERR_INVALID_ARG


def test_rows_and_store_without_a_tensor():
    x = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16, device=DEV)
    c, f = torch.zeros(1, 1, 8, 64, dtype=torch.int8, device=DEV), torch.ones(1, 1, 1, device=DEV)
    pos, spec = torch.zeros(1, 8, 1, dtype=torch.int32, device=DEV), sd().rope_spec((64,), (1e4,))
    for call in (lambda: sd().safedit_rope_rows([x], [x], None, spec), lambda: sd().safedit_rope_rows([x], [None], pos, spec),
                 lambda: sd().safedit_rope_rows([x], [x], pos, None), lambda: sd().safedit_state8_store([None], [c], [f], 16),
                 lambda: sd().safedit_state8_store([x], [c], [None], 16),
                 lambda: sd().safedit_state8_store([x], [c], [f], 16, rotate=[True], rope=spec)):
        with pytest.raises(sd().SafeditError) as e:
            call()
        assert e.value.code == sd().ERR_INVALID_ARG
    expect_status(0)
