"""Verification where a row's largest logit, in units of the temperature, is large: its reference has to cancel exactly."""

import math

import pytest
import torch

from test_gpu_verify_draft import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V", [(torch.float32, 1), (torch.float32, 301), (torch.float32, 1023), (torch.bfloat16, 1),
                                     (torch.bfloat16, 301), (torch.bfloat16, 1021)], ids=str)
@pytest.mark.parametrize("top,temp", [(30000.0, 1.0), (100.0, 0.1), (37.3, 0.05)])
def test_the_largest_logit_past_the_last_whole_vector(dtype, V, top, temp):
    """A token that fills no 16-byte vector carries the row: its probability is 1 and its logarithm 0."""
    import sparse_attention_decode_gb300 as msa
    w = make(31, 3, 2, V, dtype)
    w["temp"][:] = temp
    w["logits"][..., -1] = top
    w["logits"][1, 1, V // 2] = top  # two tokens share the row, one of them inside a vector
    w["tokens"][0], w["u"][0] = V - 1, 0.5  # drafts that carry their rows are accepted
    w["tokens"][1, 0], w["u"][1, 0] = V - 1, 0.5
    assert check(msa, w) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("temp", [1e-6, 3e-8, 1e-8, 1e-12, 1e-30, 1e-39])
def test_temperatures_next_to_zero(dtype, temp):
    """p goes to one at the largest logit, shared where several are equal."""
    import sparse_attention_decode_gb300 as msa
    w = make(32, 6, 2, 517, dtype)
    w["temp"][:] = temp
    w["logits"][1, :, 7:9] = 11.0
    w["logits"][2] *= 0.0
    w["logits"][3] += 300.0
    w["logits"][4] -= 40.0
    assert check(msa, w) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_rows_of_nothing_but_the_lowest_value(dtype):
    """Equal logits are a uniform row, also at the type's lowest value; -inf beside them stays out."""
    import sparse_attention_decode_gb300 as msa
    w = make(33, 4, 2, 300, dtype)
    w["logits"][:] = torch.finfo(dtype).min
    w["logits"][1, :, ::2] = -math.inf
    w["logits"][2] = torch.finfo(dtype).max
    w["temp"][3] = 0.3
    assert check(msa, w) == 0


def test_an_infinite_temperature_is_a_uniform_row():
    import sparse_attention_decode_gb300 as msa
    w = make(34, 3, 2, 301, torch.float32)
    w["temp"][:] = math.inf
    assert check(msa, w) == 0
