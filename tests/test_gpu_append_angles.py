"""Rotation at the last positions and the largest frequencies, against angles reduced exactly."""

import math
from fractions import Fraction

import pytest
import torch

import test_gpu_cache_append as append

pytestmark = pytest.mark.gpu

TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")  # 80 digits


def reduced(position, freq):
    x = Fraction(position) * Fraction(freq)  # a fp32 value is a fraction
    return float(x - TURN * round(x / TURN))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
def test_angles_of_the_last_positions(monkeypatch, inter, e4m3):
    import sparse_attention_decode_gb300 as msa
    w = append.make(95, [40], [8], 2, 4, 32, inter, False, "hnd", e4m3)
    w["inv"] = torch.tensor([1.0, 1024.0, -1024.0, 1023.9999, 700.3, 0.1, 3.1415927, 1e-3, 2.0 ** -31, 1e-9, 1e-20, 1e-45, 0.0,
                             -6.2831855, 511.5, 2.0 ** -100])
    w["positions"] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 77, 2 ** 30 + 1, -(2 ** 29) - 3, 1987654321, 2 ** 24 + 1, 1],
                                  dtype=torch.int32)
    angle = torch.tensor([[reduced(int(p), float(f)) for f in w["inv"].double()] for p in w["positions"].tolist()],
                         dtype=torch.float64)
    formula = append.plain

    def plain(x, weight, eps, at, inv_freq, is_inter):
        if inv_freq is None:
            return formula(x, weight, eps, at, inv_freq, is_inter)
        y = x.double()
        z, size = y.clone(), y.abs()
        a, b = (slice(0, 32, 2), slice(1, 32, 2)) if is_inter else (slice(0, 16), slice(16, 32))
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        z[..., a], z[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
        return z, size * 2.0 ** -19 + 1e-37  # as append.plain has it, with 2^-22 of the angle: 2^-20 + 2^-22 at most
    monkeypatch.setattr(append, "plain", plain)
    got = append.call(msa, w)
    assert got["fault"] == 0
    append.verify(w, got)


def test_the_reduction():
    assert reduced(0, 1.0) == 0.0 and abs(reduced(1, 1.0) - 1.0) < 1e-15
    assert abs(math.sin(reduced(10 ** 6, 1.0)) - math.sin(1e6)) < 1e-9
