"""CPU replay of the E4M3 terms of the attention over all pages, for every bf16 query mantissa and every f16 weight."""

import os
import re

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_decode_gb300", "csrc", "paged_attn.cuh")).read()


def terms_of(name):
    """(what goes into each term, what comes back out of it, the terms' unit over the one before), as the kernel has them."""
    body = re.search(r"struct %s \{(.*?)\n\};" % name, SRC, re.S).group(1)
    f16 = lambda what: [torch.tensor(int(x, 16) & 0xFFFF, dtype=torch.int32).to(torch.int16).view(torch.float16).double().item()  # noqa: E731
                        for x in re.findall(r"0x[0-9a-f]+", re.search(what + r"\[\w+\] = \{(.*?)\}", body).group(1))]
    step = 1.0 / float(re.search(r"kStep = 1\.0f / (\d+)\.0f", body).group(1))
    return f16("kDown"), f16("kBack"), step


def held(name, x):
    """x (f16 values in 64 bits) as the sum of its terms, in 64 bits; every operation in f16 as in the kernel."""
    down, back, step = terms_of(name)
    left, total = x.clone(), torch.zeros_like(x)
    for i, d in enumerate(down):
        code = (left * d).to(torch.float16).float().clamp(-448, 448).to(torch.float8_e4m3fn).double()
        total += code / down[0] * step ** i
        if i + 1 < len(down):
            exact = left + code * back[i]
            left = exact.to(torch.float16).double()
            assert torch.equal(left, exact)  # what a term leaves is exact
            assert back[i] == -step ** i / down[0]
    return total


def test_query_values():
    mantissas = 1 + torch.arange(128).double() / 128
    x = torch.cat([mantissas * 2.0 ** e for e in range(-40, 15)]).to(torch.float16).double()
    kept = torch.cat([mantissas * 2.0 ** e for e in range(-40, 15)])
    for sign in (1.0, -1.0):
        off = (held("QueryTerms", sign * x) - sign * kept).abs()
        assert not bool(off[kept >= 1.0].any())  # the row's largest is below 2^15: 2^-14 of it and more
        assert float(off.max()) <= 2.0 ** -8     # and at least 2^14: 2^-22 of it


def test_weights():
    """Products of weight and V scale, the largest of a row at 2^9 to 2^10 when its unit was chosen, 2^15 at most since."""
    x = torch.arange(1, 0x7801, dtype=torch.int32).to(torch.int16).view(torch.float16).double()
    assert float(x.max()) == 2.0 ** 15
    off = (held("WeightTerms", x) - x).abs()
    # 2^-9 in the terms, 2^-11 before in f16: 2^-8 of itself, or 2^-21 of 2^9
    assert bool(((off <= 2.0 ** -8.5 * x) | (off <= 2.0 ** -12.5)).all())
