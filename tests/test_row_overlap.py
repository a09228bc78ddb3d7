"""Outputs that overlap strided inputs are refused, those that lie between their rows are not; by the library's own answer,
against sets of bytes.  Host only: the addresses are placeholders that are never dereferenced."""

import ctypes
import random
import time

import pytest
import torch

import test_attention_abi as abi

lib = abi.lib
BASE, FAR = 1 << 30, 1 << 44
REFUSED, PAST_EVERY_CHECK = 1, 4  # (there is no GPU behind the checks here)


@pytest.fixture(autouse=True)
def host_only():
    if torch.cuda.is_available():
        pytest.skip("host-only check: never hand placeholder pointers to a process with a GPU")


def at(n):
    return ctypes.c_void_p(n)


def append(**kw):
    """Addresses in bytes, strides in elements; what is not given is far away."""
    from sparse_attention_decode_gb300 import _attention as A, _serving  # noqa: F401
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)
    rows = kw.pop("rows", 4)
    a = dict(q=FAR, qs=1024, qh=1, oq=2 * FAR, os=1024, k=3 * FAR, ks=1024, v=4 * FAR, vs=1024, heads=1)
    a.update(kw)
    for n in ("q", "oq", "k", "v"):
        a[n] = at(a[n])
    far = at(5 * FAR)
    return A._fn("msa_cache_append")(*a.values(), None, None, 1e-6, far, 64, 0, None, far, st, far, st, 10, far, 8, far, far,
                                     rows, 1, 0, 1024, far, 256, None)


def shared(a, a_stride, a_width, b, b_stride, b_width, rows):
    """All in units of 16 bytes."""
    covered = {a + i * a_stride + j for i in range(rows) for j in range(a_width)}
    return any(b + i * b_stride + j in covered for i in range(rows) for j in range(b_width))


@pytest.mark.parametrize("against", ["q", "k", "v"])
def test_rows_of_the_append(lib, against):
    """Rows of out_q, 1 or 2 heads of 256 bytes, beside rows of one input."""
    r = random.Random({"q": 1, "k": 2, "v": 3}[against])
    seen = set()
    for _ in range(3000):
        rows, heads, mine = r.randint(1, 7), r.randint(1, 2), r.randint(1, 2)
        other = heads if against == "q" else mine
        sizes = [16 * heads + r.choice([0, r.randint(0, 6), r.randint(0, 60)]), 16 * other + r.choice([0, 1, r.randint(0, 60)])]
        if r.random() < 0.4:
            sizes[1] = sizes[0] = max(sizes)
        shift = r.randint(-140, 140)
        if against == "q" and shift == 0:
            continue  # in place
        want = shared(0, sizes[0], 16 * heads, shift, sizes[1], 16 * other, rows)
        kw = {"oq": BASE, "os": sizes[0] * 8, "qh": heads, "qs": 8 * 1024, "heads": mine, against: BASE + 16 * shift,
              {"q": "qs", "k": "ks", "v": "vs"}[against]: sizes[1] * 8, "rows": rows}
        assert append(**kw) == (REFUSED if want else PAST_EVERY_CHECK), (kw, want)
        seen.add((want, sizes[0] == sizes[1], rows > 1))
    assert len(seen) >= 7


def test_in_place_queries(lib):
    assert append(q=BASE, qs=2048, oq=BASE, os=2048) == PAST_EVERY_CHECK
    assert append(q=BASE, qs=2048, oq=BASE, os=1024) == REFUSED
    assert append(q=BASE, qs=2048, oq=BASE + 256, os=2048) == PAST_EVERY_CHECK  # a row of one head is 256 bytes
    assert append(q=BASE, qs=2048, oq=BASE + 240, os=2048) == REFUSED
    assert append(q=BASE, qs=2048, qh=2, oq=BASE + 256, os=2048) == REFUSED     # a head on


def test_many_rows_of_any_distance_are_looked_at_at_once(lib):
    """2^20 rows whose strides come together after 2^11 rows, or never share a byte."""
    start = time.perf_counter()
    n, kw = 1 << 20, dict(oq=BASE, os=8 * 2048 + 8, rows=1 << 20)
    assert append(**kw, q=BASE + 256, qs=8 * 2048) == REFUSED
    assert append(oq=BASE, os=4096, rows=n, q=BASE + 256, qs=8192) == PAST_EVERY_CHECK
    assert append(oq=BASE, os=4096, rows=n, q=BASE + 256 - 16, qs=8192) == REFUSED
    assert append(oq=BASE, os=6144, rows=n, k=BASE + 2 * n * 4096 + 1024, ks=4096) == PAST_EVERY_CHECK
    assert time.perf_counter() - start < 1.0


def paged(q, qs, out, batch, heads):
    from sparse_attention_decode_gb300 import _attention as A, _serving  # noqa: F401
    st, far = A._Strides(4 * 128 * 128, 128, 128 * 128), at(FAR)
    return A._fn("msa_attention_paged")(at(q), qs, far, st, far, st, 10, far, 8, far, batch, 1, heads, 1, 1024, 1.0, at(out), None,
                                        far, 1 << 40, None)


def test_output_of_the_attention_over_all_pages(lib):
    """An output between two query rows is no overlap."""
    assert paged(BASE, 1024, BASE + 512, 2, 1) == PAST_EVERY_CHECK  # rows of 256 bytes, 2 KiB apart; 512 bytes of output
    assert paged(BASE, 1024, BASE + 2048 - 512, 2, 1) == PAST_EVERY_CHECK
    assert paged(BASE, 1024, BASE + 240, 2, 1) == paged(BASE, 1024, BASE + 2048 - 496, 2, 1) == REFUSED
    r, seen = random.Random(4), set()
    for _ in range(3000):
        rows, heads = r.randint(1, 6), r.randint(1, 2)
        stride, shift = 16 * heads + r.choice([0, r.randint(0, 200)]), r.randint(-250, 700)
        want = shared(0, stride, 16 * heads, shift, 16 * heads, 16 * heads, rows)
        assert paged(BASE, stride * 8, BASE + 16 * shift, rows, heads) == (REFUSED if want else PAST_EVERY_CHECK)
        seen.add((want, rows > 1, 0 < shift < (rows - 1) * stride))
    assert len(seen) >= 5
