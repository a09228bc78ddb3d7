"""The split of attention over all pages as the kernels have it: csrc/paged_split.cuh compiled for the host and asked what each
CTA takes of random batches, and where the join looks for the parts of cut units."""

import ctypes
import os
import random
import re
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_decode_gb300", "csrc")
LEADS = [int(x) for x in re.search(r"kPagedLead\[2\] = \{(\d+), (\d+)\}", open(os.path.join(CSRC, "paged.cu")).read()).groups()]


def compiled(tmp, *more):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    out = os.path.join(tmp, "paged_split.so")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", *more, f"-I{CSRC}", "-o", out,
                    os.path.join(ROOT, "tests", "paged_split_host.cpp")], check=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("split")))


def check(host, lens, limit, row_tiles, kv_heads, lead, grid, threads):
    seq = (ctypes.c_int32 * (len(lens) + 1))(*lens)
    batch = (seq, limit, len(lens), row_tiles, kv_heads, lead, grid)
    length = [n if 0 <= n <= limit else 0 for n in lens]
    pages = {(b, u): -(-n // 128) for b, n in enumerate(length) for u in range(row_tiles * kv_heads) if n}
    out = np.zeros((sum(pages.values()) + 1, 7), dtype=np.int32)
    into = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))  # noqa: E731
    n = host.taken(*batch, threads, into(out), len(out))
    assert n >= 0
    rows = {}
    for cta, part, b, u, j, run, tokens in out[:n].tolist():
        assert run > 0 and 0 <= part < 2 * grid and part // 2 == cta and tokens == length[b]
        rows.setdefault((b, u), []).append((j, run, cta, part))
    assert sorted(rows) == sorted(pages)
    used, cut = {}, {}
    for at, n in pages.items():
        assert [r[0] for r in rows[at]] == [sum(r[1] for r in rows[at][:i]) for i in range(len(rows[at]))]  # each page once, in order
        assert sum(r[1] for r in rows[at]) == n
        got = np.full(len(rows[at]) + 2, -1, dtype=np.int32)
        count = host.parts_of_unit(*batch, *at, into(got), len(got))
        assert count == len(rows[at])
        if count > 1:
            assert got[:count].tolist() == [r[3] for r in rows[at]]
            cut[at] = got[:count].tolist()
            for r in rows[at]:
                assert used.setdefault(r[3], at) == at  # a part is one unit's
    found = {}
    for x in range(grid - 1):
        got = np.full(2 * grid + 2, -1, dtype=np.int32)
        count = host.parts_at_end(*batch, threads, x, into(got), len(got))
        if count:
            assert tuple(got[:2].tolist()) not in found  # one block a unit
            found[tuple(got[:2].tolist())] = got[2:2 + count].tolist()
    assert found == cut


@pytest.mark.parametrize("lead", LEADS)
def test_random_batches(host, lead):
    r = random.Random(9)
    for _ in range(600):
        lens = [r.choice([0, 1, 127, 128, 129, r.randint(0, 700), r.randint(0, 7000), -3, 10 ** 6]) for _ in range(r.choice([1, 2, 5, 40]))]
        check(host, lens, 8000, r.choice([1, 1, 2, 3]), r.choice([1, 2, 4, 8]), lead, r.choice([1, 2, 7, 152]),
              r.choice([256, 288, 352, 576]))


@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("lens", [[1], [8700], [131072], [10600, 0, 1, 4800, 1, 19100, 61637, 49000], [200] * 700, [128] * 37 + [60000],
                                  [0, 0], [0] * 300 + [5] + [0] * 300], ids=lambda n: f"{len(n)}x{max(n)}")
def test_batches(host, lens, lead):
    check(host, lens, 131072, 1, 4, lead, 152, 352)


@pytest.mark.parametrize("mistake", [("longer = more * (range + 1)", "longer = more * range"), ("< from - lead", "<= from - lead"),
                                     ("(g < more ? g : more)", "0"), ("left += j < 0 ? j : 0;", ""),
                                     ("left -= run() + p.lead;", "left -= run();"), ("x - from - u * each - p.lead", "x - from - u * each")])
def test_the_check_sees_a_mistake_in_the_source(tmp_path, mistake):
    text = open(os.path.join(CSRC, "paged_split.cuh")).read()
    assert text.count(mistake[0]) == 1
    (tmp_path / "paged_split.cuh").write_text(text.replace(*mistake))
    wrong = compiled(str(tmp_path), f"-I{tmp_path}")
    with pytest.raises(AssertionError):
        test_random_batches(wrong, LEADS[0])
