"""The serving operators' C ABI: include/msa_attention.h, the binding and the library agree; refusals before any GPU work."""

import ctypes
import os
import re
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "msa_attention.h")


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no CUDA toolkit")
    from sparse_attention_decode_gb300 import build
    build.build()
    import sparse_attention_decode_gb300 as msa
    return msa.load()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def declared():
    return sorted(set(re.findall(r"\b(msa_\w+)\s*\(", header())))


def test_header_binding_and_library_agree(lib):
    import sparse_attention_decode_gb300 as msa
    assert declared() == sorted(msa.ATTENTION_EXPORTED)
    for name in declared():
        assert callable(getattr(msa, name)) and hasattr(lib, name), name
    for name, value in re.findall(r"#define (MSA_\w+) (0x[0-9a-f]+|\d+)u?", header()):
        assert getattr(msa, name) == int(value, 0), name


def test_the_binding_passes_as_many_arguments_as_the_header_declares():
    from sparse_attention_decode_gb300 import _attention
    for name, args in re.findall(r"\b(msa_\w+)\s*\(([^)]*)\)", header()):
        assert len(_attention._ARGTYPES[name][0]) == len(args.split(",")), name


def test_prefix_workspace_bytes(lib):
    import sparse_attention_decode_gb300 as msa
    n = msa.msa_attention_prefix_workspace_bytes
    assert n(2, 64, 4, 4133) == 256 + ((256 + 4) * 256 + 2 * 64) * 129 * 4 + 1024
    sizes = [n(r, 64, 4, 4096) for r in (1, 8, 9, 16, 17, 1000)]
    assert sizes == sorted(sizes)
    assert [n(-1, 64, 4, 1), n(1, 3, 4, 1), n(1, 6, 4, 1), n(1, 4, 0, 1), n(1, 4, 4, -1)] == [0] * 5


def test_null_pointers_and_bad_sizes_are_refused_before_any_gpu_work(lib):
    import torch
    from sparse_attention_decode_gb300 import _attention as A
    if torch.cuda.is_available():
        pytest.skip("host-only check: never hand placeholder pointers to a process with a GPU")
    fake = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)

    def sparse(**kw):
        a = dict(q=fake, qs=512, k=fake, ks=st, v=fake, vs=st, pages=10, table=fake, stride=8, seq=fake, batch=2, q_len=1,
                 heads=4, group=1, limit=1024, ids=fake, sel=4, topk=16, scale=1.0, out=fake, lse=None, mass=None,
                 ws=fake, bytes=256, stream=None)
        a.update(kw)
        return A._fn("msa_attention_sparse")(*a.values())

    assert sparse(q=None) == 1 and sparse(k=None) == 1 and sparse(ids=None) == 1 and sparse(ws=None) == 1
    assert sparse(scale=0.0) == 1 and sparse(scale=float("nan")) == 1 and sparse(sel=3) == 1 and sparse(topk=0) == 1
    assert sparse(qs=511) == 1 and sparse(qs=256) == 1 and sparse(ks=A._Strides(4 * 128 * 128, 4, 128 * 128)) == 1
    assert sparse(ks=A._Strides(4 * 128 * 128, 132, 128 * 128)) == 1 and sparse(q=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert sparse(topk=33) == 2 and sparse(group=65, qs=4 * 65 * 128) == 2 and sparse(batch=5000) == 2
    assert sparse(pages=1 << 25) == 2 and sparse(bytes=255) == 3 and sparse(batch=0) == 0

    def prefix(**kw):
        a = dict(q=fake, qs=512, k=fake, ks=st, v=fake, vs=st, pages=10, shared=fake, n=fake, bound=1000, table=fake,
                 stride=8, seq=fake, batch=2, q_len=1, heads=4, group=1, limit=1024, scale=1.0, out=fake, lse=None,
                 ws=fake, bytes=1 << 40, stream=None)
        a.update(kw)
        return A._fn("msa_attention_prefix")(*a.values())

    assert prefix(shared=None) == 1 and prefix(n=None) == 1 and prefix(bound=-1) == 1 and prefix(scale=-1.0) == 1
    assert prefix(batch=5000) == 2 and prefix(q_len=65) == 2 and prefix(bytes=1000) == 3 and prefix(batch=0) == 0

    def evict(**kw):
        a = dict(table=fake, stride=8, seq=fake, w=fake, cols=8, batch=1, heads=2, limit=1024, budget=4, sink=1, window=2,
                 out=fake, ostride=8, oseq=fake, ow=fake, freed=fake, n=fake, ws=fake, bytes=256, stream=None)
        a.update(kw)
        return A._fn("msa_cache_evict")(*a.values())

    assert evict(w=None) == 1 and evict(window=0) == 1 and evict(budget=2) == 1 and evict(stride=7) == 1
    assert evict(cols=40000, stride=40000, ostride=40000) == 2 and evict(bytes=0) == 3 and evict(batch=0) == 0

    def verify(**kw):
        a = dict(logits=fake, bf16=0, sb=400, si=100, draft=fake, tokens=fake, u=fake, race=fake, temp=None, n=None,
                 batch=2, drafts=3, vocab=100, out=fake, acc=fake, lp=None, ws=fake, bytes=256, stream=None)
        a.update(kw)
        return A._fn("msa_verify_draft")(*a.values())

    assert verify(logits=None) == 1 and verify(si=99) == 1 and verify(vocab=0) == 1 and verify(draft=None) == 1
    assert verify(logits=ctypes.c_void_p((1 << 20) + 1)) == 1 and verify(drafts=64, sb=6500) == 2 and verify(bytes=9) == 3
    assert verify(batch=0) == 0 and verify(draft=None, drafts=0, batch=0) == 0
    f = A._fn("msa_cache_accumulate")
    assert f(fake, 8, fake, fake, None, 1, 1, 2, 2, 33, fake, 256, None) == 2
    assert f(None, 8, fake, fake, None, 1, 1, 2, 2, 3, fake, 256, None) == 1
    assert f(fake, 8, fake, fake, None, 1, 1, 3, 2, 3, fake, 256, None) == 1


def test_tensors_off_the_gpu_and_wrong_layouts_are_refused():
    import torch
    import sparse_attention_decode_gb300 as msa
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(AssertionError, match="one CUDA device"):
        msa.msa_cache_accumulate(z(1, 2, 8), z(1, 2, 3, dtype=torch.int32), z(1, 2, 3), z(256, dtype=torch.uint8))
    with pytest.raises(AssertionError, match="one CUDA device"):
        msa.msa_verify_draft(z(1, 2, 9), z(1, 1, 9), z(1, 1, dtype=torch.int32), z(1, 1), z(1, 9),
                             z(1, 2, dtype=torch.int32), z(1, dtype=torch.int32), z(256, dtype=torch.uint8))
