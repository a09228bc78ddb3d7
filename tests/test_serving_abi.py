"""The C ABI of include/msa_serving.h: header, binding and library agree; refusals before any GPU work."""

import ctypes
import os
import re

import pytest
import torch

import test_attention_abi as abi

lib = abi.lib
HEADER = os.path.join(abi.ROOT, "include", "msa_serving.h")


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_binding_and_library_agree(lib):
    import sparse_attention_decode_gb300 as msa
    names = sorted(set(re.findall(r"\b(msa_\w+)\s*\(", header())))
    assert names == sorted(msa.SERVING_EXPORTED)
    for name in names:
        assert callable(getattr(msa, name)) and hasattr(lib, name), name
    for name, value in re.findall(r"#define (MSA_\w+) (0x[0-9a-f]+|\d+)u?", header()):
        assert getattr(msa, name) == int(value, 0), name


def test_the_binding_passes_as_many_arguments_as_the_header_declares():
    from sparse_attention_decode_gb300 import _serving
    for name, args in re.findall(r"\b(msa_\w+)\s*\(([^)]*)\)", header()):
        assert len(_serving._ARGTYPES[name][0]) == len(args.split(",")), name


def test_null_pointers_and_bad_sizes_are_refused_before_any_gpu_work(lib):
    from sparse_attention_decode_gb300 import _attention as A, _serving  # noqa: F401
    if torch.cuda.is_available():
        pytest.skip("host-only check: never hand placeholder pointers to a process with a GPU")
    fake, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)  # never dereferenced: validation fails first
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)

    def append(**kw):
        a = dict(q=fake, qs=1024, qh=8, oq=fake, os=1024, k=fake, ks=512, v=fake, vs=512, heads=4, qw=None, kw=None, eps=1e-6,
                 freq=fake, rot=64, inter=0, pos=None, kc=fake, kst=st, vc=fake, vst=st, pages=10, table=fake, stride=8,
                 seq=fake, cu=None, rows=4, batch=2, q_len=2, limit=1024, ws=fake, bytes=256, stream=None)
        a.update(kw)
        return A._fn("msa_cache_append")(*a.values())

    for kw in (dict(k=None), dict(kc=None), dict(vc=None), dict(v=None), dict(oq=None), dict(q=None), dict(freq=None),
               dict(seq=None), dict(table=None), dict(ws=None), dict(k=odd), dict(q=odd), dict(ks=511), dict(ks=504),
               dict(qs=1000), dict(os=1016), dict(rows=3), dict(q_len=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(rot=-16), dict(heads=0), dict(qh=0), dict(batch=-1), dict(pages=0),
               dict(kst=A._Strides(4 * 128 * 128, 4, 128 * 128)), dict(ws=odd)):
        assert append(**kw) == 1, kw
    for kw in (dict(rot=24), dict(rot=144), dict(batch=5000, rows=10000), dict(pages=1 << 25), dict(heads=2000, ks=256000)):
        assert append(**kw) == 2, kw
    assert append(bytes=255) == 3
    assert append(batch=0, rows=0) == 0 and append(batch=0, rows=0, k=None, q=None, oq=None, ws=None) == 0
    assert append(v=None, vc=None) == 4 and append(cu=fake, rows=3, q_len=0) == 4  # past every check: there is no GPU here

    def paged(**kw):
        a = dict(q=fake, qs=512, k=fake, ks=st, v=fake, vs=st, pages=10, table=fake, stride=8, seq=fake, batch=2, q_len=1,
                 heads=4, group=1, limit=1024, scale=1.0, out=fake, lse=None, ws=fake, bytes=1 << 40, stream=None)
        a.update(kw)
        return A._fn("msa_attention_paged")(*a.values())

    for kw in (dict(q=None), dict(k=None), dict(out=None), dict(ws=None), dict(table=None), dict(seq=None), dict(scale=0.0),
               dict(scale=float("nan")), dict(q=odd), dict(qs=511), dict(qs=256), dict(group=0), dict(limit=0),
               dict(ks=A._Strides(4 * 128 * 128, 132, 128 * 128))):
        assert paged(**kw) == 1, kw
    assert paged(group=65, qs=4 * 65 * 128) == 2 and paged(batch=5000) == 2 and paged(q_len=65) == 2 and paged(pages=1 << 25) == 2
    assert paged(bytes=100) == 3 and paged(batch=0) == 0

    def logprobs(**kw):
        a = dict(logits=fake, bf16=0, stride=100, tokens=fake, given=2, temp=None, rows=3, vocab=100, n=4, out=fake, ent=None,
                 ids=fake, top=fake, ws=fake, bytes=256, stream=None)
        a.update(kw)
        return A._fn("msa_token_logprobs")(*a.values())

    for kw in (dict(logits=None), dict(tokens=None), dict(out=None), dict(ids=None), dict(top=None), dict(ws=None),
               dict(logits=odd), dict(stride=99), dict(vocab=0), dict(given=-1), dict(n=-1), dict(rows=-1), dict(ws=odd)):
        assert logprobs(**kw) == 1, kw
    assert logprobs(n=33) == 2 and logprobs(given=257) == 2 and logprobs(vocab=1 << 25, stride=1 << 25) == 2
    assert logprobs(bytes=9) == 3 and logprobs(rows=0) == 0 and logprobs(rows=0, logits=None, ws=None) == 0


def test_overlaps_and_sizes_past_32_bits_are_refused(lib):
    from sparse_attention_decode_gb300 import _attention as A, _serving  # noqa: F401
    if torch.cuda.is_available():
        pytest.skip("host-only check: never hand placeholder pointers to a process with a GPU")
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)

    def paged(**kw):
        a = dict(q=at(0), qs=512, k=at(0), ks=st, v=at(0), vs=st, pages=10, table=at(0), stride=8, seq=at(0), batch=4, q_len=1,
                 heads=4, group=1, limit=1024, scale=1.0, out=at(1 << 16), lse=None, ws=at(0), bytes=1 << 40, stream=None)
        a.update(kw)
        return A._fn("msa_attention_paged")(*a.values())

    assert paged() == 4  # past every check: there is no GPU here
    for n in (0, 16, 4096 - 16):  # four rows of 1024 bytes
        assert paged(out=at(n)) == 1 and paged(q=at(n), out=at(0)) == 1, n
    assert paged(out=at(4096)) == 4 and paged(q=at(4096), out=at(0)) == 4
    assert paged(qs=1024, out=at(4096)) == 1 and paged(qs=1024, out=at(7168)) == 4  # the last row ends at 7 KiB
    big = dict(stride=1 << 24, limit=(1 << 31) - 1, out=at(1 << 40))
    assert paged(**big, batch=8) == 4 and paged(**big, batch=17) == 2


def test_paged_workspace_bytes(lib):
    import sparse_attention_decode_gb300 as msa
    n = msa.msa_attention_paged_workspace_bytes
    assert [n(-1, 64, 4), n(1, 3, 4), n(1, 6, 4), n(1, 4, 0)] == [0] * 4
    sizes = [n(r, 64, 4) for r in (0, 1, 2, 4, 8, 100, 10000)]
    assert sizes == sorted(sizes) and sizes[0] >= 256


class Stand:
    """The parts of a tensor that the binding looks at; `device` as if on that GPU."""

    def __init__(self, shape, dtype=torch.float32, stride=None, device=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self._stride = tuple(stride) if stride else torch.empty(shape, device="meta").stride()
        self.nbytes = 4 * self.shape.numel()

    def stride(self):
        return self._stride

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self._stride == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 0 if 0 in self.shape else 1 << 20


I32, BF16, U8 = torch.int32, torch.bfloat16, torch.uint8


@pytest.fixture
def calls(monkeypatch):
    """The library replaced by a recorder; device 0 is current."""
    from sparse_attention_decode_gb300 import _attention as A, _serving  # noqa: F401
    got = []

    def entry(name):
        def call(*args):
            assert len(args) == len(A._ARGTYPES[name][0])
            got.append((name, args))
            return 0
        return call
    monkeypatch.setattr(A, "_fn", entry)
    monkeypatch.setattr(A, "_current_device", lambda: 0)
    monkeypatch.setattr(A, "_stream", lambda stream, t: 0)
    return got


def append(device=0, cols=8, stride=8, **kw):
    from sparse_attention_decode_gb300 import _serving as S
    t = lambda *s, dtype=BF16, stride=None: Stand(s, dtype, stride, device)  # noqa: E731
    S.msa_cache_append(t(2, 2, 128, stride=(2560, 128, 1)), t(2, 2, 128, stride=(2560, 128, 1)), t(10, 128, 2, 128),
                       t(10, 128, 2, 128), t(2, cols, dtype=I32, stride=(stride, 1)), t(2, dtype=I32), t(256, dtype=U8),
                       q=t(2, 16, 128, stride=(2560, 128, 1)), out_q=t(2, 16, 128), inv_freq=t(32, dtype=torch.float32), **kw)


def paged(device=0, cols=8, stride=8, **kw):
    from sparse_attention_decode_gb300 import _serving as S
    t = lambda *s, dtype=BF16, stride=None: Stand(s, dtype, stride, device)  # noqa: E731
    S.msa_attention_paged(t(2, 8, 128), t(10, 128, 2, 128), t(10, 128, 2, 128), t(2, cols, dtype=I32, stride=(stride, 1)),
                          t(2, dtype=I32), t(2, 8, 128), t(256, dtype=U8), scale=0.1, **kw)


def logprobs(device=0):
    from sparse_attention_decode_gb300 import _serving as S
    t = lambda *s, dtype=torch.float32: Stand(s, dtype, device=device)  # noqa: E731
    S.msa_token_logprobs(t(2, 9), t(2, 3, dtype=I32), t(2, 3), t(256, dtype=U8))


@pytest.mark.parametrize("call", [append, paged, logprobs])
def test_tensors_on_a_gpu_that_is_not_current_are_refused(calls, monkeypatch, call):
    from sparse_attention_decode_gb300 import _attention as A
    call()
    assert len(calls) == 1
    with pytest.raises(AssertionError, match="current"):
        call(device=1)
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    call(device=1)
    assert len(calls) == 2
    with pytest.raises(AssertionError, match="current"):
        call()


@pytest.mark.parametrize("call,limit_at", [(append, 29), (paged, 14)])
def test_a_request_is_no_longer_than_its_columns_of_the_table(calls, call, limit_at):
    for given, want in ((None, 1024), (700, 700), (12800, 1024)):
        calls.clear()
        call(max_model_len=given, cols=8, stride=100)
        assert calls[0][1][limit_at] == want and 100 in calls[0][1]


def test_the_distances_of_a_projection_s_rows_are_passed_on(calls):
    append()
    args = calls[0][1]
    assert args[1] == 2560 and args[2] == 16 and args[4] == 2048 and args[6] == args[8] == 2560 and args[14] == 64
