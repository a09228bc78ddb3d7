"""The serving operators' binding on stand-ins for CUDA tensors: what it refuses, and the numbers it hands to C."""

import ctypes

import pytest
import torch

from sparse_attention_decode_gb300 import _attention as A


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


I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The library replaced by a recorder; device 0 is current."""
    got = []

    def entry(name):
        def call(*args):
            want = A._ARGTYPES[name][0]
            assert len(args) == len(want)
            got.append((name, args))
            return 0
        return call
    monkeypatch.setattr(A, "_fn", entry)
    monkeypatch.setattr(A, "_current_device", lambda: 0)
    monkeypatch.setattr(A, "_stream", lambda stream, t: 0)
    return got


def sparse(device=0, batch=2, cols=8, stride=8, **kw):
    d = dict(device=device)
    A.msa_attention_sparse(
        Stand((batch, 8, 128), BF16, **d), Stand((10, 128, 2, 128), BF16, **d), Stand((10, 128, 2, 128), BF16, **d),
        Stand((batch, cols), I32, (stride, 1), **d), Stand((batch,), I32, **d), Stand((batch, 2, 4), I32, **d),
        Stand((batch, 8, 128), BF16, **d), Stand((256,), torch.uint8, **d), scale=0.1, **kw)


def prefix(device=0, batch=2, cols=8, stride=8, pages=3, **kw):
    d = dict(device=device)
    A.msa_attention_prefix(
        Stand((batch, 8, 128), BF16, **d), Stand((10, 128, 2, 128), BF16, **d), Stand((10, 128, 2, 128), BF16, **d),
        Stand((pages,), I32, **d), Stand((1,), I32, **d), Stand((batch, cols), I32, (stride, 1), **d), Stand((batch,), I32, **d),
        Stand((batch, 8, 128), BF16, **d), Stand((256,), torch.uint8, **d), scale=0.1, **kw)


def accumulate(device=0):
    d = dict(device=device)
    A.msa_cache_accumulate(Stand((2, 2, 8), **d), Stand((2, 2, 4), I32, **d), Stand((2, 2, 4), **d),
                           Stand((256,), torch.uint8, **d))


def evict(device=0, **kw):
    t = lambda *s, dtype=I32: Stand(s, dtype, device=device)  # noqa: E731
    A.msa_cache_evict(t(2, 8), t(2), t(2, 2, 8, dtype=torch.float32), 4, 1, 2, t(2, 8), t(2), t(2, 2, 8, dtype=torch.float32),
                      t(2, 8), t(2), t(256, dtype=torch.uint8), **kw)


def verify(device=0):
    t = lambda *s, dtype=torch.float32: Stand(s, dtype, device=device)  # noqa: E731
    A.msa_verify_draft(t(2, 3, 9), t(2, 2, 9), t(2, 2, dtype=I32), t(2, 2), t(2, 9), t(2, 3, dtype=I32), t(2, dtype=I32),
                       t(256, dtype=torch.uint8))


@pytest.mark.parametrize("call", [sparse, prefix, accumulate, evict, verify])
def test_tensors_on_a_gpu_that_is_not_current_are_refused(calls, monkeypatch, call):
    """The kernels are launched on the current device: there the addresses would be another's."""
    call()
    assert len(calls) == 1
    with pytest.raises(AssertionError, match="current"):
        call(device=1)
    assert len(calls) == 1
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    call(device=1)  # the same call, once that device is current
    assert len(calls) == 2
    with pytest.raises(AssertionError, match="current"):
        call()
    assert len(calls) == 2


@pytest.mark.parametrize("call,limit_at", [(sparse, 14), (prefix, 17), (evict, 7)])
def test_a_request_is_no_longer_than_its_columns_of_the_table(calls, call, limit_at):
    """A table that is some columns of a wider one: what lies behind them is not the request's, and past the last row no
    one's."""
    columns = {} if call is evict else dict(cols=8, stride=100)
    for given, want in ((None, 1024), (700, 700), (1024, 1024), (12800, 1024), (1 << 20, 1024)):
        calls.clear()
        call(max_model_len=given, **columns)
        assert calls[0][1][limit_at] == want
    if columns:
        assert 100 in calls[0][1]  # the rows' distance is passed on as it is
