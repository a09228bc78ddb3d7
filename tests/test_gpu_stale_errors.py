"""A call answers for its own launches: an error that an earlier runtime call left behind in the thread is not its own."""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def runtimes():
    """The CUDA runtimes of this process."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line}
    return [ctypes.CDLL(p) for p in sorted(paths)]


def test_accumulation_after_a_failed_runtime_call():
    import sparse_attention_decode_gb300 as msa
    w = torch.zeros(1, 1, 4, device="cuda")
    ids = torch.tensor([[[2, 0]]], dtype=torch.int32, device="cuda")
    mass = torch.tensor([[[3.0, 4.0]]], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    msa.load()
    found = runtimes()
    assert found
    try:
        for rt in found:
            assert rt.cudaSetDevice(12345) != 0  # refused on the host; the error stays in the thread
        msa.msa_cache_accumulate(w, ids, mass, ws)
    finally:
        for rt in found:
            rt.cudaGetLastError()
    assert w.flatten().tolist() == [4.0, 0.0, 3.0, 0.0]
    assert msa.msa_indexer_get_error(ws) == 0
