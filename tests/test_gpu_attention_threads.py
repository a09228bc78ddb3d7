"""Host threads that share a GPU, each with its own stream, workspace and outputs."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def race(*bodies, rounds):
    """Runs the bodies in a thread each, started together; what they raised."""
    raised, start = [], threading.Barrier(len(bodies))

    def work(body):
        stream = torch.cuda.Stream()
        torch.zeros(1, device="cuda")  # the thread's first CUDA call
        try:
            start.wait()
            for _ in range(rounds):
                body(stream)
        except Exception as e:  # handed to the test
            raised.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_attention_with_and_without_the_mass(e4m3):
    """The two calls ask for different amounts of shared memory."""
    import sparse_attention_decode_gb300 as msa
    B, H, G, k, pages = 80, 4, 16, 32, 4  # more lists than clusters of two that run at once: no list is split
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn(pages, H, PAGE, D, device="cuda", generator=g)
    kv = kv.to(torch.float8_e4m3fn) if e4m3 else kv.to(torch.bfloat16)
    kv = kv.permute(0, 2, 1, 3)
    scale = torch.ones(pages, H, PAGE, device="cuda")
    q = torch.randn(B, H * G, D, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    seq = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    ids = torch.full((B, H, k), -1, dtype=torch.int32, device="cuda")
    ids[:, :, 5] = 0

    def body(mass):
        out, ws = torch.empty_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

        def call(stream):
            if e4m3:
                msa.msa_attention_sparse_fp8(q, kv, scale, kv, scale, table, seq, ids, out, ws, scale=0.1,
                                             out_mass=mass, stream=stream)
            else:
                msa.msa_attention_sparse(q, kv, kv, table, seq, ids, out, ws, scale=0.1, out_mass=mass, stream=stream)
        return call, out

    with_mass, a = body(torch.empty(B, H, k, device="cuda"))
    without, b = body(None)
    raised = race(with_mass, without, rounds=3000)
    torch.cuda.synchronize()
    assert not raised, raised[0]
    assert torch.equal(a, b)


def test_eviction_of_narrow_and_wide_tables():
    import sparse_attention_decode_gb300 as msa

    def body(cols):
        table = torch.arange(cols, dtype=torch.int32, device="cuda")[None].contiguous()
        seq = torch.full((1,), PAGE * cols, dtype=torch.int32, device="cuda")
        w = torch.rand(1, 1, cols, device="cuda")
        out = (torch.empty_like(table), torch.empty_like(seq), torch.empty_like(w), torch.empty_like(table),
               torch.empty_like(seq))
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        return (lambda stream: msa.msa_cache_evict(table, seq, w, 10, 1, 2, *out, ws, stream=stream)), out

    narrow, a = body(1028)
    wide, b = body(32768)
    raised = race(narrow, wide, rounds=3000)
    torch.cuda.synchronize()
    assert not raised, raised[0]
    assert a[1].item() == b[1].item() == 10 * PAGE
