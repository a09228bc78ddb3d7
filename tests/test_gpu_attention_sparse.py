"""Attention over selected blocks against plain attention in 64 bits."""

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def make(seed, lens, q_len, H, G, sel, k, layout, e4m3, spare=2):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    cols = max(1, max(-(-n // PAGE) for n in lens))
    pages = sum(-(-n // PAGE) for n in lens) + spare
    kp, ks = ref.make_pool(g, pages, H, layout, e4m3)
    vp, vs = ref.make_pool(g, pages, H, layout, e4m3)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, cols), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        nb = -(-n // PAGE)
        table[b, :nb] = perm[at:at + nb]
        at += nb
    ref.spoil((kp, vp), table, lens)
    ids = torch.full((B * q_len, sel, k), -1, dtype=torch.int32)
    for r in range(B * q_len):
        nb = max(0, -(-(lens[r // q_len] - (q_len - 1 - r % q_len)) // PAGE))
        for h in range(sel):
            order = torch.randperm(nb, generator=g)[:k].to(torch.int32) if nb else torch.zeros(0, dtype=torch.int32)
            slots = torch.randperm(k, generator=g)[:len(order)]  # unused slots anywhere
            ids[r, h, slots] = order
    q = torch.randn(B * q_len, H * G, D, generator=g).to(torch.bfloat16)
    return dict(q=q, kp=kp, ks=ks, vp=vp, vs=vs, table=table, lens=lens, ids=ids, q_len=q_len, scale=D ** -0.5)


def call(msa, w, lse=True, mass=True, q=None, stream=None):
    dev = {n: ref.to_cuda(w[n]) for n in ("kp", "ks", "vp", "vs")}
    q = w["q"].cuda() if q is None else q
    R, Hq = q.shape[:2]
    H, k = w["kp"].shape[2], w["ids"].shape[2]
    out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o_lse = torch.full((R, Hq), 7.0, device="cuda") if lse else None
    o_mass = torch.full((R, H, k), 7.0, device="cuda") if mass else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    seq = torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    args = (w["table"].cuda(), seq, w["ids"].cuda(), out, ws)
    kw = dict(scale=w["scale"], q_len=w["q_len"], out_lse=o_lse, out_mass=o_mass, stream=stream)
    torch.cuda.synchronize()
    if w["ks"] is None:
        msa.msa_attention_sparse(q, dev["kp"], dev["vp"], *args, **kw)
    else:
        msa.msa_attention_sparse_fp8(q, dev["kp"], dev["ks"], dev["vp"], dev["vs"], *args, **kw)
    torch.cuda.synchronize()
    return out, o_lse, o_mass, msa.msa_indexer_get_error(ws)


def verify(msa, w, **kw):
    out, lse, mass, fault = call(msa, w, **kw)
    want = ref.sparse(w["q"], w["kp"], w["ks"], w["vp"], w["vs"], w["table"], w["lens"], w["ids"], w["scale"],
                      w["q_len"])
    ref.check(out, want[0], "out")
    if lse is not None:
        ref.check(lse, want[1], "lse")
    if mass is not None:
        ref.check(mass, want[2], "mass")
    return fault


CASES = [
    # lens, q_len, kv heads, group, selection heads, k, layout
    ([1], 1, 4, 16, 4, 16, "hnd"),
    ([0, 1, 127, 128, 129, 5000], 1, 4, 16, 4, 16, "hnd"),
    ([2, 0, 130, 3000], 4, 4, 6, 4, 16, "nhd"),
    ([700, 4097], 2, 8, 1, 4, 5, "wide"),
    ([2600], 1, 1, 13, 1, 32, "hnd"),
    ([300, 2000], 1, 2, 32, 1, 7, "nhd"),
    ([300, 2000, 640], 3, 2, 64, 2, 3, "hnd"),
    ([40, 9000], 1, 3, 17, 3, 1, "wide"),
    ([130 + 7 * i for i in range(90)], 1, 4, 16, 4, 16, "hnd"),  # no split of a list
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}q{c[1]}h{c[2]}g{c[3]}k{c[5]}{c[6]}")
def test_matches_64_bits(case, e4m3):
    import sparse_attention_decode_gb300 as msa
    lens, q_len, H, G, sel, k, layout = case
    assert verify(msa, make(11, lens, q_len, H, G, sel, k, layout, e4m3)) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_peaked_rows_and_large_values(e4m3):
    """One token takes nearly all weight; scores up to hundreds; V scales over four decades."""
    import sparse_attention_decode_gb300 as msa
    w = make(5, [1500, 900], 1, 4, 16, 4, 16, "hnd", e4m3)
    w["q"] = (w["q"].float() * 30).to(torch.bfloat16)
    if e4m3:
        w["vs"] = w["vs"] * torch.logspace(-3, 1, PAGE)[torch.randperm(PAGE, generator=torch.Generator().manual_seed(3))]
        w["vs"][:, :, 5] = 0.0
    assert verify(msa, w) == 0


def test_optional_outputs_strided_queries_and_streams():
    import sparse_attention_decode_gb300 as msa
    w = make(6, [1200, 77], 2, 4, 16, 4, 16, "hnd", False)
    base = verify(msa, w)
    assert base == 0
    whole = call(msa, w)[0]
    wide = torch.zeros(4, 96, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:80] = w["q"].cuda()
    s = torch.cuda.Stream()
    for kw in (dict(lse=False), dict(mass=False), dict(lse=False, mass=False), dict(q=wide[:, 16:80]), dict(stream=s)):
        assert torch.equal(call(msa, w, **kw)[0], whole), kw


def test_split_lists_give_the_same_bits_each_time():
    import sparse_attention_decode_gb300 as msa
    w = make(7, [4000], 1, 4, 16, 4, 32, "hnd", False)
    first = call(msa, w)
    for _ in range(5):
        again = call(msa, w)
        assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))


def test_a_captured_call_follows_its_inputs():
    import sparse_attention_decode_gb300 as msa
    w = make(8, [1000, 500], 1, 4, 16, 4, 16, "hnd", False)
    kp, vp, table = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), w["table"].cuda()
    q, ids, seq = w["q"].cuda(), w["ids"].cuda(), torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
    run = lambda: msa.msa_attention_sparse(q, kp, vp, table, seq, ids, out, ws, scale=w["scale"])  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    w["q"] = w["q"].flip(0).contiguous()
    w["lens"] = [900, 500]
    w["ids"] = torch.where(w["ids"] == 7, torch.full_like(w["ids"], -1), w["ids"])  # block 7 went with the shorter length
    q.copy_(w["q"])
    ids.copy_(w["ids"])
    seq.copy_(torch.tensor(w["lens"], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.sparse(w["q"], w["kp"], None, w["vp"], None, w["table"], w["lens"], w["ids"], w["scale"], 1)
    ref.check(out, want[0], "out")


def test_bad_device_data_is_absent_and_reported():
    import sparse_attention_decode_gb300 as msa
    w = make(9, [1000, 600, 400, 300], 1, 4, 16, 4, 6, "hnd", False)
    w["table"][0, 2] = 10 ** 6  # a page outside the pool
    w["ids"][1, 2, 0] = 5  # past request 1's last block
    w["ids"][1, 2, 1] = 2 ** 30
    lens = list(w["lens"])
    w["lens"] = [1000, 600, -4, 10 ** 6]
    fault = call(msa, w)[3]
    assert fault == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_BLOCK_ID | msa.MSA_FAULT_SEQ_LEN
    w["lens"] = [1000, 600, 0, 0]
    out, lse, mass, _ = call(msa, dict(w, lens=[1000, 600, -4, 10 ** 6]))
    w["ids"][1, 2, :2] = -1
    want = ref.sparse(w["q"], w["kp"], None, w["vp"], None, w["table"], w["lens"], w["ids"], w["scale"], 1)
    for got, r, name in zip((out, lse, mass), want, ("out", "lse", "mass")):
        ref.check(got, r, name)
    assert lens != w["lens"]


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    w = make(10, [300], 1, 2, 4, 2, 4, "hnd", False)
    kp, vp, table = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), w["table"].cuda()
    q, ids, seq = w["q"].cuda(), w["ids"].cuda(), torch.tensor([300], dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def status(**kw):
        a = dict(q=q, k=kp, v=vp, table=table, seq=seq, ids=ids, out=out, ws=ws, scale=0.1)
        a.update(kw)
        try:
            msa.msa_attention_sparse(a["q"], a["k"], a["v"], a["table"], a["seq"], a["ids"], a["out"], a["ws"],
                                     scale=a["scale"])
        except msa.MsaError as e:
            return e.status
        except AssertionError:
            return "refused"
        return 0

    assert status() == 0
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert status(scale=bad) == msa.MSA_ERR_INVALID_ARG
    assert status(ws=ws[:128]) == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    for bad in (ws.cpu(), torch.zeros(512, dtype=torch.uint8, device="cuda")[::2]):  # on the host; with gaps
        assert status(ws=bad) == "refused"
    assert status(ids=torch.full((1, 2, 33), -1, dtype=torch.int32, device="cuda")) == msa.MSA_ERR_UNSUPPORTED
    assert status(k=kp[:1].expand(kp.shape[0], -1, -1, -1)) == msa.MSA_ERR_INVALID_ARG
    for kw in (dict(q=q.half()), dict(k=kp[..., :64]), dict(k=kp.float()), dict(ids=ids.long()), dict(out=out[:, :4]),
               dict(seq=seq.long()), dict(k=kp[:2]), dict(ids=ids[:, :, ::2])):
        assert status(**kw) == "refused", kw


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_waits_that_run_out_empty_the_rows(e4m3):
    """The producer withholds every page: bounded waits give up, the rows are empty, the next call is exact."""
    import sparse_attention_decode_gb300 as msa
    w = make(19, [1000, 300], 2, 4, 16, 4, 16, "hnd", e4m3)
    whole = call(msa, w)
    msa.msa_indexer_test_withhold_pages(1)
    try:
        out, lse, mass, fault = call(msa, w)
    finally:
        msa.msa_indexer_test_withhold_pages(0)
    assert fault == msa.MSA_FAULT_TIMEOUT
    assert not bool(out.any()) and bool((lse == -float("inf")).all()) and not bool(mass.any())
    again = call(msa, w)
    assert again[3] == 0 and all(torch.equal(a, b) for a, b in zip(again[:3], whole[:3]))
