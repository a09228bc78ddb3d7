"""Attention of a batch that shares a prefix against plain attention in 64 bits."""

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def make(seed, prefix, lens, q_len, H, G, layout, spare=2):
    g = torch.Generator().manual_seed(seed)
    cols = max(1, max(-(-n // PAGE) for n in lens))
    n_prefix = -(-prefix // PAGE)
    pages = n_prefix + sum(-(-n // PAGE) for n in lens) + spare
    kp, _ = ref.make_pool(g, pages, H, layout, False)
    vp, _ = ref.make_pool(g, pages, H, layout, False)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    shared = torch.cat([perm[:n_prefix], torch.full((1,), -9, dtype=torch.int32)])  # one entry past the prefix
    table = torch.full((len(lens), cols), -7, dtype=torch.int32)
    at = n_prefix
    for b, n in enumerate(lens):
        nb = -(-n // PAGE)
        table[b, :nb] = perm[at:at + nb]
        at += nb
    ref.spoil((kp, vp), table, lens)
    if prefix:
        ref.spoil((kp, vp), shared[None], [prefix])
    q = torch.randn(len(lens) * q_len, H * G, D, generator=g).to(torch.bfloat16)
    return dict(q=q, kp=kp, vp=vp, shared=shared, prefix=prefix, table=table, lens=lens, q_len=q_len, scale=D ** -0.5)


def reference(w):
    R, Hq = w["q"].shape[:2]
    H = w["kp"].shape[2]
    G = Hq // H
    out, tol = torch.zeros(R, H, G, D, dtype=torch.float64), torch.zeros(R, H, G, D, dtype=torch.float64)
    lse, lse_tol = torch.zeros(R, H, G, dtype=torch.float64), torch.zeros(R, H, G, dtype=torch.float64)
    ok = lambda page, n: n > 0 and 0 <= page < w["kp"].shape[0]  # noqa: E731
    for h in range(H):
        pre = [(int(w["shared"][j]), min(PAGE, w["prefix"] - j * PAGE)) for j in range(-(-w["prefix"] // PAGE))]
        cat = lambda pool, parts: torch.cat([torch.zeros(0, D, dtype=torch.float64)] + [  # noqa: E731
            ref.gather(pool, None, page, h, n) for page, n in parts if ok(page, n)])
        pk, pv = cat(w["kp"], pre), cat(w["vp"], pre)
        for r in range(R):
            b = r // w["q_len"]
            n = w["lens"][b] - (w["q_len"] - 1 - r % w["q_len"])
            own = [(int(w["table"][b, j]), min(PAGE, n - j * PAGE)) for j in range(max(0, -(-n // PAGE)))]
            keys, vals = torch.cat([pk, cat(w["kp"], own)]), torch.cat([pv, cat(w["vp"], own)])
            out[r, h], lse[r, h], _, tol[r, h], lse_tol[r, h] = ref.row(
                w["q"][r, h * G:(h + 1) * G].double(), keys, vals, w["scale"])
    return (out.view(R, Hq, D), tol.view(R, Hq, D)), (lse.view(R, Hq), lse_tol.view(R, Hq))


def call(msa, w, lse=True, q=None, stream=None, ws=None):
    q = w["q"].cuda() if q is None else q
    R, Hq = q.shape[:2]
    H = w["kp"].shape[2]
    out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o_lse = torch.full((R, Hq), 7.0, device="cuda") if lse else None
    bound = PAGE * w["shared"].shape[0]
    if ws is None:
        ws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(R, Hq, H, bound), dtype=torch.uint8, device="cuda")
    args = (ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), w["shared"].cuda(),
            torch.tensor([w["prefix"]], dtype=torch.int32, device="cuda"), w["table"].cuda(),
            torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), out, ws)
    torch.cuda.synchronize()
    msa.msa_attention_prefix(q, *args, scale=w["scale"], q_len=w["q_len"], out_lse=o_lse, stream=stream)
    torch.cuda.synchronize()
    return out, o_lse, msa.msa_indexer_get_error(ws)


def verify(msa, w, **kw):
    out, lse, fault = call(msa, w, **kw)
    want = reference(w)
    ref.check(out, want[0], "out")
    if lse is not None:
        ref.check(lse, want[1], "lse")
    return fault


CASES = [
    # prefix, own lengths, q_len, kv heads, group, layout
    (1, [0], 1, 1, 1, "hnd"),
    (0, [0, 1, 300], 1, 2, 16, "hnd"),
    (127, [0, 1, 128, 129], 1, 4, 16, "nhd"),
    (128, [5, 700], 4, 4, 8, "hnd"),
    (129, [0, 1, 2, 3, 400], 4, 2, 3, "wide"),
    (1000, [10] * 17, 1, 4, 16, "hnd"),
    (5000, [3, 0], 1, 2, 16, "nhd"),
    (2050, [40 * i for i in range(20)], 1, 1, 13, "hnd"),
    (1500, [100, 1, 0, 260, 390], 4, 2, 16, "wide"),
    (700, [i for i in range(40)], 2, 2, 7, "hnd"),
    (640, [130, 20, 9], 3, 1, 64, "nhd"),
    (20000, [77], 1, 1, 16, "hnd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"p{c[0]}b{len(c[1])}q{c[2]}h{c[3]}g{c[4]}{c[5]}")
def test_matches_64_bits(case):
    import sparse_attention_decode_gb300 as msa
    prefix, lens, q_len, H, G, layout = case
    assert verify(msa, make(12, prefix, lens, q_len, H, G, layout)) == 0


def test_peaked_rows():
    import sparse_attention_decode_gb300 as msa
    w = make(13, 3000, [200, 0, 500, 64], 1, 2, 16, "hnd")
    w["q"] = (w["q"].float() * 30).to(torch.bfloat16)
    assert verify(msa, w) == 0


def test_a_score_that_grows_along_the_prefix():
    """Every page brings a new maximum, so every running sum is rescaled again and again."""
    import sparse_attention_decode_gb300 as msa
    w = make(14, 2500, [300, 20], 2, 2, 16, "hnd")
    up = torch.nn.functional.normalize(torch.randn(D, generator=torch.Generator().manual_seed(1)), dim=0)
    for j in range(20):
        w["kp"][int(w["shared"][j])] += (up * (4.0 * j)).to(torch.bfloat16)
    ref.spoil((w["kp"], w["vp"]), w["shared"][None], [2500])
    w["q"] = (w["q"].float() + 5 * up).to(torch.bfloat16)
    assert verify(msa, w) == 0


def test_repeated_calls_strided_queries_and_streams():
    import sparse_attention_decode_gb300 as msa
    w = make(15, 4100, [30 * i for i in range(33)], 1, 2, 16, "hnd")
    out, lse, _ = call(msa, w)
    wide = torch.zeros(33, 48, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:40] = w["q"].cuda()
    H, Hq = 2, 32
    ws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(33, Hq, H, 8000), dtype=torch.uint8, device="cuda")
    for kw in (dict(ws=ws), dict(ws=ws), dict(ws=ws, lse=False), dict(q=wide[:, 8:40]), dict(stream=torch.cuda.Stream())):
        again = call(msa, w, **kw)
        assert torch.equal(again[0], out) and (again[1] is None or torch.equal(again[1], lse)), kw


def test_a_captured_call_follows_its_lengths():
    import sparse_attention_decode_gb300 as msa
    w = make(16, 3000, [200, 500, 64], 1, 2, 16, "hnd")
    kp, vp, shared, table = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), w["shared"].cuda(), w["table"].cuda()
    q, seq = w["q"].cuda(), torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    n = torch.tensor([3000], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(3, 32, 2, PAGE * shared.shape[0]), dtype=torch.uint8,
                     device="cuda")
    run = lambda: msa.msa_attention_prefix(q, kp, vp, shared, n, table, seq, out, ws, scale=w["scale"])  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for prefix, lens in ((1000, [130, 0, 1]), (3000, [200, 500, 64]), (0, [1, 2, 3])):
        n.fill_(prefix)
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref.check(out, reference(dict(w, prefix=prefix, lens=lens))[0], "out")


def test_bad_device_data_is_absent_and_reported():
    import sparse_attention_decode_gb300 as msa
    w = make(17, 1500, [1000, 600, 400, 300], 1, 2, 16, "hnd")
    w["shared"][3] = 10 ** 6
    w["table"][0, 2] = -3
    out, lse, fault = call(msa, dict(w, lens=[1000, 600, -4, 10 ** 6]))
    assert fault == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_SEQ_LEN
    want = reference(dict(w, lens=[1000, 600, 0, 0]))
    ref.check(out, want[0], "out")
    ref.check(lse, want[1], "lse")
    out, lse, fault = call(msa, dict(w, prefix=10 ** 6))
    assert fault == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_SEQ_LEN
    ref.check(out, reference(dict(w, prefix=0))[0], "out")


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    w = make(18, 300, [300], 1, 2, 4, "hnd")
    ws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(1, 8, 2, 512), dtype=torch.uint8, device="cuda")
    assert call(msa, w, ws=ws)[2] == 0
    with pytest.raises(msa.MsaError) as e:
        call(msa, w, ws=ws[:-256] if ws.numel() > 256 else ws[:128])
    assert e.value.status == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    for bad in (0.0, float("nan"), -1.0):
        with pytest.raises(msa.MsaError) as e:
            call(msa, dict(w, scale=bad))
        assert e.value.status == msa.MSA_ERR_INVALID_ARG
    for kw in (dict(q=w["q"].half()), dict(kp=w["kp"][:, :64]), dict(shared=w["shared"].long())):
        with pytest.raises(AssertionError):
            call(msa, dict(w, **kw))


@pytest.mark.parametrize("rows", [2, 40], ids=["one_tile", "two_tiles"])
def test_waits_that_run_out_empty_the_rows(rows):
    """The producers withhold every page: bounded waits give up, the rows are empty, the next call is exact."""
    import sparse_attention_decode_gb300 as msa
    w = make(19, 3000, [100 + i for i in range(rows)], 1, 2, 16, "hnd")
    whole = call(msa, w)
    msa.msa_indexer_test_withhold_pages(1)
    try:
        out, lse, fault = call(msa, w)
    finally:
        msa.msa_indexer_test_withhold_pages(0)
    assert fault == msa.MSA_FAULT_TIMEOUT
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    again = call(msa, w)
    assert again[2] == 0 and torch.equal(again[0], whole[0]) and torch.equal(again[1], whole[1])


def test_many_units_of_a_single_page():
    """A CTA's range holds several units of one page each: one of the two chains has nothing to do in any of them."""
    import sparse_attention_decode_gb300 as msa
    for prefix, heads in ((100, 8), (128, 7), (300, 5)):
        w = make(20, prefix, [3, 200, 0], 1, heads, 4, "hnd")
        assert verify(msa, w) == 0
