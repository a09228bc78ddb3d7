"""Attention over all of a request's pages against plain attention in 64 bits."""

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def make(seed, lens, q_len, H, G, layout, e4m3, spare=2):
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
    q = torch.randn(B * q_len, H * G, D, generator=g).to(torch.bfloat16)
    return dict(q=q, kp=kp, ks=ks, vp=vp, vs=vs, table=table, lens=list(lens), q_len=q_len, scale=D ** -0.5)


def call(msa, w, lse=True, q=None, stream=None, ws=None):
    dev = {n: ref.to_cuda(w[n]) for n in ("kp", "ks", "vp", "vs")}
    q = w["q"].cuda() if q is None else q
    R, Hq = q.shape[:2]
    H = w["kp"].shape[2]
    out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o_lse = torch.full((R, Hq), 7.0, device="cuda") if lse else None
    if ws is None:
        ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(R, Hq, H), dtype=torch.uint8, device="cuda")
    seq = torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    args = (w["table"].cuda(), seq, out, ws)
    kw = dict(scale=w["scale"], q_len=w["q_len"], out_lse=o_lse, stream=stream)
    torch.cuda.synchronize()
    if w["ks"] is None:
        msa.msa_attention_paged(q, dev["kp"], dev["vp"], *args, **kw)
    else:
        msa.msa_attention_paged_fp8(q, dev["kp"], dev["ks"], dev["vp"], dev["vs"], *args, **kw)
    torch.cuda.synchronize()
    return out, o_lse, msa.msa_indexer_get_error(ws)


def plain(w):
    """out, lse and their bounds, 64 bits on the CPU."""
    q, H, q_len = w["q"], w["kp"].shape[2], w["q_len"]
    R, Hq = q.shape[:2]
    G = Hq // H
    out, tol = torch.zeros(R, Hq, D, dtype=torch.float64), torch.zeros(R, Hq, D, dtype=torch.float64)
    lse, lse_tol = torch.zeros(R, Hq, dtype=torch.float64), torch.zeros(R, Hq, dtype=torch.float64)
    for b in range(len(w["lens"])):
        n = int(w["lens"][b])
        for h in range(H):
            parts = [(int(w["table"][b, j]), min(PAGE, n - j * PAGE)) for j in range(-(-n // PAGE))]
            ok = torch.cat([torch.full((m,), 0 <= p < w["kp"].shape[0]) for p, m in parts] + [torch.zeros(0, dtype=torch.bool)])
            page = lambda p: p if 0 <= p < w["kp"].shape[0] else 0  # noqa: E731
            none = [torch.zeros(0, D, dtype=torch.float64)]
            keys = torch.cat([ref.gather(w["kp"], w["ks"], page(p), h, m) for p, m in parts] + none)
            vals = torch.cat([ref.gather(w["vp"], w["vs"], page(p), h, m) for p, m in parts] + none)
            for i in range(q_len):
                seen = max(0, n - (q_len - 1 - i))
                r, heads, use = b * q_len + i, slice(h * G, (h + 1) * G), ok[:seen]
                o, l, _, t, lt = ref.row(q[r, heads].double(), keys[:seen][use], vals[:seen][use], w["scale"])
                out[r, heads], lse[r, heads], tol[r, heads], lse_tol[r, heads] = o, l, t, lt
    return (out, tol), (lse, lse_tol)


def verify(msa, w, **kw):
    out, lse, fault = call(msa, w, **kw)
    want = plain(w)
    ref.check(out, want[0], "out")
    if lse is not None:
        ref.check(lse, want[1], "lse")
    return fault


CASES = [
    # lens, q_len, kv heads, group, layout
    ([1], 1, 4, 16, "hnd"),
    ([0, 1, 127, 128, 129, 5000], 1, 4, 16, "hnd"),
    ([2, 0, 130, 3000], 4, 4, 6, "nhd"),
    ([700, 4097], 2, 8, 1, "wide"),
    ([20000], 1, 1, 13, "hnd"),
    ([300, 2000], 1, 2, 32, "nhd"),
    ([300, 2000, 640, 3], 4, 2, 16, "hnd"),  # 64 rows a head
    ([260, 1900], 3, 1, 64, "hnd"),          # 192 rows: several tiles
    ([40, 9000], 1, 3, 17, "wide"),
    ([513, 300], 5, 2, 7, "nhd"),            # 35 rows
    ([130 + 7 * i for i in range(90)], 1, 4, 3, "hnd"),
    ([0, 0, 0], 2, 2, 4, "hnd"),
    ([1, 2, 3, 1, 1], 4, 1, 8, "nhd"),       # positions that see nothing
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}q{c[1]}h{c[2]}g{c[3]}{c[4]}")
def test_matches_64_bits(case, e4m3):
    import sparse_attention_decode_gb300 as msa
    lens, q_len, H, G, layout = case
    assert verify(msa, make(41, lens, q_len, H, G, layout, e4m3)) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 4])
def test_peaked_rows_and_large_values(e4m3, q_len):
    """One token takes nearly all weight; scores up to hundreds; V scales over four decades."""
    import sparse_attention_decode_gb300 as msa
    w = make(42, [1500, 900], q_len, 4, 16, "hnd", e4m3)
    w["q"] = (w["q"].float() * 30).to(torch.bfloat16)
    if e4m3:
        w["vs"] = w["vs"] * torch.logspace(-3, 1, PAGE)[torch.randperm(PAGE, generator=torch.Generator().manual_seed(3))]
        w["vs"][:, :, 5] = 0.0
    assert verify(msa, w) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_along_the_request(e4m3, rising):
    """Every page outgrows the maximum so far, or none does."""
    import sparse_attention_decode_gb300 as msa
    w = make(43, [2500, 1300], 2, 2, 4, "hnd", e4m3)
    for b, n in enumerate(w["lens"]):
        nb = -(-n // PAGE)
        for j in range(nb):
            f = 0.2 + 1.5 * (j if rising else nb - 1 - j)
            page = int(w["table"][b, j])
            if e4m3:
                w["ks"][page] *= f
            else:
                w["kp"][page] = (w["kp"][page].float() * f).to(torch.bfloat16)
    ref.spoil((w["kp"], w["vp"]), w["table"], w["lens"])
    assert verify(msa, w) == 0


def test_optional_outputs_strided_queries_and_streams():
    import sparse_attention_decode_gb300 as msa
    w = make(44, [1200, 77], 2, 4, 16, "hnd", False)
    assert verify(msa, w) == 0
    whole = call(msa, w)[0]
    wide = torch.zeros(4, 96, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:80] = w["q"].cuda()
    for kw in (dict(lse=False), dict(q=wide[:, 16:80]), dict(stream=torch.cuda.Stream())):
        assert torch.equal(call(msa, w, **kw)[0], whole), kw


def test_the_same_bits_each_time_and_a_workspace_of_any_history():
    import sparse_attention_decode_gb300 as msa
    w = make(45, [9000, 333, 0, 128], 1, 4, 16, "hnd", False)
    big = make(46, [500] * 40, 4, 4, 16, "nhd", False)
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(160, 64, 4), dtype=torch.uint8, device="cuda")
    first = call(msa, w, ws=ws)
    for _ in range(3):
        call(msa, big, ws=ws)
        again = call(msa, w, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(first[:2], again[:2]))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_captured_call_follows_its_inputs(e4m3):
    import sparse_attention_decode_gb300 as msa
    w = make(47, [6000, 500], 1, 4, 16, "hnd", e4m3)
    kp, vp, ks, vs, table = (ref.to_cuda(w[n]) for n in ("kp", "vp", "ks", "vs", "table"))
    q, seq = w["q"].cuda(), torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(2, 64, 4), dtype=torch.uint8, device="cuda")

    def run():
        if e4m3:
            msa.msa_attention_paged_fp8(q, kp, ks, vp, vs, table, seq, out, ws, scale=w["scale"])
        else:
            msa.msa_attention_paged(q, kp, vp, table, seq, out, ws, scale=w["scale"])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens in ([5000, 500], [0, 1], [128, 499]):
        w["q"] = w["q"].flip(0).contiguous()
        w["lens"] = lens
        q.copy_(w["q"])
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref.check(out, plain(w)[0], "out")


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_graphs_that_share_a_workspace(e4m3):
    """Two calls one after the other in a graph, and two graphs in turn, all on one workspace."""
    import sparse_attention_decode_gb300 as msa
    sets = [make(51, [6000, 500], 1, 4, 16, "hnd", e4m3), make(52, [300] * 30, 4, 2, 16, "nhd", e4m3),
            make(53, [20000], 2, 1, 16, "hnd", e4m3)]
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(120, 64, 1), dtype=torch.uint8, device="cuda")
    runs = []
    for w in sets:
        kp, vp, ks, vs, table = (ref.to_cuda(w[n]) for n in ("kp", "vp", "ks", "vs", "table"))
        q, seq = w["q"].cuda(), torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
        out = torch.zeros_like(q)
        if e4m3:
            args, call_of = (q, kp, ks, vp, vs, table, seq, out, ws), msa.msa_attention_paged_fp8
        else:
            args, call_of = (q, kp, vp, table, seq, out, ws), msa.msa_attention_paged
        runs.append((lambda f=call_of, a=args, w=w: f(*a, scale=w["scale"], q_len=w["q_len"]), out, call(msa, w)[0]))
    graphs = []
    for which in ((0, 1), (2, 0)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in which:
                runs[i][0]()
        graphs.append((graph, which))
    for _ in range(20):
        for graph, which in graphs:
            for _, out, _ in runs:
                out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            for i in range(3):
                assert torch.equal(runs[i][1], runs[i][2]) if i in which else bool((runs[i][1] == 7.0).all())
    assert msa.msa_indexer_get_error(ws) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_bad_device_data_is_absent_and_reported(e4m3):
    import sparse_attention_decode_gb300 as msa
    w = make(48, [1000, 600, 400, 300], 2, 4, 16, "hnd", e4m3)
    w["table"][0, 2] = 10 ** 6  # a page outside the pool
    w["table"][1, 0] = -1
    w["table"][1, 4] = w["kp"].shape[0]
    bad = dict(w, lens=[1000, 600, -4, 10 ** 6])
    out, lse, fault = call(msa, bad)
    assert fault == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_SEQ_LEN
    w["lens"] = [1000, 600, 0, 0]
    want = plain(w)
    ref.check(out, want[0], "out")
    ref.check(lse, want[1], "lse")


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    w = make(49, [300], 1, 2, 4, "hnd", False)
    kp, vp, table = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), w["table"].cuda()
    q, seq = w["q"].cuda(), torch.tensor([300], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(1, 8, 2), dtype=torch.uint8, device="cuda")

    def status(**kw):
        a = dict(q=q, k=kp, v=vp, table=table, seq=seq, out=out, ws=ws, scale=0.1)
        a.update(kw)
        try:
            msa.msa_attention_paged(a["q"], a["k"], a["v"], a["table"], a["seq"], a["out"], a["ws"], scale=a["scale"])
        except msa.MsaError as e:
            return e.status
        except AssertionError:
            return "refused"
        return 0

    assert status() == 0
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert status(scale=bad) == msa.MSA_ERR_INVALID_ARG
    assert status(ws=ws[:128]) == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    assert status(k=kp[:1].expand(kp.shape[0], -1, -1, -1)) == msa.MSA_ERR_INVALID_ARG
    assert status(out=q) == msa.MSA_ERR_INVALID_ARG  # read after it is written
    for kw in (dict(q=q.half()), dict(k=kp[..., :64]), dict(k=kp.float()), dict(out=out[:, :4]), dict(seq=seq.long()),
               dict(k=kp[:2]), dict(ws=ws.cpu()), dict(q=q[:, :3])):
        assert status(**kw) == "refused", kw


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("group", [16, 32, 64])
def test_waits_that_run_out_empty_the_rows(e4m3, group):
    """The producer withholds every page: bounded waits give up, the rows are empty, the next call is exact."""
    import sparse_attention_decode_gb300 as msa
    w = make(50, [9000, 0, 300, 2000], 1, 4, group, "hnd", e4m3)
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(4, 4 * group, 4), dtype=torch.uint8, device="cuda")
    whole = call(msa, w, ws=ws)
    assert whole[2] == 0
    msa.msa_indexer_test_withhold_pages(1)
    try:
        out, lse, fault = call(msa, w, ws=ws)
    finally:
        msa.msa_indexer_test_withhold_pages(0)
    assert fault == msa.MSA_FAULT_TIMEOUT
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    again = call(msa, w, ws=ws)
    assert again[2] == 0 and all(torch.equal(a, b) for a, b in zip(again[:2], whole[:2]))
