"""New tokens appended, blocks picked, attention over the picked and over all pages, log probabilities: one graph a step."""


import pytest
import torch

import attention_ref as ref
import test_attention_abi as abi
import test_gpu_attention_paged as paged
import test_gpu_cache_append as append
import test_gpu_token_logprobs as logprobs
from test_gpu_attention_threads import race
from test_gpu_fresh_threads import in_a_thread

lib = abi.lib

PAGE, D, K, SINK, WINDOW = 128, 128, 6, 1, 2
START, Q_LEN, STEPS, VOCAB = [700, 1, 131, 2001, 253], 2, 3, 1003


def blocks_hold_up(ids, q, keys, seen):
    """ids of one index head: every pinned block, then none whose maximum is below one left out (up to fp32 sums)."""
    nb = -(-seen // PAGE)
    if nb == 0:
        return all(i < 0 for i in ids)
    x = (keys[:seen].double() @ q.double())
    off = float((keys[:seen].double().abs() @ q.double().abs()).max()) * 2.0 ** -17
    top = [float(x[i * PAGE:(i + 1) * PAGE].max()) for i in range(nb)]
    pins = {i for i in range(nb) if i < SINK or i >= nb - WINDOW}
    got = [i for i in ids if i >= 0]
    if len(set(got)) != len(got) or len(got) != min(K, nb) or not pins <= set(got):
        return False
    left = [top[i] for i in range(nb) if i not in got]
    return not left or min([top[i] for i in got if i not in pins], default=float("inf")) >= max(left) - 2 * off


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_steps_of_a_captured_layer(e4m3):
    import sparse_attention_decode_gb300 as msa
    B, H, Hq, rows = len(START), 4, 16, len(START) * Q_LEN
    final = [n + (STEPS - 1) * Q_LEN for n in START]
    w = append.make(91, final, [Q_LEN] * B, H, Hq, 64, False, True, "hnd", e4m3)
    iw = append.make(92, final, [Q_LEN] * B, 1, 4, 64, False, True, "hnd", e4m3, values=False)
    iw["table"] = w["table"]
    g = torch.Generator().manual_seed(93)
    head = torch.randn(Hq * D, VOCAB, generator=g).cuda() * 0.2
    dev = {n: ref.to_cuda(w[n]) for n in ("kp", "vp", "ks", "vs", "table")}
    ik, iks = ref.to_cuda(iw["kp"]), ref.to_cuda(iw["ks"])
    x, ix = w["x"].cuda(), iw["x"].cuda()
    seq, limit = torch.tensor(START, dtype=torch.int32, device="cuda"), PAGE * w["table"].shape[1]
    empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, iq = empty(rows, Hq, D, dtype=torch.bfloat16), empty(rows, 4, D, dtype=torch.bfloat16)
    ids, scores = empty(B, Q_LEN, 4, K, dtype=torch.int32), empty(B, Q_LEN, 4, K)
    sparse, full, logits = torch.empty_like(q), torch.empty_like(q), empty(rows, VOCAB)
    tokens = torch.randint(0, VOCAB, (rows, 2), generator=g, dtype=torch.int32).cuda()
    temperature = (0.5 + torch.rand(rows, generator=g)).cuda()
    lp, ent, top_ids, top = empty(rows, 2), empty(rows), empty(rows, 5, dtype=torch.int32), empty(rows, 5)
    ws = torch.zeros(msa.msa_indexer_workspace_bytes_mq(B, limit, K, q_len=Q_LEN), dtype=torch.uint8, device="cuda")
    pws = torch.zeros(msa.msa_attention_paged_workspace_bytes(rows, Hq, H), dtype=torch.uint8, device="cuda")
    rope = lambda v: dict(inv_freq=v["inv"].cuda(), q_weight=v["qw"].cuda(), k_weight=v["kw"].cuda(), eps=1e-5,  # noqa: E731
                          q_len=Q_LEN)
    rope_w, rope_i = rope(w), rope(iw)

    def step():
        new = dict(q=x[:, :Hq], out_q=q, **rope_w)
        index = dict(q=ix[:, :4], out_q=iq, **rope_i)
        at = (dev["table"], seq, ws)
        pick = (dev["table"], seq, K, SINK, WINDOW, ids, scores, ws)
        blocks = dict(scale=D ** -0.5, q_len=Q_LEN)
        if e4m3:
            msa.msa_cache_append_fp8(ix[:, 4:5], None, ik, iks, None, None, *at, **index)
            msa.msa_cache_append_fp8(x[:, Hq:Hq + H], x[:, Hq + H:], dev["kp"], dev["ks"], dev["vp"], dev["vs"], *at, **new)
            msa.msa_indexer_decode_mq_fp8(iq.view(B, Q_LEN, 4, D), ik[:, :, 0], iks[:, 0], *pick, max_model_len=limit)
            cache = (dev["kp"], dev["ks"], dev["vp"], dev["vs"], dev["table"], seq)
            msa.msa_attention_sparse_fp8(q, *cache, ids.view(rows, 4, K), sparse, ws, **blocks)
            msa.msa_attention_paged_fp8(q, *cache, full, pws, **blocks)
        else:
            msa.msa_cache_append(ix[:, 4:5], None, ik, None, *at, **index)
            msa.msa_cache_append(x[:, Hq:Hq + H], x[:, Hq + H:], dev["kp"], dev["vp"], *at, **new)
            msa.msa_indexer_decode_mq(iq.view(B, Q_LEN, 4, D), ik[:, :, 0], *pick, max_model_len=limit)
            cache = (dev["kp"], dev["vp"], dev["table"], seq)
            msa.msa_attention_sparse(q, *cache, ids.view(rows, 4, K), sparse, ws, **blocks)
            msa.msa_attention_paged(q, *cache, full, pws, **blocks)
        torch.mm(full.view(rows, Hq * D).float(), head, out=logits)
        msa.msa_token_logprobs(logits, tokens, lp, ws, temperature=temperature, out_entropy=ent, out_top_ids=top_ids,
                               out_top_logprobs=top)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # (the library product's first call)
        torch.mm(full.view(rows, Hq * D).float(), head, out=logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(STEPS):
        for v, gpu in ((w, x), (iw, ix)):
            v["x"] = torch.randn(v["x"].shape, generator=g).to(torch.bfloat16)
            gpu.copy_(v["x"])
            v["lens"] = [n + i * Q_LEN for n in START]
            v["token"] = [n - Q_LEN + j for n in v["lens"] for j in range(Q_LEN)]
        q.fill_(7.0)
        iq.fill_(7.0)
        seq.copy_(torch.tensor(w["lens"], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert msa.msa_indexer_get_error(ws) == 0 and msa.msa_indexer_get_error(pws) == 0
        cpu = {n: None if dev[n] is None else dev[n].cpu() for n in ("kp", "vp", "ks", "vs")}
        append.verify(w, dict(q=q.cpu(), **cpu))
        icpu = dict(kp=ik.cpu(), ks=None if iks is None else iks.cpu(), vp=None, vs=None)
        append.verify(iw, dict(q=iq.cpu(), **icpu))
        w.update(cpu)
        iw.update(icpu)
        for r in range(rows):
            b, seen = r // Q_LEN, w["token"][r] + 1
            keys = torch.cat([ref.gather(iw["kp"], iw["ks"], int(p), 0, PAGE) for p in w["table"][b] if p >= 0])
            for h in range(4):
                assert blocks_hold_up(ids[b, r % Q_LEN, h].tolist(), iq[r, h].cpu(), keys, seen), (i, r, h)
        qc = q.cpu()
        want = ref.sparse(qc, w["kp"], w["ks"], w["vp"], w["vs"], w["table"], w["lens"], ids.view(rows, 4, K).cpu(), D ** -0.5,
                          Q_LEN)
        ref.check(sparse, want[0], "sparse")
        ref.check(full, paged.plain(dict(w, q=qc, q_len=Q_LEN, scale=D ** -0.5))[0], "full")
        want = logprobs.plain(logits.cpu(), tokens.cpu(), temperature.cpu(), 5)
        assert logprobs.near(lp, want[0], want[4]) and logprobs.near(ent, want[1], want[5])
        assert torch.equal(top_ids.cpu(), want[2]) and logprobs.near(top, want[3], want[4])


def make_calls(msa, seed, e4m3=False):
    """One call of each operator on its own tensors: (call(stream), outputs)."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    w = append.make(seed, [300, 20, 129], [2] * 3, 4, 24, 64, False, True, "hnd", e4m3)
    dev = {n: ref.to_cuda(w[n]) for n in ("kp", "vp", "ks", "vs", "table", "x")}
    seq, q = torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), z(6, 24, D, dtype=torch.bfloat16)
    ws, x, inv, kw = z(256, dtype=torch.uint8), dev["x"], w["inv"].cuda(), w["kw"].cuda()
    p = paged.make(seed + 1, [5000, 0, 777], 2, 4, 16, "hnd", e4m3)
    pd = {n: ref.to_cuda(p[n]) for n in ("kp", "vp", "ks", "vs", "table", "q")}
    pseq, out = torch.tensor(p["lens"], dtype=torch.int32, device="cuda"), torch.empty_like(pd["q"])
    pws = z(msa.msa_attention_paged_workspace_bytes(6, 64, 4), dtype=torch.uint8)
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits, tokens = torch.randn(5, 50001, device="cuda", generator=g), z(5, 2, dtype=torch.int32)
    lp, ids, top, lws = z(5, 2), z(5, 7, dtype=torch.int32), z(5, 7), z(256, dtype=torch.uint8)

    def put(stream):
        new = dict(q=x[:, :24], out_q=q, inv_freq=inv, k_weight=kw, q_len=2, stream=stream)
        if e4m3:
            msa.msa_cache_append_fp8(x[:, 24:28], x[:, 28:], dev["kp"], dev["ks"], dev["vp"], dev["vs"], dev["table"], seq, ws,
                                     **new)
        else:
            msa.msa_cache_append(x[:, 24:28], x[:, 28:], dev["kp"], dev["vp"], dev["table"], seq, ws, **new)

    def attend(stream):
        kw = dict(scale=p["scale"], q_len=2, stream=stream)
        if e4m3:
            msa.msa_attention_paged_fp8(pd["q"], pd["kp"], pd["ks"], pd["vp"], pd["vs"], pd["table"], pseq, out, pws, **kw)
        else:
            msa.msa_attention_paged(pd["q"], pd["kp"], pd["vp"], pd["table"], pseq, out, pws, **kw)

    def answer(stream):
        msa.msa_token_logprobs(logits, tokens, lp, lws, out_top_ids=ids, out_top_logprobs=top, stream=stream)
    return [(put, (q, dev["kp"], dev["vp"])), (attend, (out,)), (answer, (lp, ids, top))], (ws, pws, lws)


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_thread_s_first_call(e4m3):
    import sparse_attention_decode_gb300 as msa
    calls, spaces = make_calls(msa, 94, e4m3)
    handle = torch.cuda.current_stream().cuda_stream
    for call, outs in calls:
        call(handle)
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs[:1]:
            o.zero_()
        torch.cuda.synchronize()
        in_a_thread(lambda: call(handle))
        assert all(append.same(a.cpu(), b.cpu()) for a, b in zip(outs, want))
    assert not any(msa.msa_indexer_get_error(s) for s in spaces)


@pytest.mark.gpu
def test_threads_and_streams_at_once():
    """Every operator in both types, each on its own stream with its own workspace."""
    import sparse_attention_decode_gb300 as msa
    sets = [make_calls(msa, 95 + i, e4m3) for i, e4m3 in enumerate((False, True, False))]
    calls = [c for s in sets for c in s[0]]
    for call, _ in calls:
        call(None)
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in calls]
    raised = race(*[c for c, _ in calls], rounds=300)
    torch.cuda.synchronize()
    assert not raised, raised[0]
    for (_, outs), w in zip(calls, want):
        assert all(append.same(a.cpu(), b.cpu()) for a, b in zip(outs, w))
    assert not any(msa.msa_indexer_get_error(x) for s in sets for x in s[1])


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_pages_past_4_gib(e4m3):
    """Byte and element offsets that 32 bits do not hold."""
    import sparse_attention_decode_gb300 as msa
    H, Hq, pages = 4, 24, 100000 if e4m3 else 50000  # 6.6 * 10^9 bytes a pool
    w = append.make(98, [300, 140, 5], [3, 1, 2], H, Hq, 64, False, True, "hnd", e4m3)
    few = w["kp"].shape[0]
    far = torch.arange(few) * ((pages - 1) // (few - 1))
    far[-1] = pages - 1
    table = torch.where(w["table"] >= 0, far[w["table"].clamp(min=0).long()].to(torch.int32), w["table"])
    assert int(table.max()) * H * PAGE * D * (1 if e4m3 else 2) > 2 ** 32
    pool = lambda small: torch.empty(pages, H, PAGE, D, dtype=small.dtype, device="cuda").permute(0, 2, 1, 3)  # noqa: E731
    dev = dict(kp=pool(w["kp"]), vp=pool(w["vp"]))
    for n in dev:
        dev[n][far.cuda()] = w[n].cuda()
    for n in ("ks", "vs"):
        dev[n] = None
        if e4m3:
            dev[n] = torch.zeros(pages, H, PAGE, device="cuda")
            dev[n][far.cuda()] = w[n].cuda()
    x, q = w["x"].cuda(), torch.full((6, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu, seq = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 3, 4, 6], w["lens"]))
    ws = torch.zeros(msa.msa_attention_paged_workspace_bytes(3, Hq, H), dtype=torch.uint8, device="cuda")
    new = dict(q=x[:, :Hq], out_q=q, q_weight=w["qw"].cuda(), k_weight=w["kw"].cuda(), eps=1e-5, inv_freq=w["inv"].cuda(),
               cu_seqlens_q=cu)
    k, v, at = x[:, Hq:Hq + H], x[:, Hq + H:], (table.cuda(), seq)
    last = torch.empty(3, Hq, D, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([2, 3, 5], device="cuda")
    if e4m3:
        msa.msa_cache_append_fp8(k, v, dev["kp"], dev["ks"], dev["vp"], dev["vs"], *at, ws, **new)
        msa.msa_attention_paged_fp8(q[rows], dev["kp"], dev["ks"], dev["vp"], dev["vs"], *at, last, ws, scale=0.1)
    else:
        msa.msa_cache_append(k, v, dev["kp"], dev["vp"], *at, ws, **new)
        msa.msa_attention_paged(q[rows], dev["kp"], dev["vp"], *at, last, ws, scale=0.1)
    torch.cuda.synchronize()
    assert msa.msa_indexer_get_error(ws) == 0
    cpu = {n: None if dev[n] is None else dev[n][far.cuda()].cpu() for n in dev}
    append.verify(w, dict(q=q.cpu(), **cpu))
    w.update(cpu)
    ref.check(last, paged.plain(dict(w, q=q[rows].cpu(), q_len=1, scale=0.1))[0], "out")


def test_an_empty_batch_needs_no_pointers(lib):
    from sparse_attention_decode_gb300 import _attention as A
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)
    new = (None, 512, 4, None, 512, None, 512, None, 512, 4, None, None, 0.0, None, 0, 0, None)
    assert A._fn("msa_cache_append")(*new, None, st, None, st, 10, None, 8, None, None, 0, 0, 1, 1024, None, 0, None) == 0
    new = (None, 512, 4, None, 512, None, 512, None, 512, 4, None, None, 0.0, None, 0, 0, None)
    assert A._fn("msa_cache_append_fp8")(*new, None, st, None, None, st, None, 10, None, 8, None, None, 0, 0, 1, 1024, None, 0,
                                         None) == 0
    assert A._fn("msa_attention_paged")(None, 512, None, st, None, st, 10, None, 8, None, 0, 1, 4, 1, 1024, 1.0, None, None,
                                        None, 0, None) == 0
    assert A._fn("msa_attention_paged_fp8")(None, 512, None, st, None, None, st, None, 10, None, 8, None, 0, 1, 4, 1, 1024,
                                            1.0, None, None, None, 0, None) == 0
    assert A._fn("msa_token_logprobs")(None, 0, 100, None, 1, None, 0, 100, 0, None, None, None, None, None, 0, None) == 0
    # sizes are looked at all the same
    assert A._fn("msa_token_logprobs")(None, 0, 100, None, 1, None, 0, 100, 33, None, None, None, None, None, 0, None) == 2
    assert A._fn("msa_attention_paged")(None, 512, None, st, None, st, 10, None, 8, None, 0, 0, 4, 1, 1024, 1.0, None, None,
                                        None, 0, None) == 1


@pytest.mark.gpu
def test_calls_on_an_empty_batch():
    import sparse_attention_decode_gb300 as msa
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32, bf16 = torch.int32, torch.bfloat16
    kv, ws, codes, scale = z(4, 128, 2, 128, dtype=bf16), z(256, dtype=torch.uint8), z(4, 128, 2, 128, dtype=torch.uint8), z(4, 2, 128)
    q, k, table, seq = z(0, 8, 128, dtype=bf16), z(0, 2, 128, dtype=bf16), z(0, 5, dtype=i32), z(0, dtype=i32)
    msa.msa_cache_append(k, k, kv, kv, table, seq, ws, q=q, out_q=q)
    msa.msa_cache_append_fp8(k, k, codes, scale, codes, scale, table, seq, ws, cu_seqlens_q=z(1, dtype=i32))
    pws = z(msa.msa_attention_paged_workspace_bytes(0, 8, 2), dtype=torch.uint8)
    msa.msa_attention_paged(q, kv, kv, table, seq, q, pws, scale=0.1)
    msa.msa_attention_paged_fp8(q, codes, scale, codes, scale, table, seq, q, pws, scale=0.1, q_len=3)
    msa.msa_token_logprobs(z(0, 9), z(0, 2, dtype=i32), z(0, 2), ws, out_top_ids=z(0, 3, dtype=i32), out_top_logprobs=z(0, 3))
    # requests without a new token among them
    table, seq, cu = z(2, 5, dtype=i32), z(2, dtype=i32), z(3, dtype=i32)
    msa.msa_cache_append(k, k, kv, kv, table, seq, ws, cu_seqlens_q=cu)
    torch.cuda.synchronize()
    assert msa.msa_indexer_get_error(ws) == 0 and not bool(kv.any())


@pytest.mark.gpu
def test_the_example_s_new_stages():
    """Appended tokens, attention over all pages and the answer's log probabilities of the example's step."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import serve_step as ex
    lens, q_len, H, Hq = [700, 130, 2900], ex.DRAFTS + 1, ex.KV_HEADS, ex.KV_HEADS * ex.GROUP
    s = ex.make_step(lens, prompt=300, vocab=500, seed=4)
    before = {n: s[n].cpu() for n in ("k", "v", "index_k", "table", "qkv", "index_qk", "inv_freq", "positions", "logits")}
    r = ex.step(s, budget=100)
    assert r["faults"] == 0
    w = dict(lens=lens, owner=[b for b in range(3) for _ in range(q_len)], token=[n - q_len + i for n in lens for i in range(q_len)],
             positions=before["positions"], inv=before["inv_freq"], inter=False, qw=torch.ones(D), kw=torch.ones(D),
             table=before["table"], ks=None, vs=None, q_len=q_len, scale=D ** -0.5)
    assert before["positions"].tolist() == w["token"]

    def rows(x, Hq, H, kp, vp, got):
        for part, at, want in ((x[:, :Hq], None, got["q"]), (x[:, Hq:Hq + H], kp, got["kp"]), (x[:, Hq + H:], vp, got["vp"])):
            if want is None:
                continue
            values = at is vp and at is not None
            y, tol = append.plain(part, None if values else torch.ones(D), 1e-6, before["positions"], None if values else w["inv"],
                                  False)
            z = want if at is None else torch.stack([want[int(before["table"][b, t // PAGE]), t % PAGE]
                                                     for b, t in zip(w["owner"], w["token"])])
            assert bool(((z.double() - y).abs() <= tol + 2.0 ** -8 * y.abs()).all())
    got = dict(q=s["q"].cpu(), kp=s["k"].cpu(), vp=s["v"].cpu())
    rows(before["qkv"], Hq, H, before["k"], before["v"], got)
    rows(before["index_qk"], 4, 1, before["index_k"].unsqueeze(2), None,
         dict(q=s["index_q"].cpu(), kp=s["index_k"].cpu().unsqueeze(2), vp=None))
    ref.check(r["every"], paged.plain(dict(w, q=got["q"], kp=got["kp"], vp=got["vp"]))[0], "every")
    tokens = r["tokens"].view(-1, 1).cpu()
    want = logprobs.plain(before["logits"].view(len(tokens), -1), tokens, None, 5)
    assert logprobs.near(r["again"], want[0], want[4]) and logprobs.near(r["entropy"], want[1], want[5])
    assert torch.equal(r["top_ids"].cpu(), want[2]) and logprobs.near(r["top"], want[3], want[4])
    assert bool(((r["again"].view_as(r["logp"]) - r["logp"]).abs() <= 2 ** -15 * (1 + r["logp"].abs())).all())
