"""Appending to the paged caches, with norm, rotation and quantisation, against the formulas in 64 bits."""

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def plain(x, weight, eps, at, inv_freq, inter):
    """y of [rows, heads, 128] in 64 bits, and what each value's error may be.

    fp32 arithmetic: the angle off by 2^-22.3 rad (its fraction of a turn rounded to fp32), sine and cosine by 2 ulp more,
    the norm by 2^-21, five products and sums by 2^-24 each: below 2^-20 of |a| + |b| of a pair; taken as 2^-19.
    """
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    size = y.abs()
    if inv_freq is not None and len(inv_freq):
        r = 2 * len(inv_freq)
        a, b = (range(0, r, 2), range(1, r, 2)) if inter else (range(r // 2), range(r // 2, r))
        turn = at[:, None, None].double() * inv_freq.double()
        ya, yb = y[..., list(a)], y[..., list(b)]
        z, size = y.clone(), size.clone()
        z[..., list(a)] = ya * turn.cos() - yb * turn.sin()
        z[..., list(b)] = yb * turn.cos() + ya * turn.sin()
        size[..., list(a)] = size[..., list(b)] = ya.abs() + yb.abs()
        y = z
    return y, size * 2.0 ** -19 + 1e-37


def make(seed, lens, new, H, Hq, rot, inter, norm, layout, e4m3, values=True, shift=None, spare=3):
    """`new`: new tokens of each request; the projection's rows stand side by side in one tensor."""
    g = torch.Generator().manual_seed(seed)
    cols = max(1, max(-(-n // PAGE) for n in lens))
    pages = sum(-(-n // PAGE) for n in lens) + spare
    kp, ks = ref.make_pool(g, pages, H, layout, e4m3)
    vp, vs = ref.make_pool(g, pages, H, layout, e4m3) if values else (None, None)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), cols), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        nb = -(-n // PAGE)
        table[b, :nb] = perm[at:at + nb]
        at += nb
    rows = sum(new)
    x = torch.randn(rows, Hq + 2 * H, D, generator=g) * torch.logspace(-2, 1, max(rows, 1))[:rows, None, None]
    owner = [b for b, n in enumerate(new) for _ in range(n)]
    token = [lens[b] - new[b] + i for b in range(len(lens)) for i in range(new[b])]
    inv = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None
    weight = lambda: torch.rand(D, generator=g) + 0.5 if norm else None  # noqa: E731
    return dict(x=x.to(torch.bfloat16), Hq=Hq, H=H, kp=kp, ks=ks, vp=vp, vs=vs, table=table, lens=list(lens), new=list(new),
                owner=owner, token=token, inv=inv, inter=inter, qw=weight(), kw=weight(), values=values,
                positions=None if shift is None else torch.tensor(token, dtype=torch.int32) + shift)


def call(msa, w, ragged=False, q=True, stream=None, **kw):
    """The call's out_q, caches and fault word, back on the CPU."""
    x, Hq, H = w["x"].cuda(), w["Hq"], w["H"]
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    dev = {n: ref.to_cuda(w[n]) for n in ("kp", "vp")}
    dev.update(ks=put(w["ks"]), vs=put(w["vs"]))
    out_q = torch.full((x.shape[0], Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    more = dict(k_weight=put(w["kw"]), inv_freq=put(w["inv"]), interleaved=w["inter"], positions=put(w["positions"]),
                eps=1e-5, stream=stream)
    if q:
        more.update(q=x[:, :Hq], out_q=out_q, q_weight=put(w["qw"]))
    if ragged:
        more["cu_seqlens_q"] = torch.tensor([sum(w["new"][:b]) for b in range(len(w["new"]) + 1)], dtype=torch.int32,
                                            device="cuda")
    else:
        more["q_len"] = w["new"][0]
    more.update(kw)
    k, v = x[:, Hq:Hq + H], x[:, Hq + H:] if w["values"] else None
    seq = torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    if w["ks"] is None:
        msa.msa_cache_append(k, v, dev["kp"], dev["vp"], w["table"].cuda(), seq, ws, **more)
    else:
        msa.msa_cache_append_fp8(k, v, dev["kp"], dev["ks"], dev["vp"], dev["vs"], w["table"].cuda(), seq, ws, **more)
    torch.cuda.synchronize()
    fault = msa.msa_indexer_get_error(ws)
    back = lambda t: None if t is None else t.cpu()  # noqa: E731
    return dict(q=out_q.cpu(), fault=fault, **{n: back(dev[n]) for n in ("kp", "ks", "vp", "vs")})


def same(a, b):
    """Equal bit for bit (NaN included)."""
    return a is b is None or torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def verify(w, got, q=True, absent=()):
    """Every output and every other slot of the caches; `absent`: rows that have to be left as they were."""
    token = torch.tensor(w["token"])
    at = token if w["positions"] is None else w["positions"]
    Hq, H, x = w["Hq"], w["H"], w["x"]
    live = [r for r, t in enumerate(w["token"]) if t >= 0 and r not in absent]
    if q:
        y, tol = plain(x[:, :Hq], w["qw"], 1e-5, at, w["inv"], w["inter"])
        bound = tol + 2.0 ** -8 * y.abs()
        off = (got["q"].double() - y).abs()[live] - bound[live]
        assert not live or float(off.max()) <= 0, float(off.max())
        rest = [r for r in range(len(token)) if r not in live]
        assert bool((got["q"][rest] == 7.0).all())
    else:
        assert bool((got["q"] == 7.0).all())
    key = plain(x[:, Hq:Hq + H], w["kw"], 1e-5, at, w["inv"], w["inter"])
    value = plain(x[:, Hq + H:], None, 0.0, at, None, False)
    for (y, tol), n, s in ((key, "kp", "ks"),) + (((value, "vp", "vs"),) if w["values"] else ()):
        want, scale = w[n].clone(), None if w[s] is None else w[s].clone()
        for r in live:
            page, slot = int(w["table"][w["owner"][r], w["token"][r] // PAGE]), w["token"][r] % PAGE
            if scale is None:
                z = got[n][page, slot].double()
                assert bool(((z - y[r]).abs() <= tol[r] + 2.0 ** -8 * y[r].abs()).all()), (n, r)
            else:
                unit = got[s][page, :, slot].double()
                top = y[r].abs().amax(-1)
                assert bool(((unit - top / 448).abs() <= (tol[r].amax(-1) + 2.0 ** -22 * top) / 448).all()), (s, r)
                z = got[n][page, slot].view(torch.float8_e4m3fn).double() * unit[:, None]
                # half a step: 2^-4 of a normal value, half of 2^-9 of the scale below; the quotient by 2^-18 more
                bound = tol[r] + 2.0 ** -4 * y[r].abs() + (2.0 ** -10 * unit + 2.0 ** -18 * top)[:, None]
                assert bool(((z - y[r]).abs() <= bound).all()), (n, r)
                scale[page, :, slot] = got[s][page, :, slot]
            want[page, slot] = got[n][page, slot]
        assert same(got[n], want), n  # nothing else changed
        assert scale is None or same(got[s], scale), s


CASES = [
    # lens, new, kv heads, query heads, rotary dim, interleaved, norm, layout, ragged
    ([1], [1], 4, 64, 64, False, True, "hnd", False),
    ([5, 128, 129, 1000], [1] * 4, 4, 24, 128, False, True, "nhd", False),
    ([3, 0, 2, 130, 256], [4] * 5, 2, 26, 128, True, False, "hnd", False),
    ([700, 258], [2] * 2, 8, 8, 16, False, True, "wide", False),
    ([300, 40, 0, 129, 513], [260, 1, 0, 129, 77], 4, 20, 48, False, True, "nhd", True),
    ([200], [200], 1, 4, 0, False, True, "hnd", True),
    ([131, 7], [130, 7], 3, 17, 96, True, True, "wide", True),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}h{c[2]}q{c[3]}r{c[4]}{'i' * c[5]}{c[7]}")
def test_matches_64_bits(case, e4m3):
    import sparse_attention_decode_gb300 as msa
    lens, new, H, Hq, rot, inter, norm, layout, ragged = case
    w = make(21, lens, new, H, Hq, rot, inter, norm, layout, e4m3)
    got = call(msa, w, ragged=ragged)
    assert got["fault"] == 0
    verify(w, got)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_keys_alone_and_without_queries(e4m3):
    """A single-head cache of keys, as the indexer reads it."""
    import sparse_attention_decode_gb300 as msa
    w = make(22, [300, 140], [3, 3], 1, 4, 128, False, True, "hnd", e4m3, values=False)
    got = call(msa, w)
    assert got["fault"] == 0
    verify(w, got)
    bare = call(msa, w, q=False)
    verify(w, bare, q=False)
    assert same(bare["kp"], got["kp"])


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
def test_far_positions_and_large_frequencies(inter):
    """Angles of far, negative and unordered positions keep their fraction of a turn."""
    import sparse_attention_decode_gb300 as msa
    w = make(23, [40], [8], 2, 4, 32, inter, False, "hnd", False)
    w["inv"] = torch.tensor([1.0, 0.3, -0.7, 6.5, 40.0, 3e-4, 1e-9, 0.0] + [2.0 ** -i for i in range(8)])
    w["positions"] = torch.tensor([0, 1 << 20, 3, 1 << 24, 12345678, -5, -(1 << 22), 99], dtype=torch.int32)
    got = call(msa, w)
    assert got["fault"] == 0
    verify(w, got)


def test_zero_tiny_and_large_heads():
    import sparse_attention_decode_gb300 as msa
    for e4m3 in (False, True):
        w = make(24, [200], [6], 2, 4, 64, False, False, "hnd", e4m3)
        w["x"][1] = 0.0
        w["x"][2] = (w["x"][2].float() * 1e-37).to(torch.bfloat16)
        w["x"][3] = (w["x"][3].float() * 1e30).to(torch.bfloat16)
        w["x"][4, :, 1:] = 0.0
        got = call(msa, w)
        if e4m3:  # below 2^-117: zero by definition
            for n, s in (("kp", "ks"), ("vp", "vs")):
                page, slot = int(w["table"][0, w["token"][2] // PAGE]), w["token"][2] % PAGE
                assert not bool(got[s][page, :, slot].any()) and not bool(got[n][page, slot].any())
            w["x"][2] = 0.0
            got["q"][2] = 0.0
        verify(w, got)


def test_in_place_queries_streams_and_graphs():
    import sparse_attention_decode_gb300 as msa
    w = make(25, [300, 20], [2, 2], 2, 10, 64, False, True, "hnd", False)
    base = call(msa, w)
    s = torch.cuda.Stream()
    assert same(call(msa, w, stream=s)["q"], base["q"])
    x = w["x"].cuda()
    kp, vp, ws = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), torch.zeros(256, dtype=torch.uint8, device="cuda")
    seq, table = torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), w["table"].cuda()
    more = dict(q_weight=w["qw"].cuda(), k_weight=w["kw"].cuda(), eps=1e-5, inv_freq=w["inv"].cuda(), q_len=2)
    run = lambda: msa.msa_cache_append(x[:, 10:12], x[:, 12:], kp, vp, table, seq, ws, q=x[:, :10], out_q=x[:, :10],  # noqa: E731
                                       **more)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    torch.cuda.synchronize()
    assert torch.equal(x.cpu(), w["x"])  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    assert same(x[:, :10].cpu(), base["q"]) and same(kp.cpu(), base["kp"]) and same(vp.cpu(), base["vp"])
    # the next step's lengths: the same graph writes the next slots
    w["lens"] = [302, 22]
    w["token"] = [t + 2 for t in w["token"]]
    x.copy_(w["x"])
    seq.copy_(torch.tensor(w["lens"], dtype=torch.int32))
    w["kp"], w["vp"] = base["kp"], base["vp"]
    graph.replay()
    torch.cuda.synchronize()
    verify(w, dict(q=x[:, :10].cpu(), kp=kp.cpu(), vp=vp.cpu(), ks=None, vs=None))


def test_rows_behind_the_last_request_are_left():
    import sparse_attention_decode_gb300 as msa
    w = make(26, [100, 50], [5, 3], 2, 4, 64, False, True, "hnd", True)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")  # of 8 rows, 6 belong to requests
    w["owner"], w["token"] = [0] * 3 + [1] * 3 + [0, 0], [97, 98, 99, 47, 48, 49, -1, -1]
    got = call(msa, w, ragged=True, cu_seqlens_q=cu)
    assert got["fault"] == 0
    verify(w, got)


def test_bad_device_data_is_absent_and_reported():
    import sparse_attention_decode_gb300 as msa
    w = make(27, [300, 40, 129, 60], [1] * 4, 2, 4, 64, False, True, "hnd", False)
    w["table"][0, 2] = 10 ** 6  # a page outside the pool: its key and value go nowhere, the query is prepared
    table = w["table"].clone()
    got = call(msa, w)
    assert got["fault"] == msa.MSA_FAULT_PAGE_ID
    y, tol = plain(w["x"][:, :4], w["qw"], 1e-5, torch.tensor(w["token"]), w["inv"], False)
    assert bool(((got["q"].double() - y).abs() <= tol + 2.0 ** -8 * y.abs()).all())
    w["lens"] = [300, -1, 10 ** 6, 60]
    assert torch.equal(table, w["table"])
    got = call(msa, w)
    assert got["fault"] == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_SEQ_LEN
    assert bool((got["q"][1:3] == 7.0).all()) and not bool((got["q"][3] == 7.0).any())
    w = make(28, [10, 20, 30, 40], [2] * 4, 2, 4, 64, False, True, "hnd", False)
    for bad in ([0, 2, 1, 6, 8], [0, 2, 4, 6, 90], [-3, 2, 4, 6, 8], [5, 6, 7, 8, 8], [0, 8, 8, 8, 8]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        got = call(msa, w, ragged=True, cu_seqlens_q=cu)
        broken = bad != [0, 8, 8, 8, 8]
        assert got["fault"] == (msa.MSA_FAULT_SEQ_LEN if broken else 0), bad


MANY = [
    # more rows than the GPU has SMs, lines of 24 heads and more (and of fewer): lens, new, kv heads, query heads, ...
    ([50 + 9 * i for i in range(9)], [40] * 9, 3, 26, 64, True, "wide"),
    ([400, 3, 0, 170], [200, 3, 0, 170], 24, 0, 48, False, "nhd"),
    ([160], [160], 8, 207, 128, False, "hnd"),   # the longest line that fits twice an SM
    ([160], [160], 8, 208, 128, True, "hnd"),    # and one more
    ([130, 180], [100, 77], 1, 21, 0, True, "hnd"),
    ([200], [200], 5, 13, 32, False, "hnd"),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{sum(c[1])}h{c[2]}q{c[3]}r{c[4]}{'i' * c[5]}{c[6]}")
def test_many_rows(case, e4m3):
    import sparse_attention_decode_gb300 as msa
    lens, new, H, Hq, rot, inter, layout = case
    w = make(29, lens, new, H, Hq, rot, inter, True, layout, e4m3, shift=5)
    got = call(msa, w, ragged=True, q=Hq > 0)
    assert got["fault"] == 0
    verify(w, got, q=Hq > 0)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_many_rows_of_keys_alone(e4m3):
    import sparse_attention_decode_gb300 as msa
    w = make(30, [60] * 4, [41] * 4, 25, 0, 32, False, True, "hnd", e4m3, values=False)
    got = call(msa, w, q=False)
    assert got["fault"] == 0
    verify(w, got, q=False)


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
def test_many_rows_padded_in_place_and_captured(inter):
    """Requests shorter than q_len, rows behind the last request, queries prepared where they are."""
    import sparse_attention_decode_gb300 as msa
    w = make(31, [90, 7, 0, 40], [45] * 4, 2, 24, 64, inter, True, "hnd", False)
    got = call(msa, w)
    assert got["fault"] == 0
    verify(w, got)
    x = w["x"].cuda()
    kp, vp, ws = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), torch.zeros(256, dtype=torch.uint8, device="cuda")
    seq, table = torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), w["table"].cuda()
    more = dict(q_weight=w["qw"].cuda(), k_weight=w["kw"].cuda(), eps=1e-5, inv_freq=w["inv"].cuda(), q_len=45,
                interleaved=inter)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_cache_append(x[:, 24:26], x[:, 26:], kp, vp, table, seq, ws, q=x[:, :24], out_q=x[:, :24], **more)
    graph.replay()
    torch.cuda.synchronize()
    live = [r for r, t in enumerate(w["token"]) if t >= 0]
    assert same(x[live, :24].cpu(), got["q"][live]) and same(kp.cpu(), got["kp"]) and same(vp.cpu(), got["vp"])
    left = [r for r, t in enumerate(w["token"]) if t < 0]
    assert same(x[left].cpu(), w["x"][left]) and same(x[:, 24:].cpu(), w["x"][:, 24:])
    w = make(32, [100, 120], [95, 90], 2, 24, 64, inter, True, "hnd", False)
    cu = torch.tensor([0, 90, 180], dtype=torch.int32, device="cuda")  # of 185 rows
    w["owner"] = [0] * 90 + [1] * 95
    w["token"] = list(range(10, 100)) + list(range(30, 120)) + [-1] * 5
    got = call(msa, w, ragged=True, cu_seqlens_q=cu)
    assert got["fault"] == 0
    verify(w, got)


def test_many_rows_with_bad_device_data():
    import sparse_attention_decode_gb300 as msa
    w = make(33, [300, 40, 129, 60], [40] * 4, 2, 24, 64, False, True, "hnd", False)
    w["table"][0, 2] = 10 ** 6
    w["lens"] = [300, -1, 10 ** 6, 60]
    got = call(msa, w)
    assert got["fault"] == msa.MSA_FAULT_PAGE_ID | msa.MSA_FAULT_SEQ_LEN
    at = torch.tensor(w["token"])
    y, tol = plain(w["x"][:, :24], w["qw"], 1e-5, at, w["inv"], False)
    live = list(range(40)) + list(range(120, 160))
    assert bool(((got["q"].double() - y).abs() <= tol + 2.0 ** -8 * y.abs())[live].all())
    assert bool((got["q"][40:120] == 7.0).all())
    for bad in ([0, 90, 30, 160, 160], [0, 40, 80, 120, 9000], [-3, 40, 80, 120, 160], [0, 160, 160, 160, 160]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        w["lens"] = [300, 40, 129, 60]
        assert call(msa, w, ragged=True, cu_seqlens_q=cu)["fault"] & msa.MSA_FAULT_SEQ_LEN == \
            (msa.MSA_FAULT_SEQ_LEN if bad != [0, 160, 160, 160, 160] else 0), bad


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8

    def status(fp8=False, **kw):
        code = u8 if fp8 else torch.bfloat16
        a = dict(k=z(2, 2, 128), v=z(2, 2, 128), kc=z(4, 128, 2, 128, dtype=code), vc=z(4, 128, 2, 128, dtype=code),
                 ks=z(4, 2, 128, dtype=f32), vs=z(4, 2, 128, dtype=f32), table=z(2, 3, dtype=i32), seq=z(2, dtype=i32),
                 ws=z(256, dtype=u8))
        more = {n: kw.pop(n) for n in list(kw) if n not in a}
        a.update(kw)
        try:
            if fp8:
                msa.msa_cache_append_fp8(a["k"], a["v"], a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["seq"], a["ws"],
                                         **more)
            else:
                msa.msa_cache_append(a["k"], a["v"], a["kc"], a["vc"], a["table"], a["seq"], a["ws"], **more)
        except msa.MsaError as e:
            return e.status
        except AssertionError:
            return "refused"
        return 0

    assert status() == 0 and status(fp8=True) == 0
    for eps in (-1.0, float("nan"), float("inf")):
        assert status(eps=eps) == msa.MSA_ERR_INVALID_ARG
    assert status(inv_freq=z(12, dtype=f32)) == msa.MSA_ERR_UNSUPPORTED  # 24 dims
    assert status(inv_freq=z(72, dtype=f32)) == msa.MSA_ERR_UNSUPPORTED  # 144 dims
    assert status(ws=z(128, dtype=u8)) == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    wide = z(2, 4, 2, 128)[:, 1]
    assert status(k=wide, v=wide) == 0
    off = z(4 * 128 * 2 + 4)[4:].view(2, 4, 128)[:, :2]
    assert status(k=off) == msa.MSA_ERR_INVALID_ARG  # not on 16 bytes
    twice = z(4, 4, 128)  # the same first row, other strides
    assert status(q=twice[:2], out_q=twice[::2]) == msa.MSA_ERR_INVALID_ARG
    assert status(q=twice[::2], out_q=twice[::2]) == 0
    for kw in (dict(k=z(2, 2, 128, dtype=f32)), dict(k=z(2, 3, 128)), dict(v=None), dict(vc=None), dict(q=z(2, 4, 128)),
               dict(q=z(2, 4, 128), out_q=z(2, 5, 128)), dict(q_len=2), dict(positions=z(3, dtype=i32)),
               dict(inv_freq=z(32, dtype=torch.float64)), dict(k_weight=z(64, dtype=f32)), dict(seq=z(3, dtype=i32)),
               dict(cu_seqlens_q=z(2, dtype=i32)), dict(ws=torch.zeros(256, dtype=u8)), dict(fp8=True, ks=None),
               dict(fp8=True, vs=None), dict(fp8=True, ks=z(4, 128, 2, dtype=f32)), dict(k=z(2, 2, 256)[..., ::2])):
        assert status(**kw) == "refused", kw.keys()
