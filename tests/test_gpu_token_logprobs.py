"""Token log probabilities, entropy and alternatives against 64 bits."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


def plain(logits, tokens, temp, n):
    """(log probabilities, entropy, ids, their log probabilities) and the bounds of the fp32 evaluation.

    A term 2^y is off by (|y| + 3) 2^-23 relatively (y rounded twice, the exponential 2 ulp); a sum of a row's terms, in
    at most 64 steps a thread and 16 joins, by 2^-17.7 more.
    """
    R, V = logits.shape
    lp, ent = torch.full(tokens.shape, 0.0, dtype=torch.float64), torch.zeros(R, dtype=torch.float64)
    ids, top = torch.full((R, n), -1, dtype=torch.int32), torch.full((R, n), -INF, dtype=torch.float64)
    lp_tol, ent_tol = torch.zeros(R, dtype=torch.float64), torch.zeros(R, dtype=torch.float64)
    for r in range(R):
        raw = torch.nan_to_num(logits[r].double(), nan=-INF, neginf=-INF)
        order = torch.sort(-raw, stable=True).indices
        t = 1.0 if temp is None else float(temp[r])
        some = bool(raw.max() > -INF)
        if not some:
            z, p = raw, torch.zeros_like(raw)
        elif t > 0:
            z = (raw - raw.max()) / t
            z = z - z.logsumexp(0)
            p = z.exp()
            y = torch.where(p > 0, (raw - raw.max()).abs() / t / math.log(2), torch.zeros_like(p))
            ent[r] = -(p * z)[p > 0].sum()
            lp_tol[r] = float((p * (y + 3)).sum()) * 2.0 ** -23 + 2.0 ** -17
            ent_tol[r] = float((p * (y * y + 3 * y)).sum()) * 2.0 ** -22 + float((p * y).sum() + 1) * 2.0 ** -17 + 2.0 ** -17
        else:
            p = torch.zeros_like(raw)
            p[order[0]] = 1.0
            z = p.log()
        for j, x in enumerate(tokens[r].tolist()):
            lp[r, j] = 0.0 if x < 0 else float(z[x]) if x < V else -INF
        keep = order[:n][raw[order[:n]] > -INF]
        ids[r, :len(keep)] = keep.to(torch.int32)
        top[r, :len(keep)] = z[keep]
    return lp, ent, ids, top, lp_tol, ent_tol


def call(msa, logits, tokens, temp=None, n=0, entropy=True, stream=None):
    R, m = tokens.shape
    out = torch.full((R, m), 7.0, device="cuda")
    ent = torch.full((R,), 7.0, device="cuda") if entropy else None
    ids = torch.full((R, n), 7, dtype=torch.int32, device="cuda") if n else None
    top = torch.full((R, n), 7.0, device="cuda") if n else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    msa.msa_token_logprobs(logits, tokens.cuda(), out, ws, temperature=None if temp is None else temp.cuda(),
                           out_entropy=ent, out_top_ids=ids, out_top_logprobs=top, stream=stream)
    torch.cuda.synchronize()
    return out, ent, ids, top, msa.msa_indexer_get_error(ws)


def near(got, want, tol):
    got = got.double().cpu()
    tol = tol.view(-1, *[1] * (got.dim() - 1)) + 2.0 ** -22 * torch.where(want.abs() < INF, want.abs(), 0.0 * want.abs().clamp(max=0))
    same = (got == want) | ((want < -3.4e38) & (got == -INF))  # below fp32's range
    return bool((same | ((got - want).abs() <= tol)).all())


def verify(msa, logits, tokens, temp, n, **kw):
    got = call(msa, logits, tokens, temp, n, **kw)
    want = plain(logits.float().cpu(), tokens, temp, n)
    assert near(got[0], want[0], want[4])
    assert near(got[1], want[1], want[5])
    if n:
        assert torch.equal(got[2].cpu(), want[2])
        assert near(got[3], want[3], want[4])
    return got[4]


CASES = [
    # rows, vocabulary, given tokens, alternatives
    (1, 1, 1, 1), (3, 7, 2, 9), (2, 31, 0, 32), (5, 1000, 3, 0), (1, 32000, 1, 5), (4, 50257, 8, 20), (9, 100003, 2, 1),
    (160, 4099, 1, 32), (500, 777, 1, 3), (2, 163840, 256, 32),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_matches_64_bits(case, dtype):
    import sparse_attention_decode_gb300 as msa
    R, V, m, n = case
    g = torch.Generator().manual_seed(31)
    wide = (torch.randn(R, V + 5, generator=g) * 3).to(dtype).cuda()
    tokens = torch.randint(0, V, (R, m), generator=g, dtype=torch.int32)
    temp = 0.3 + torch.rand(R, generator=g)
    temp[1::4] = 0.0
    for off in (0, 1, 3):  # rows that start anywhere
        assert verify(msa, wide[:, off:off + V], tokens, temp if off else None, n) == 0


@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "two values", "one hot", "one thread", "huge"])
@pytest.mark.parametrize("n", [1, 20, 32])
def test_orders_that_are_hard_on_a_running_list(kind, n):
    import sparse_attention_decode_gb300 as msa
    V = 30011
    x = {"rising": torch.arange(V) * 1e-3, "falling": -torch.arange(V) * 1e-3, "equal": torch.full((V,), 2.5),
         "two values": (torch.arange(V) % 7 == 3).float(), "one hot": torch.zeros(V).index_fill_(0, torch.tensor([V - 2]), 90.0),
         "one thread": torch.where(torch.arange(V) // 4 % 256 == 9, torch.arange(V) * 1e-2, torch.zeros(V)),
         "huge": torch.linspace(-3e38, 3e38, V, dtype=torch.float64)}[kind][None].float().cuda().contiguous()
    tokens = torch.tensor([[0, V - 1, V // 2, 36]], dtype=torch.int32)
    for temp in (None, torch.tensor([0.0])):
        assert verify(msa, x, tokens, temp, n) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_masked_vocabularies(dtype):
    """-inf, NaN, the type's lowest value; rows that leave a few tokens or none."""
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(33)
    V = 5003
    x = (torch.randn(8, V, generator=g) * 3).to(dtype)
    low = torch.finfo(dtype).min
    drop = torch.rand(8, V, generator=g)
    x[drop < 0.3] = -INF
    x[drop > 0.7] = low
    x[1] = -INF
    x[2] = -INF
    x[2, 77] = -4.0
    x[3] = low
    x[3, 4000] = 1.0
    x[4] = low
    x[5, ::3] = float("nan")
    x[6] = -INF
    x[6, 100:110] = 0.5
    x[7] = -0.0
    x[7, ::2] = 0.0
    tokens = torch.tensor([[77, 4000, 0, -1, 105, -9]] * 8, dtype=torch.int32)
    for temp in (None, torch.full((8,), 0.7), torch.zeros(8)):
        assert verify(msa, x.cuda(), tokens, temp, 12) == 0


def test_small_and_large_temperatures():
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(34)
    x = (torch.randn(8, 9001, generator=g) * 3).cuda()
    x[:, 17] = x.max() + 1.0
    temp = torch.tensor([1e-3, 1e-30, 1e-40, 50.0, 1e6, -1.0, float("nan"), 1.0])
    tokens = torch.tensor([[17, 3]] * 8, dtype=torch.int32)
    got = call(msa, x, tokens, temp, 2)
    want = plain(x.cpu(), tokens, temp, 2)
    rows = [0, 1, 3, 4, 5, 6, 7]  # 1e-40: a logit over it may pass fp32's range
    assert near(got[0][rows], want[0][rows], want[4][rows]) and near(got[1], want[1], want[5])
    assert torch.equal(got[2].cpu(), want[2]) and got[0][2].tolist() == [0.0, -INF]


def test_optional_outputs_streams_and_graphs():
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(35)
    x = torch.randn(3, 20000, generator=g).cuda()
    tokens = torch.tensor([[1, 2], [3, 4], [5, 6]], dtype=torch.int32)
    base = call(msa, x, tokens, None, 4)
    for kw in (dict(n=0), dict(n=4, entropy=False), dict(n=4, stream=torch.cuda.Stream())):
        got = call(msa, x, tokens, None, **kw)
        assert torch.equal(got[0], base[0]) and (got[2] is None or torch.equal(got[2], base[2]))
    dev, out, ws = tokens.cuda(), torch.zeros(3, 2, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    ids, top = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, device="cuda")
    msa.msa_token_logprobs(x, dev, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_token_logprobs(x, dev, out, ws, out_top_ids=ids, out_top_logprobs=top)
    y = torch.randn(3, 20000, generator=g)
    x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    want = plain(y, tokens, None, 4)
    assert near(out, want[0], want[4]) and torch.equal(ids.cpu(), want[2]) and near(top, want[3], want[4])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(7, 300007), (45, 120011), (100, 33333), (420, 20003)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_rows_of_many_stages(shape, dtype):
    """Rows of each share of a row's blocks, long enough to go round the ring; largest logits anywhere and masked runs."""
    import sparse_attention_decode_gb300 as msa
    R, V = shape
    g = torch.Generator(device="cuda").manual_seed(37)
    x = (torch.randn(R, V, device="cuda", generator=g) * 2).to(dtype)
    x[0, V - 60:] = 9.0  # ties at the end
    x[1 % R, :V // 2] = -INF
    x[2 % R, V // 3:] = torch.finfo(dtype).min
    x[3 % R] = -INF
    x[4 % R] = torch.linspace(-20, 20, V, device="cuda").to(dtype)
    x[5 % R] = torch.linspace(20, -20, V, device="cuda").to(dtype)
    tokens = torch.randint(0, V, (R, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(38))
    temp = torch.full((R,), 0.8)
    temp[6 % R] = 0.0
    assert verify(msa, x, tokens, temp, 20) == 0


@pytest.mark.parametrize("R", [1, 45, 90, 400])
def test_rising_rows_with_elements_behind_the_last_vector(R):
    """Candidates that wait when a row's last elements join them: more than one warp's buffer would hold at once."""
    import sparse_attention_decode_gb300 as msa
    V = 120011
    x = torch.linspace(-20, 20, V, device="cuda").to(torch.bfloat16).expand(R, V).contiguous()  # long runs of equal logits
    first = int((x[0] == x[0, -1]).nonzero()[0])
    want = torch.arange(first, first + 20, dtype=torch.int32).expand(R, 20)
    tokens = torch.zeros(R, 1, dtype=torch.int32)
    for _ in range(30):
        assert torch.equal(call(msa, x, tokens, None, 20)[2].cpu(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_rows_past_4_gib(dtype):
    """Rows whose distance, in elements, 32 bits do not hold."""
    import sparse_attention_decode_gb300 as msa
    V, apart = 5001, 2 ** 32 // 2 + 3
    far = torch.empty(2 * apart + V, dtype=dtype, device="cuda").as_strided((3, V), (apart, 1))
    far.copy_(torch.randn(3, V, generator=torch.Generator().manual_seed(39)) * 3)
    tokens = torch.tensor([[0, 5000], [17, 4], [2500, 1]], dtype=torch.int32)
    assert verify(msa, far, tokens, None, 9) == 0


def test_tokens_outside_the_vocabulary_are_reported():
    import sparse_attention_decode_gb300 as msa
    x = torch.zeros(2, 100, device="cuda")
    got = call(msa, x, torch.tensor([[99, 100], [-1, 2 ** 31 - 1]], dtype=torch.int32))
    assert got[4] == msa.MSA_FAULT_TOKEN
    assert got[0][0, 1] == -INF and got[0][1].tolist() == [0.0, -INF] and abs(float(got[0][0, 0]) + math.log(100)) < 1e-5


def test_the_same_bits_each_time():
    import sparse_attention_decode_gb300 as msa
    x = torch.randn(40, 60001, device="cuda", generator=torch.Generator(device="cuda").manual_seed(36))
    tokens = torch.randint(0, 60001, (40, 3), dtype=torch.int32)
    first = call(msa, x, tokens, None, 20)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first[:4], call(msa, x, tokens, None, 20)[:4]))


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32

    def status(logits=z(2, 9), tokens=z(2, 1, dtype=i32), out=z(2, 1), ws=z(256, dtype=torch.uint8), **kw):
        try:
            msa.msa_token_logprobs(logits, tokens, out, ws, **kw)
        except msa.MsaError as e:
            return e.status
        except AssertionError:
            return "refused"
        return 0

    assert status() == 0
    assert status(ws=z(64, dtype=torch.uint8)) == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    assert status(out_top_ids=z(2, 33, dtype=i32), out_top_logprobs=z(2, 33)) == msa.MSA_ERR_UNSUPPORTED
    assert status(tokens=z(2, 257, dtype=i32), out=z(2, 257)) == msa.MSA_ERR_UNSUPPORTED
    assert status(logits=z(1, 9).expand(2, 9)) == msa.MSA_ERR_INVALID_ARG  # rows on top of one another
    for kw in (dict(logits=z(2, 9, dtype=torch.float16)), dict(logits=z(2, 18)[:, ::2]), dict(tokens=z(2, 1, dtype=torch.int64)),
               dict(out=z(2, 2)), dict(temperature=z(3)), dict(out_entropy=z(1)), dict(out_top_ids=z(2, 3, dtype=i32)),
               dict(out_top_ids=z(2, 3, dtype=i32), out_top_logprobs=z(2, 4)), dict(logits=torch.zeros(2, 9))):
        assert status(**kw) == "refused", kw.keys()
