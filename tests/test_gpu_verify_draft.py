"""Verification of drafted tokens against its definition in 64 bits."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def plain(logits, draft, tokens, u, race, temp, n_draft):
    """The definition, request by request: tokens, accepted counts, log-probabilities and how close a decision was."""
    B, rows, V = logits.shape
    out = torch.full((B, rows), -1, dtype=torch.int32)
    acc, lp = torch.zeros(B, dtype=torch.int32), torch.zeros(B, rows, dtype=torch.float64)
    margin = math.inf
    for b in range(B):
        t, i = float(temp[b]), 0
        while True:
            z = logits[b, i].double()
            z = torch.where(z.isnan(), torch.full_like(z, -math.inf), z)
            if not bool((z > -math.inf).any()):
                acc[b] = i
                break
            if t > 0:
                logp = torch.log_softmax(z / t, 0)
            else:
                logp = torch.full_like(z, -math.inf)
                logp[int((z == z.max()).nonzero()[0])] = 0.0
            p = logp.exp()
            if i < int(n_draft[b]):
                x = int(tokens[b, i])
                uq = float(u[b, i].double() * draft[b, i, x].double()) if 0 <= x < V else 0.0
                px = float(p[x]) if 0 <= x < V else 0.0
                if 0 <= x < V:
                    margin = min(margin, abs(uq - px) / max(uq, px, 1e-300)) if t > 0 else margin
                    if uq < px:
                        out[b, i], lp[b, i] = x, logp[x]
                        i += 1
                        continue
                rest = (p - draft[b, i].double()).clamp_min(0)
                if t > 0 and bool((rest > 0).any()):
                    p = rest
            score = p / race[b].double()
            top = score.topk(2).values if V > 1 else torch.stack([score[0], score[0] * 0])
            margin = min(margin, float((top[0] - top[1]) / top[0]))
            x = int(score.argmax())
            out[b, i], lp[b, i], acc[b] = x, logp[x], i
            break
    return out, acc, lp, margin


def make(seed, B, S, V, dtype, greedy=0, near=0.6):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, S + 1, V, generator=g) * 2.5
    temp = 0.5 + torch.rand(B, generator=g)
    draft = torch.softmax((logits[:, :S] + near * torch.randn(B, S, V, generator=g)) / temp[:, None, None], 2)
    race = torch.empty(B, V).exponential_(generator=g)
    tokens = (draft / torch.empty(B, S, V).exponential_(generator=g)).argmax(2).to(torch.int32) if S else \
        torch.zeros(B, 0, dtype=torch.int32)
    logits = logits.to(dtype)
    temp[:greedy] = 0.0
    if greedy and S:
        tokens[0, 0] = int(logits[0, 0].float().argmax())
    return dict(logits=logits, draft=draft, tokens=tokens, u=torch.rand(B, S, generator=g), race=race, temp=temp,
                n_draft=torch.randint(0, S + 1, (B,), generator=g).to(torch.int32))


def call(msa, w, logits=None, n_draft=True, stream=None):
    d = {k: v.cuda() for k, v in w.items()}
    logits = d["logits"] if logits is None else logits
    B, rows, _ = logits.shape
    out = torch.full((B, rows), 9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    lp = torch.full((B, rows), 9.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    msa.msa_verify_draft(logits, d["draft"], d["tokens"], d["u"], d["race"], out, acc, ws, temperature=d["temp"],
                         n_draft=d["n_draft"] if n_draft else None, out_logprobs=lp, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), acc.cpu(), lp.cpu().double(), msa.msa_indexer_get_error(ws)


def check(msa, w, **kw):
    out, acc, lp, fault = call(msa, w, **kw)
    n = w["n_draft"] if kw.get("n_draft", True) else torch.full_like(w["n_draft"], w["draft"].shape[1])
    r_out, r_acc, r_lp, margin = plain(w["logits"], w["draft"], w["tokens"], w["u"], w["race"], w["temp"], n)
    assert margin > 1e-5  # fp32 decides these inputs as 64 bits do: its probabilities are good to 1e-6
    assert torch.equal(out, r_out) and torch.equal(acc, r_acc)
    # (l - m) / T to 2 ulp, ln Z to 1e-6 and the result's rounding
    assert bool(((lp - r_lp).abs() <= 4e-6 + 2.0 ** -22 * r_lp.abs() + 2.0 ** -22 * 40).all())
    return fault


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,S,V,greedy", [(1, 3, 32000, 0), (5, 0, 1000, 1), (9, 3, 1, 2), (7, 1, 7, 1), (16, 5, 1021, 4),
                                          (3, 63, 257, 1), (4, 3, 100003, 1), (40, 2, 4096, 5)])
def test_matches_64_bits(B, S, V, greedy, dtype):
    import sparse_attention_decode_gb300 as msa
    assert check(msa, make(21, B, S, V, dtype, greedy)) == 0


def test_defaults_strided_logits_and_streams():
    import sparse_attention_decode_gb300 as msa
    w = make(22, 6, 3, 999, torch.bfloat16)
    base = call(msa, w)[:3]
    wide = torch.zeros(6, 7, 1111, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5, 5:1004] = w["logits"].cuda()
    for kw in (dict(logits=wide[:, 1:5, 5:1004]), dict(stream=torch.cuda.Stream())):
        assert all(torch.equal(a, b) for a, b in zip(call(msa, w, **kw)[:3], base))
    check(msa, w, n_draft=False)


def test_masked_logits_and_rows_without_any():
    import sparse_attention_decode_gb300 as msa
    w = make(23, 8, 3, 500, torch.float32, greedy=2)
    keep = torch.rand(8, 4, 500, generator=torch.Generator().manual_seed(1)) < 0.05
    keep[4:, 0] = True
    w["logits"] = torch.where(keep, w["logits"], torch.full_like(w["logits"], -math.inf))
    w["logits"][0, 0] = -math.inf  # a greedy and two drawing requests meet a row with nothing in it
    w["logits"][3] = -math.inf
    w["logits"][5, 0] = float("nan")
    w["logits"][6, 0, 100:] = float("nan")
    assert check(msa, w) == 0
    assert call(msa, w)[0][3].tolist() == [-1] * 4


def test_the_lowest_value_of_the_type_and_large_logits():
    import sparse_attention_decode_gb300 as msa
    w = make(24, 4, 2, 300, torch.float32)
    w["logits"][0, :, 10:] = torch.finfo(torch.float32).min
    w["logits"][1] *= 1000.0
    w["logits"][2] += 30000.0
    assert check(msa, w) == 0


def test_draft_equal_to_the_target_and_ties():
    """q = p refuses nothing but by rounding, and a refusal with an empty residual draws from p; greedy ties go low."""
    import sparse_attention_decode_gb300 as msa
    w = make(25, 4, 1, 64, torch.float32, greedy=1)
    w["n_draft"][:] = 1
    w["draft"][1:] = 1.0  # above p everywhere: the residual is empty
    w["u"][:] = 0.999
    w["logits"][0, 0, :] = 1.0
    w["tokens"][0, 0] = 0
    out, acc, _, _ = call(msa, w)
    assert acc.tolist() == [1, 0, 0, 0]
    check(msa, w)


def test_accepted_and_drawn_tokens_follow_the_target():
    """Over many requests on one target the first emitted token is distributed as the target's."""
    import sparse_attention_decode_gb300 as msa
    B, V = 4096, 8
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(1, 2, V, generator=g).expand(B, 2, V).contiguous()
    draft = torch.softmax(torch.randn(1, 1, V, generator=g), 2).expand(B, 1, V).contiguous()
    tokens = (draft / torch.empty(B, 1, V).exponential_(generator=g)).argmax(2).to(torch.int32)
    w = dict(logits=logits, draft=draft, tokens=tokens, u=torch.rand(B, 1, generator=g),
             race=torch.empty(B, V).exponential_(generator=g), temp=torch.ones(B),
             n_draft=torch.ones(B, dtype=torch.int32))
    first = call(msa, w)[0][:, 0].long()
    p = torch.softmax(logits[0, 0].double(), 0)
    got = torch.bincount(first, minlength=V).double() / B
    assert bool(((got - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all())


def test_bad_device_data_is_refused_and_reported():
    import sparse_attention_decode_gb300 as msa
    w = make(26, 4, 2, 50, torch.float32)
    w["n_draft"][:] = 2
    w["tokens"][0, 0] = 50
    w["tokens"][1, 0] = -1
    assert check(msa, w) == msa.MSA_FAULT_TOKEN
    bad = dict(w, n_draft=torch.tensor([2, 2, 3, -1], dtype=torch.int32))
    out, acc, lp, fault = call(msa, bad)
    assert fault == msa.MSA_FAULT_TOKEN | msa.MSA_FAULT_SEQ_LEN
    w["n_draft"][2:] = 0
    assert torch.equal(out, call(msa, w)[0])


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    w = {k: v.cuda() for k, v in make(27, 2, 1, 20, torch.float32).items()}
    out, acc = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(**kw):
        a = dict(w, ws=ws)
        a.update(kw)
        msa.msa_verify_draft(a["logits"], a["draft"], a["tokens"], a["u"], a["race"], out, acc, a["ws"])

    run()
    with pytest.raises(msa.MsaError) as e:
        run(ws=ws[:64])
    assert e.value.status == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(msa.MsaError) as e:
        run(logits=w["logits"][:1].expand(2, -1, -1))
    assert e.value.status == msa.MSA_ERR_INVALID_ARG
    for kw in (dict(logits=w["logits"].half()), dict(race=w["race"][:1]), dict(tokens=w["tokens"].long()),
               dict(draft=w["draft"].bfloat16()), dict(logits=w["logits"][:, :, ::2])):
        with pytest.raises(AssertionError):
            run(**kw)
