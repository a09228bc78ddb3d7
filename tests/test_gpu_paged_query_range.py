"""E4M3 attention over all pages: query rows with values far apart, and near the ends of bf16, against 64 bits."""

import pytest
import torch

import attention_ref as ref
import test_gpu_attention_paged as paged

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128


def make(seed, lens, q_len, q, quiet=False):
    """`q`: what becomes of the queries; `quiet`: dim 0 of the keys is 0, so that scores are what the other dims give."""
    w = paged.make(seed, lens, q_len, 2, 16, "hnd", True)
    w["q"] = q(w["q"].double()).to(torch.bfloat16)
    if quiet:
        w["kp"][..., 0] = 0
        ref.spoil((w["kp"],), w["table"], w["lens"])
    return w


def verify(msa, w, held):
    """held: what a query value is off by at most, relative to its row's largest."""
    out, lse, fault = paged.call(msa, w)
    assert fault == 0
    (want, tol), (want_lse, lse_tol) = paged.plain(w)
    G = w["q"].shape[1] // 2
    off = torch.zeros_like(lse_tol)
    for r in range(w["q"].shape[0]):
        b = r // w["q_len"]
        for h in range(2):
            for j in range(-(-w["lens"][b] // PAGE)):
                k = ref.gather(w["kp"], w["ks"], int(w["table"][b, j]), h, min(PAGE, w["lens"][b] - j * PAGE))
                heads = slice(h * G, (h + 1) * G)
                top = w["q"][r, heads].double().abs().amax(-1)
                off[r, heads] = torch.maximum(off[r, heads], held * top * float(k.abs().sum(1).max()) * w["scale"])
    ref.check(lse, (want_lse, lse_tol + off), "lse")
    spread = torch.zeros_like(want)  # a score off by x takes a weight off by x, relatively, and their sum by as much
    for r in range(want.shape[0]):
        b = r // w["q_len"]
        for h in range(2):
            at = [(int(w["table"][b, j]), min(PAGE, w["lens"][b] - j * PAGE)) for j in range(-(-w["lens"][b] // PAGE))]
            if at:
                v = torch.cat([ref.gather(w["vp"], w["vs"], p, h, m) for p, m in at])
                spread[r, h * G:(h + 1) * G] = v.abs().amax(0)
    ref.check(out, (want, tol + 2 * off[..., None] * spread * (1 + off[..., None])), "out")


def outlier(k):
    def f(q):
        q = q.clamp(-4, 4)
        q[..., 0] = 2.0 ** k * 1.5
        return q
    return f


@pytest.mark.parametrize("q_len", [1, 2, 4])
@pytest.mark.parametrize("lens", [[1, 1, 2, 1], [700, 129]], ids=["short", "long"])
def test_values_far_below_the_row_s_largest_are_exact(lens, q_len):
    """Values of 1/8 and more beside 1.5 x 2^10: within 2^-14 of it.  With one token the logsumexp is its score."""
    import sparse_attention_decode_gb300 as msa

    def q(x):
        x = outlier(10)(x)
        return torch.where(x.abs() < 0.125, torch.full_like(x, 0.125), x)
    verify(msa, make(71, lens, q_len, q, quiet=True), 0.0)


@pytest.mark.parametrize("k", [14, 18, 20])
def test_values_further_below_keep_2_to_minus_22_of_the_largest(k):
    import sparse_attention_decode_gb300 as msa
    verify(msa, make(72, [1, 1, 2, 1, 300], 1, outlier(k), quiet=True), 2.0 ** -22)


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("power", [125, 120, 110, -90, -105, -109])
def test_rows_near_the_ends_of_bf16(power, q_len):
    """Queries of 2^power, keys the other way round: ordinary scores."""
    import sparse_attention_decode_gb300 as msa
    w = make(73, [300, 1000, 1], q_len, lambda q: q.clamp(-7.9, 7.9) * 2.0 ** (power - 1 if power == 125 else power))
    w["ks"] = (w["ks"].double() * 2.0 ** -power).float()
    verify(msa, w, 0.0)


def test_output_between_two_query_rows():
    import sparse_attention_decode_gb300 as msa
    for e4m3 in (False, True):
        w = paged.make(74, [700, 300], 1, 2, 16, "hnd", e4m3)
        whole = paged.call(msa, w)
        kp, vp, ks, vs = (ref.to_cuda(w[n]) for n in ("kp", "vp", "ks", "vs"))
        room = torch.full((2, 4 * 32, D), 7.0, dtype=torch.bfloat16, device="cuda")
        room[:, :32] = w["q"].cuda()
        q, out = room[:, :32], room[0, 48:112].view(2, 32, D)
        args = (w["table"].cuda(), torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), out,
                torch.zeros(msa.msa_attention_paged_workspace_bytes(2, 32, 2), dtype=torch.uint8, device="cuda"))
        if e4m3:
            msa.msa_attention_paged_fp8(q, kp, ks, vp, vs, *args, scale=w["scale"])
        else:
            msa.msa_attention_paged(q, kp, vp, *args, scale=w["scale"])
        torch.cuda.synchronize()
        assert torch.equal(out, whole[0]) and torch.equal(room[:, :32].cpu(), w["q"])
        assert bool((room[0, 32:48] == 7.0).all()) and bool((room[0, 112:] == 7.0).all()) and bool((room[1, 32:] == 7.0).all())
