"""E4M3 attention over all pages where whole pages have V scales of 0, tiny or huge ones, against plain attention in 64 bits.

A row's weights x V scales are held relative to the largest of them so far; where all of them have been 0 there is none.
"""

import pytest
import torch

import attention_ref as ref
import test_gpu_attention_paged as paged

pytestmark = pytest.mark.gpu

PAGE, D = 128, 128

# a page's V scales, by its place in the request of n pages, times what they are
SCALES = {
    "first_pages_zero": lambda j, n: 0.0 if j < 2 else 1.0,
    "small_after_zero": lambda j, n: 0.0 if j < 3 else 1e-5,
    "tiny_after_zero": lambda j, n: 0.0 if j < 3 else 1e-24,
    "only_the_last": lambda j, n: 1.0 if j == n - 1 else 0.0,
    "every_second": lambda j, n: float(j % 2),
    "every_second_odd": lambda j, n: float(1 - j % 2),
    "a_few": lambda j, n: float(j % 5 == 3),
    "tiny_then_ordinary": lambda j, n: 1e-30 if j < 3 else 1.0,
    "huge_after_zero": lambda j, n: 0.0 if j < 3 else 1e6,
    "huge_then_zero": lambda j, n: 1e6 if j < 1 else 0.0,
    "tiny_then_huge": lambda j, n: 1e-30 if j < 3 else 1e7,
    "huge_in_the_last": lambda j, n: 1e7 if j == n - 1 else 1e-30,  # some rows see nothing of it
    "huge_then_tiny": lambda j, n: 1e6 if j < 1 else 1e-32,
}
# a page's keys: scores that stay, pass the last page's by a few bits at a time or by many, or fall
KEYS = {
    "level": lambda j, n: 1.0,
    "rising": lambda j, n: 0.2 + 0.4 * j,
    "leaping": lambda j, n: 0.2 + 2.5 * j,
    "falling": lambda j, n: 0.2 + 0.4 * (n - j),
}


def make(seed, lens, q_len, H, G, scales, keys):
    w = paged.make(seed, lens, q_len, H, G, "hnd", True)
    for b, n in enumerate(lens):
        nb = -(-n // PAGE)
        for j in range(nb):
            page = int(w["table"][b, j])
            w["vs"][page] *= SCALES[scales](j, nb)
            w["ks"][page] *= KEYS[keys](j, nb)
    return w


def least_product(w):
    """What holding a product of weight and V scale to 2^-21 of its row's largest leaves of the output's values."""
    q, H, q_len = w["q"].double(), w["kp"].shape[2], w["q_len"]
    G = q.shape[1] // H
    more = torch.zeros(q.shape, dtype=torch.float64)
    for b, n in enumerate(w["lens"]):
        at = [(int(w["table"][b, j]), min(PAGE, n - j * PAGE)) for j in range(-(-n // PAGE))]
        for h in range(H if n else 0):
            keys = torch.cat([ref.gather(w["kp"], w["ks"], p, h, m) for p, m in at])
            codes = torch.cat([ref.gather(w["vp"], torch.ones_like(w["vs"]), p, h, m) for p, m in at]).abs()
            unit = torch.cat([w["vs"][p, h, :m] for p, m in at]).double()
            for i in range(q_len):
                seen = n - (q_len - 1 - i)
                if seen > 0:
                    r, heads = b * q_len + i, slice(h * G, (h + 1) * G)
                    p = torch.softmax((q[r, heads] @ keys[:seen].T) * w["scale"], 1)
                    more[r, heads] = (p * unit[:seen]).amax(1, keepdim=True) * 2.0 ** -21 * codes[:seen].sum(0)
    return more


def verify(msa, w):
    out, lse, fault = paged.call(msa, w)
    assert fault == 0
    (want, tol), want_lse = paged.plain(w)
    ref.check(lse, want_lse, "lse")
    ref.check(out, (want, tol + least_product(w)), "out")


LONG = [750 + 3 * i for i in range(38)]   # with 4 heads a unit a CTA: runs of many pages
PARTS = [2500, 0, 1411]                    # parts of a page or two, which start anywhere


@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("scales", SCALES)
def test_long_runs(scales, keys):
    import sparse_attention_decode_gb300 as msa
    verify(msa, make(61, LONG, 1, 4, 2, scales, keys))


@pytest.mark.parametrize("q_len", [2, 4])
@pytest.mark.parametrize("scales", SCALES)
def test_positions_some_of_which_see_nothing_of_the_last_page(scales, q_len):
    """32 and 64 rows a unit; lengths that end with 1 to 4 tokens of a page."""
    import sparse_attention_decode_gb300 as msa
    verify(msa, make(62, [769 + i % 4 for i in range(76)], q_len, 2, 16, scales, "rising"))


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("scales", SCALES)
def test_short_parts(scales, q_len):
    import sparse_attention_decode_gb300 as msa
    verify(msa, make(63, PARTS, q_len, 2, 16, scales, "leaping"))


@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_scales_of_zero_everywhere(q_len):
    import sparse_attention_decode_gb300 as msa
    w = make(64, [1300] * 40 + [5, 0], q_len, 4, 16, "first_pages_zero", "rising")
    w["vs"].zero_()
    out, lse, fault = paged.call(msa, w)
    assert fault == 0 and not bool(out.any()) and bool(lse.isfinite()[:-q_len].all())


def test_appended_heads_of_zero():
    """Values of zero get a scale of 0 from the append; what follows them keeps its weight."""
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(65)
    lens, H = [700], 1
    w = paged.make(65, lens, 1, H, 16, "hnd", True)
    k, v = torch.randn(2, 700, H, D, generator=g).to(torch.bfloat16)
    v[:600] = 0.0
    v *= 0.01
    kp, vp = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"])
    ks, vs, table = w["ks"].cuda(), w["vs"].cuda(), w["table"].cuda()
    msa.msa_cache_append_fp8(k.cuda(), v.cuda(), kp, ks, vp, vs, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.zeros(256, dtype=torch.uint8, device="cuda"), q_len=700)
    w.update(kp=kp.cpu(), vp=vp.cpu(), ks=ks.cpu(), vs=vs.cpu())
    where = torch.arange(700)
    assert not bool(w["vs"][w["table"][0].long()[where // PAGE], 0, where % PAGE][:600].any())
    verify(msa, w)
