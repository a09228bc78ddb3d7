"""Plain 64-bit attention on paged caches and the error bounds of a bf16 / f16 tensor-core evaluation of it."""

import torch

PAGE, D = 128, 128


def gather(pool, scale, page, head, n):
    """The first n tokens of a page's head in 64 bits."""
    x = pool[page, :n, head]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale[page, head, :n, None].double()


def row(q, keys, vals, scale):
    """q [g, D], keys, vals [t, D] (64 bits): out, lse, weights and the bounds (out, lse) of the kernels' arithmetic.

    Each score is an fp32 sum of 128 products: off by at most 128 * 2^-24 of sum |q||k|, and 2 ulp of the exponential
    on top; a weight is then off by that much relatively, and by 2^-8 (bf16 keeps 8 significant bits) once more as an operand, like the output.
    """
    g = q.shape[0]
    if keys.shape[0] == 0:
        z = torch.zeros(g, D, dtype=torch.float64)
        return z, torch.full((g,), -float("inf"), dtype=torch.float64), None, z, torch.zeros(g, dtype=torch.float64)
    x = (q @ keys.T) * scale
    lse = torch.logsumexp(x, 1)
    w = (x - lse[:, None]).exp()
    out = w @ vals
    delta = ((q.abs() @ keys.abs().T) * scale).amax(1) * 2.0 ** -17 + 2.0 ** -20
    spread = w @ vals.abs()
    bound = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * delta[:, None]) * spread * 1.02 + 1e-30
    return out, lse, w, bound, delta + 2.0 ** -22 * lse.abs()


def sparse(q, kp, ks, vp, vs, table, lens, ids, scale, q_len):
    """Every row of the attention over selected blocks: out, lse, mass and their bounds, 64 bits on the CPU."""
    R, Hq = q.shape[:2]
    H = kp.shape[2]
    G, sel, k = Hq // H, ids.shape[1], ids.shape[2]
    out = torch.zeros(R, H, G, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((R, H, G), -float("inf"), dtype=torch.float64)
    lse_tol = torch.zeros(R, H, G, dtype=torch.float64)
    mass = torch.zeros(R, H, k, dtype=torch.float64)
    mass_tol = torch.zeros_like(mass)
    for r in range(R):
        n = int(lens[r // q_len]) - (q_len - 1 - r % q_len)
        for h in range(H):
            parts = []
            for j, i in enumerate(ids[r, h // (H // sel)].tolist()):
                m = min(PAGE, n - i * PAGE) if i >= 0 else 0
                page = int(table[r // q_len, i]) if m > 0 else -1
                if m > 0 and 0 <= page < kp.shape[0]:
                    parts.append((j, page, m))
            cat = lambda p, s: torch.cat([gather(p, s, page, h, m) for _, page, m in parts]) if parts else \
                torch.zeros(0, D, dtype=torch.float64)  # noqa: E731
            o, l, w, b, lb = row(q[r, h * G:(h + 1) * G].double(), cat(kp, ks), cat(vp, vs), scale)
            out[r, h], lse[r, h], tol[r, h], lse_tol[r, h] = o, l, b, lb
            at = 0
            for j, _, m in parts:
                x = w[:, at:at + m].sum(1)
                mass[r, h, j] = x.sum()
                mass_tol[r, h, j] = (x * (2 * lb + 2.0 ** -18)).sum() + 1e-30
                at += m
    return (out.view(R, Hq, D), tol.view(R, Hq, D)), (lse.view(R, Hq), lse_tol.view(R, Hq)), (mass, mass_tol)


def check(got, ref, what):
    """Every value within its bound; infinities and signs of emptiness equal."""
    want, tol = ref
    got = got.double().cpu()
    same = got == want
    off = (got - want).abs()
    bad = ~(same | (off <= tol))
    assert not bool(bad.any()), (what, int(bad.sum()), float((off - tol)[bad].max()), bad.nonzero()[0].tolist())


def make_pool(g, pages, heads, layout, e4m3):
    """A cache in [pages, 128, heads, 128] form: head-major or token-major memory, or a view of a wider buffer."""
    x = torch.randn(pages, heads, PAGE, D, generator=g)
    scale = None
    if e4m3:
        scale = torch.rand(pages, heads, PAGE, generator=g) * 0.05 + 0.001
        x = (x * 60).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x = x.to(torch.bfloat16)
    if layout == "hnd":
        return x.permute(0, 2, 1, 3), scale
    if layout == "nhd":
        return x.permute(0, 2, 1, 3).contiguous(), scale
    wide = torch.zeros(pages, PAGE, 2, heads, D, dtype=x.dtype)  # K and V of a token side by side
    wide[:, :, 1] = x.permute(0, 2, 1, 3)
    return wide[:, :, 1], scale


def to_cuda(t):
    """To the GPU in the same memory order."""
    if t is None:
        return None
    base = t._base if t._base is not None else t
    return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())


def spoil(pools, table, lens):
    """Slots past a request's last token hold no data: NaN."""
    for b, n in enumerate(lens):
        if n % PAGE:
            for p in pools:
                p[int(table[b, n // PAGE]), n % PAGE:] = 0x7F if p.dtype == torch.uint8 else float("nan")
