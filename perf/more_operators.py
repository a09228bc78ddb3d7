"""Cases of the operators that a serving step runs around the indexer: appending queries, keys and values to the paged
caches (norm, rotation and quantisation on the way), attention over all of a request's pages, and the log probabilities
of given tokens.

``run`` computes an operator in its plain form (elementary torch operations in fp32, angles in 64 bits), or, where
``own`` is true, calls the library.  ``exact`` computes it from the definition in 64 bits.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128  # head dim
PAGE = 128  # tokens in a page
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one chat request's new token in decode: only latency
        dict(name="append_one_token", op="append", dtype="bf16", layout="hnd", B=1, q_len=1, ragged=False, Hkv=4, G=16,
             rot=64, inter=False, norm=True, shift=0, len_min=8700, len_max=8700, seed=1),
        # a draft step's four positions on the E4M3 cache, after evictions: rotary positions run ahead of the slots
        dict(name="append_draft_e4m3", op="append", dtype="e4m3", layout="hnd", B=32, q_len=4, ragged=False, Hkv=4, G=16,
             rot=128, inter=False, norm=True, shift=1 << 19, len_min=0, len_max=32768, seed=2),
        # the index queries and the single-head index-K cache of a large batch (no values), interleaved pairs
        dict(name="append_index_keys", op="append", dtype="bf16", layout="hnd", B=256, q_len=1, ragged=False, Hkv=1, G=4,
             rot=128, inter=True, norm=False, shift=0, len_min=8000, len_max=8704, seed=3, values=False),
        # the prefill workload's new tokens, ragged requests, token-major cache
        dict(name="append_prefill", op="append", dtype="bf16", layout="nhd", B=4, q_len=2048, ragged=True, Hkv=4, G=16,
             rot=64, inter=False, norm=True, shift=0, len_min=4096, len_max=131072, seed=4),
        # one chat request over its whole context
        dict(name="paged_one_request", op="paged", dtype="bf16", layout="hnd", B=1, q_len=1, Hkv=4, G=16, len_min=8700,
             len_max=8700, seed=5),
        # a few long documents after a draft step: four positions, ragged, one empty request; token-major cache
        dict(name="paged_draft_ragged", op="paged", dtype="bf16", layout="nhd", B=8, q_len=4, Hkv=4, G=16, len_min=0,
             len_max=65536, seed=6),
        # one very long context on the E4M3 cache
        dict(name="paged_long_e4m3", op="paged", dtype="e4m3", layout="hnd", B=1, q_len=1, Hkv=4, G=16, len_min=131072,
             len_max=131072, seed=7),
        # an ordinary decode batch on the E4M3 cache
        dict(name="paged_e4m3_batch", op="paged", dtype="e4m3", layout="hnd", B=32, q_len=1, Hkv=4, G=16, len_min=30000,
             len_max=32768, seed=8),
        # the largest decode batch, at the small decode workload's context
        dict(name="paged_large_batch", op="paged", dtype="bf16", layout="hnd", B=256, q_len=1, Hkv=4, G=16, len_min=8000,
             len_max=8704, seed=9),
        # one request's token with five alternatives, small vocabulary
        dict(name="logprobs_one_row", op="logprobs", dtype="fp32", R=1, V=32000, m=1, n=5, masked=False, greedy=0,
             seed=10),
        # an ordinary batch with bf16 logits, an odd vocabulary masked by a grammar, some greedy requests
        dict(name="logprobs_masked_bf16", op="logprobs", dtype="bf16", R=128, V=100003, m=4, n=20, masked=True, greedy=5,
             seed=11),
        # the log probabilities of a prompt's tokens
        dict(name="logprobs_prompt", op="logprobs", dtype="fp32", R=1024, V=163840, m=1, n=1, masked=False, greedy=0,
             seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "paged", "paged", "logprobs"))
    c = dict(op=op, seed=rng.randrange(1 << 30))
    if op == "append":
        c.update(dtype=rng.choice(("bf16", "e4m3")), layout=rng.choice(("hnd", "nhd")), ragged=rng.random() < 0.4,
                 Hkv=rng.choice((1, 2, 4, 4, 8)), G=rng.randint(1, 16), rot=16 * rng.randint(0, 8),
                 inter=rng.random() < 0.4, norm=rng.random() < 0.7, shift=rng.choice((0, 0, _log_int(rng, 1, 1 << 20))),
                 len_max=_log_int(rng, 64, 131072))
        if c["ragged"]:
            c.update(B=rng.randint(1, 8), q_len=_log_int(rng, 1, min(700, c["len_max"])))
        else:
            c.update(B=_log_int(rng, 1, 256), q_len=rng.choice((1, 1, 2, 4)))
        c["len_min"] = rng.randint(0, c["len_max"])
        c["values"] = c["Hkv"] > 1
    elif op == "paged":
        c.update(dtype=rng.choice(("bf16", "e4m3")), layout=rng.choice(("hnd", "nhd")), B=_log_int(rng, 1, 128),
                 Hkv=rng.choice((1, 2, 4, 4)), G=rng.randint(1, 16), q_len=rng.choice((1, 1, 2, 4)))
        c["len_max"] = _log_int(rng, 1, min(131072, (1 << 20) // c["B"]))
        c["len_min"] = rng.randint(0, c["len_max"])
    else:
        c.update(dtype=rng.choice(("fp32", "bf16")), R=_log_int(rng, 1, 600), V=_log_int(rng, 1000, 163840),
                 m=rng.randint(1, 8), n=rng.randint(0, 32), masked=rng.random() < 0.4)
        c["greedy"] = rng.randint(0, c["R"] // 4)
    return c


def _lens(c):
    """The batch's lengths: a property of the case, so that work() can count them."""
    r = random.Random(c["seed"])
    v = [r.randint(c["len_min"], c["len_max"]) for _ in range(c["B"])]
    if c["B"] >= 4 and c["len_min"] == 0:  # lengths at which masks leave little or nothing
        v[1], v[2] = 0, 1
    return v


def _new(c):
    """New tokens of each request (append): q_len, or for a ragged batch up to q_len and no more than it has."""
    if not c["ragged"]:
        return [c["q_len"]] * c["B"]
    r = random.Random(c["seed"] + 1)
    return [min(n, c["q_len"] if b == 0 else r.randint((c["q_len"] + 1) // 2, c["q_len"])) for b, n in enumerate(_lens(c))]


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(c, g, pages, e4m3):
    """A paged cache [pages, 128 tokens, Hkv, 128] in the case's memory order: (values, scale or None)."""
    shape = (pages, c["Hkv"], PAGE, D) if c["layout"] == "hnd" else (pages, PAGE, c["Hkv"], D)
    if e4m3:
        # codes of N(0, 1) draws scaled by 1/4 .. 1/2 of the largest code a token; a scale for each token and head
        p = torch.empty(shape, device="cuda", dtype=torch.uint8)
        for at in range(0, pages, 1024):
            x = _randn(g, min(1024, pages - at), *shape[1:]).clamp_(-4, 4)
            p[at:at + 1024] = (x * 50).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = (torch.rand(pages, c["Hkv"], PAGE, device="cuda", generator=g) + 0.5) / 50
    else:
        p = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        p.normal_(generator=g)
        scale = None
    return (p.permute(0, 2, 1, 3) if c["layout"] == "hnd" else p), scale


def _workspace(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    return {"append": _prepare_append, "paged": _prepare_paged, "logprobs": _prepare_logprobs}[c["op"]](c, g)


def _prepare_append(c, g):
    B, H, Hq, lens, new = c["B"], c["Hkv"], c["Hkv"] * c["G"], _lens(c), _new(c)
    values = c.get("values", True)
    cols = max(1, -(-c["len_max"] // PAGE))
    # the requests go on from one shared prompt of up to 64 pages; the blocks that get new tokens are their own
    shared = min(64, cols)
    table = torch.randint(0, shared, (B, cols), device="cuda", generator=g, dtype=torch.int32).cpu()
    first = [max(0, n - k) // PAGE for n, k in zip(lens, new)]
    last = [-(-n // PAGE) for n in lens]
    own_pages = sum(max(0, e - s) for s, e in zip(first, last))
    perm = (torch.randperm(own_pages, device="cuda", generator=g) + shared).to(torch.int32).cpu()
    at = 0
    for b in range(B):
        n = max(0, last[b] - first[b])
        table[b, first[b]:last[b]] = perm[at:at + n]
        table[b, last[b]:] = -1
        at += n
    e4m3 = c["dtype"] == "e4m3"
    kp, ks = _pool(c, g, shared + own_pages, e4m3)
    vp, vs = _pool(c, g, shared + own_pages, e4m3) if values else (None, None)
    rows = sum(new)
    # one row of the layer's projection: query heads, key heads, value heads
    x = _randn(g, rows, Hq + 2 * H, D).mul_(1.5).to(torch.bfloat16)
    token = torch.cat([torch.arange(n - k, n) for n, k in zip(lens, new)])
    inv_freq = None
    if c["rot"]:
        inv_freq = (1.0 / 1e6 ** (torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
    s = dict(case=c, q=x[:, :Hq], k=x[:, Hq:Hq + H], v=x[:, Hq + H:] if values else None, kp=kp, ks=ks, vp=vp, vs=vs,
             table=table.cuda(), seq=_ints(lens), inv_freq=inv_freq, eps=1e-6,
             positions=(token + c["shift"]).to(torch.int32).cuda() if c["shift"] else None,
             qw=0.5 + torch.rand(D, device="cuda", generator=g) if c["norm"] else None,
             kw=0.5 + torch.rand(D, device="cuda", generator=g) if c["norm"] else None,
             out_q=torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda"), ws=_workspace(256))
    s["cu"] = _ints([sum(new[:b]) for b in range(B + 1)]) if c["ragged"] else None
    return s


def _prepare_paged(c, g):
    B, q_len, H, lens = c["B"], c["q_len"], c["Hkv"], _lens(c)
    cols = max(1, -(-c["len_max"] // PAGE))
    nb = [-(-n // PAGE) for n in lens]
    pages = sum(nb) + 1
    # pages of the whole batch in a random order, cut into rows; entries past a request's pages are -1
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).cpu()
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = 1
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    e4m3 = c["dtype"] == "e4m3"
    kp, ks = _pool(c, g, pages, e4m3)
    vp, vs = _pool(c, g, pages, e4m3)
    for b, n in enumerate(lens):  # what lies past a request's last token in its last page is not data: NaN
        if n % PAGE:
            for p in (kp, vp):
                p[int(table[b, n // PAGE]), n % PAGE:] = 0x7F if e4m3 else float("nan")
    R, Hq = B * q_len, H * c["G"]
    s = dict(case=c, q=_randn(g, R, Hq, D).to(torch.bfloat16), kp=kp, vp=vp, ks=ks, vs=vs, table=table.cuda(),
             seq=_ints(lens), scale=D ** -0.5, out=torch.empty(R, Hq, D, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(R, Hq, device="cuda"))
    if own:
        import sparse_attention_decode_gb300 as msa
        s["ws"] = _workspace(msa.msa_attention_paged_workspace_bytes(R, Hq, H))
    return s


def _prepare_logprobs(c, g):
    R, V, m, n = c["R"], c["V"], c["m"], c["n"]
    logits = _randn(g, R, V).mul_(2.5)
    if c["masked"]:  # a grammar leaves part of the vocabulary, by either of two customary marks
        gone = torch.rand(R, V, device="cuda", generator=g)
        low = torch.finfo(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32).min
        logits = torch.where(gone < 0.3, torch.full_like(logits, -math.inf), logits)
        logits = torch.where(gone > 0.8, torch.full_like(logits, low), logits)
    tokens = torch.randint(0, V, (R, m), device="cuda", generator=g)
    tokens[:, 0] = logits.argmax(1)  # mostly what was sampled: a likely token
    temp = 0.6 + 0.6 * torch.rand(R, device="cuda", generator=g)
    temp[:c["greedy"]] = 0.0
    if c["dtype"] == "bf16":
        logits = logits.to(torch.bfloat16)
    return dict(case=c, logits=logits, tokens=tokens.to(torch.int32), temp=temp,
                lp=torch.empty(R, m, device="cuda"), entropy=torch.empty(R, device="cuda"),
                ids=torch.empty(R, n, dtype=torch.int32, device="cuda"), top=torch.empty(R, n, device="cuda"),
                ws=_workspace(256))


# ---------------------------------------------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "paged": _own_paged, "logprobs": _own_logprobs}[op](state)
    return {"append": _plain_append, "paged": _plain_paged, "logprobs": _plain_logprobs}[op](state)


def _own_append(s):
    import sparse_attention_decode_gb300 as msa
    more = dict(q=s["q"], out_q=s["out_q"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], inv_freq=s["inv_freq"],
                interleaved=s["case"]["inter"], positions=s["positions"])
    if s["cu"] is not None:
        more["cu_seqlens_q"] = s["cu"]
    else:
        more["q_len"] = s["case"]["q_len"]
    if s["ks"] is None:
        msa.msa_cache_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["seq"], s["ws"], **more)
    else:
        msa.msa_cache_append_fp8(s["k"], s["v"], s["kp"], s["ks"], s["vp"], s["vs"], s["table"], s["seq"], s["ws"], **more)
    return _appended(s)


def _own_paged(s):
    import sparse_attention_decode_gb300 as msa
    more = dict(scale=s["scale"], q_len=s["case"]["q_len"], out_lse=s["lse"])
    if s["ks"] is None:
        msa.msa_attention_paged(s["q"], s["kp"], s["vp"], s["table"], s["seq"], s["out"], s["ws"], **more)
    else:
        msa.msa_attention_paged_fp8(s["q"], s["kp"], s["ks"], s["vp"], s["vs"], s["table"], s["seq"], s["out"], s["ws"],
                                    **more)
    return s["out"], s["lse"]


def _own_logprobs(s):
    import sparse_attention_decode_gb300 as msa
    msa.msa_token_logprobs(s["logits"], s["tokens"], s["lp"], s["ws"], temperature=s["temp"], out_entropy=s["entropy"],
                           out_top_ids=s["ids"], out_top_logprobs=s["top"])
    return s["lp"], s["entropy"], s["ids"], s["top"]


def _codes(pool):
    return pool.view(torch.float8_e4m3fn) if pool is not None and pool.dtype == torch.uint8 else pool


def _appended(s):
    return s["out_q"], _codes(s["kp"]), s["ks"], _codes(s["vp"]), s["vs"]


def _rows(s):
    """Request and token index of every new row."""
    c = s["case"]
    row = torch.arange(s["k"].shape[0], device="cuda")
    if s["cu"] is None:
        b = row // c["q_len"]
        return b, s["seq"].long()[b] - c["q_len"] + row % c["q_len"]
    end = s["cu"].long()[1:]
    b = (row[:, None] >= end[None]).sum(1)
    return b, s["seq"].long()[b] - (end[b] - row)


def _norm(x, weight, eps):
    if weight is None:
        return x
    return x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * weight


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(s):
    c = s["case"]
    b, token = _rows(s)
    live = token >= 0
    q, k = _norm(s["q"].float(), s["qw"], s["eps"]), _norm(s["k"].float(), s["kw"], s["eps"])
    if s["inv_freq"] is not None:
        at = token if s["positions"] is None else s["positions"]
        angle = at[:, None, None].double() * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        q, k = _rotate(q, cos, sin, c["inter"]), _rotate(k, cos, sin, c["inter"])
    s["out_q"].copy_(torch.where(live[:, None, None], q.to(torch.bfloat16), s["out_q"]))
    page = s["table"].long()[b, (token // PAGE).clamp_min(0)][live]
    slot = (token % PAGE)[live]
    for x, pool, scale in ((k, s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        if x is None:
            continue
        x = x[live].float()
        if scale is None:
            pool[page, slot] = x.to(torch.bfloat16)
        else:
            unit = x.abs().amax(-1) / E4M3_MAX
            some = torch.where(unit > 0, unit, torch.ones_like(unit))
            pool[page, slot] = (x / some[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[page, :, slot] = unit
    return _appended(s)


def _values(pool, scale, pages, head):
    """fp32 cache rows of `pages` [...] for `head` [...] (broadcast together): [..., 128 tokens, 128]."""
    x = pool.permute(0, 2, 1, 3)[pages, head]
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scale[pages, head][..., None]


def _softmax(x):
    """exp(x - max), its sum and the max over the last axis; a row with nothing in it sums to 0."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = (x - m).exp()
    return e, e.sum(-1, keepdim=True), m


def _plain_paged(s):
    c = s["case"]
    B, q_len, H, G = c["B"], c["q_len"], c["Hkv"], c["G"]
    cols = s["table"].shape[1]
    pages = s["table"].long().clamp_min(0)[:, None, :]
    head = torch.arange(H, device="cuda")[None, :, None]
    token = torch.arange(cols * PAGE, device="cuda")
    q = s["q"].float().view(B, q_len, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, q_len * G, D)
    keys = _values(s["kp"], s["ks"], pages, head).view(B, H, cols * PAGE, D)
    x = (q @ keys.transpose(2, 3)) * s["scale"]
    del keys
    sees = s["seq"][:, None] - (q_len - 1 - torch.arange(q_len, device="cuda"))
    seen = token < sees[:, None, :, None, None]
    x = torch.where(seen, x.view(B, H, q_len, G, -1), torch.full((), -math.inf, device="cuda"))
    e, l, m = _softmax(x)
    vals = _values(s["vp"], s["vs"], pages, head).view(B, H, cols * PAGE, D)
    vals = torch.where((token < s["seq"][:, None])[:, None, :, None], vals, torch.zeros((), device="cuda"))
    out = (e.view(B, H, q_len * G, -1) @ vals).view(B, H, q_len, G, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log())[..., 0].permute(0, 2, 1, 3).reshape(B * q_len, H * G)
    return out.permute(0, 2, 1, 3, 4).reshape(B * q_len, H * G, D).to(torch.bfloat16), lse


def _plain_logprobs(s):
    c = s["case"]
    n, temp = c["n"], s["temp"][:, None]
    raw = s["logits"].float()
    x = raw / torch.where(temp > 0, temp, torch.ones_like(temp))
    e, l, m = _softmax(x)
    logp = x - m - l.log()
    p = e / l
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    del e, p, x
    top, order = raw.sort(dim=1, descending=True, stable=True)
    hot = torch.arange(raw.shape[1], device="cuda") == order[:, :1]
    sure = torch.where(hot, torch.zeros((), device="cuda"), torch.full((), -math.inf, device="cuda"))
    logp = torch.where(temp > 0, logp, sure)
    entropy = torch.where(temp[:, 0] > 0, entropy, torch.zeros_like(entropy))
    ids = torch.where(top[:, :n] > -math.inf, order[:, :n], torch.full_like(order[:, :n], -1))
    best = torch.where(ids >= 0, logp.gather(1, ids.clamp_min(0)), torch.full((), -math.inf, device="cuda"))
    return logp.gather(1, s["tokens"].long()), entropy, ids.to(torch.int32), best


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "append":
        H, Hq = c["Hkv"], c["Hkv"] * c["G"]
        rows = sum(min(n, k) for n, k in zip(_lens(c), _new(c)))
        caches = 2 if c.get("values", True) else 1
        write = D + 4 if c["dtype"] == "e4m3" else 2 * D
        return dict(bytes=rows * (4 * D * Hq + caches * H * (2 * D + write)), flops=10 * D * rows * (Hq + H))
    if c["op"] == "paged":
        R, H, Hq = c["B"] * c["q_len"], c["Hkv"], c["Hkv"] * c["G"]
        a_token = 2 * D + 8 if c["dtype"] == "e4m3" else 4 * D
        return dict(bytes=sum(_lens(c)) * H * a_token + R * Hq * (4 * D + 4), flops=4 * D * Hq * c["q_len"] * sum(_lens(c)))
    size = 2 if c["dtype"] == "bf16" else 4
    return dict(bytes=c["R"] * (c["V"] * size + 8 * c["m"] + 8 * c["n"] + 8), flops=5 * c["R"] * c["V"])


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "paged": _exact_paged, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    lens, new, r = _lens(c), _new(c), c["rot"]
    token = [n - k + i for n, k in zip(lens, new) for i in range(k)]
    owner = [b for b, k in enumerate(new) for _ in range(k)]
    at = torch.tensor([t + c["shift"] for t in token], dtype=torch.float64, device="cuda")
    live = torch.tensor([i for i, t in enumerate(token) if t >= 0], dtype=torch.long, device="cuda")

    def finish(x, weight):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + s["eps"]) * weight.double()
        if r:
            z = y.clone()
            for i in range(r // 2):
                a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
                turn = (at * s["inv_freq"][i].double())[:, None]
                z[..., a] = y[..., a] * turn.cos() - y[..., b] * turn.sin()
                z[..., b] = y[..., a] * turn.sin() + y[..., b] * turn.cos()
            y = z
        return y

    out_q = s["out_q"].double()
    out_q[live] = finish(s["q"], s["qw"])[live]
    table = s["table"].cpu()
    page = torch.tensor([int(table[owner[i], token[i] // PAGE]) for i in live.tolist()], dtype=torch.long, device="cuda")
    slot = torch.tensor([token[i] % PAGE for i in live.tolist()], dtype=torch.long, device="cuda")
    got = [out_q]
    for x, pool, scale in ((finish(s["k"], s["kw"]), s["kp"], s["ks"]),
                           (None if s["v"] is None else s["v"].double(), s["vp"], s["vs"])):
        if x is None:
            got += [None, None]
        elif scale is None:
            whole = pool.double()
            whole[page, slot] = x[live]
            got += [whole, None]
        else:
            whole, unit = pool.view(torch.float8_e4m3fn).double(), scale.double()
            top = x[live].abs().amax(-1) / E4M3_MAX
            whole[page, slot] = x[live] / top.clamp_min(1e-300)[..., None]
            unit[page, :, slot] = top
            got += [whole, unit]
    return tuple(got)


def _exact_paged(s):
    c = s["case"]
    q_len, H, G = c["q_len"], c["Hkv"], c["G"]
    R = c["B"] * q_len
    out = torch.zeros(R, H, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, H, G), -math.inf, dtype=torch.float64, device="cuda")
    table = s["table"].long()
    for b, n in enumerate(_lens(c)):
        pages = table[b, :-(-n // PAGE)]
        for h in range(H if n else 0):
            kv = []
            for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
                x = pool[pages, :, h].reshape(-1, D)[:n]
                kv.append(x.double() if scale is None else
                          x.view(torch.float8_e4m3fn).double() * scale[pages, h].reshape(-1)[:n, None].double())
            for i in range(q_len):
                seen = n - (q_len - 1 - i)
                if seen > 0:
                    x = (s["q"][b * q_len + i, h * G:(h + 1) * G].double() @ kv[0][:seen].T) * s["scale"]
                    lse[b * q_len + i, h] = x.logsumexp(1)
                    out[b * q_len + i, h] = (x - x.logsumexp(1, keepdim=True)).exp() @ kv[1][:seen]
    return out.view(R, H * G, D), lse.view(R, H * G)


def _exact_logprobs(s):
    c = s["case"]
    R, n = c["R"], c["n"]
    lp = torch.zeros(R, c["m"], dtype=torch.float64, device="cuda")
    entropy = torch.zeros(R, dtype=torch.float64, device="cuda")
    ids = torch.full((R, n), -1, dtype=torch.int32, device="cuda")
    best = torch.full((R, n), -math.inf, dtype=torch.float64, device="cuda")
    temp = s["temp"].double()
    for r in range(R):
        z = s["logits"][r].double()
        order = torch.sort(-z, stable=True).indices
        if temp[r] > 0:
            z = z / temp[r]
            z = z - z.logsumexp(0)
            p = z.exp()
            entropy[r] = -(p * z)[p > 0].sum()
            z = torch.where(z < -torch.finfo(torch.float32).max, torch.full_like(z, -math.inf), z)
        else:
            p = torch.zeros_like(z)
            p[order[0]] = 1.0
            z = p.log()
        lp[r] = z[s["tokens"][r].long()]
        keep = order[:n][s["logits"][r][order[:n]] > -math.inf]
        ids[r, :len(keep)] = keep.to(torch.int32)
        best[r, :len(keep)] = z[keep]
    return lp, entropy, ids, best
