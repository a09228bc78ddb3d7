"""Cases of the serving operators that follow the indexer: attention over the selected blocks, attention of a batch
that shares a prefix, eviction by accumulated attention weight, and the verification of drafted tokens.

``run`` computes an operator in its plain form (elementary torch operations in fp32), or, where ``own`` is true,
calls the library.  ``exact`` computes it from the definition in 64 bits.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128  # head dim
PAGE = 128  # tokens in a page


# ---------------------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one chat request in decode: nothing to share, only latency
        dict(name="sparse_one_request", op="sparse", dtype="bf16", layout="hnd", B=1, q_len=1, Hkv=4, G=16, k=16,
             len_min=8700, len_max=8700, seed=1),
        # a draft step of few ragged requests, one empty and one of a single token; token-major cache, odd group
        dict(name="sparse_draft_ragged", op="sparse", dtype="bf16", layout="nhd", B=7, q_len=4, Hkv=4, G=6, k=16,
             len_min=0, len_max=33000, seed=2),
        # an ordinary decode batch on the E4M3 cache
        dict(name="sparse_e4m3_batch", op="sparse", dtype="e4m3", layout="hnd", B=32, q_len=1, Hkv=4, G=16, k=16,
             len_min=30000, len_max=32768, seed=3),
        # the largest decode batch, at the small decode workload's context
        dict(name="sparse_large_batch", op="sparse", dtype="bf16", layout="hnd", B=256, q_len=1, Hkv=4, G=16, k=16,
             len_min=8000, len_max=8704, seed=4),
        # two users on one short system prompt
        dict(name="prefix_two_requests", op="prefix", layout="hnd", B=2, q_len=1, Hkv=4, G=16, prefix=4133,
             len_min=1, len_max=200, seed=5),
        # a draft step of a few requests on a long document, ragged own tokens (one has none yet), token-major cache
        dict(name="prefix_draft_ragged", op="prefix", layout="nhd", B=8, q_len=4, Hkv=4, G=8, prefix=16384,
             len_min=0, len_max=2000, seed=6),
        # a full batch over a long shared document with conversations of their own
        dict(name="prefix_full_batch", op="prefix", layout="hnd", B=64, q_len=1, Hkv=4, G=16, prefix=32768,
             len_min=500, len_max=4096, seed=7),
        # a few requests of the small decode workload's length after a draft step
        dict(name="evict_few", op="evict", B=4, q_len=4, Hkv=4, k=16, cols=68, budget=32, len_min=1000, len_max=8700,
             sink=1, window=2, seed=8),
        # a large batch of contexts up to 2^20 tokens brought down to 2^18
        dict(name="evict_long_contexts", op="evict", B=256, q_len=1, Hkv=4, k=16, cols=8192, budget=2048,
             len_min=200000, len_max=1 << 20, sink=1, window=2, seed=9),
        # one request's three drafted tokens, small vocabulary
        dict(name="verify_one_request", op="verify", dtype="fp32", B=1, S=3, V=32000, greedy=0, seed=10),
        # an ordinary batch with bf16 logits, an odd vocabulary, ragged drafts and some greedy requests
        dict(name="verify_ragged_bf16", op="verify", dtype="bf16", B=32, S=3, V=100003, greedy=5, seed=11),
        # the largest batch
        dict(name="verify_large_batch", op="verify", dtype="fp32", B=256, S=3, V=163840, greedy=0, seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sparse", "sparse", "prefix", "evict", "verify"))
    c = dict(op=op, seed=rng.randrange(1 << 30))
    if op == "sparse":
        c.update(dtype=rng.choice(("bf16", "bf16", "e4m3")), layout=rng.choice(("hnd", "nhd")), B=_log_int(rng, 1, 160),
                 Hkv=rng.choice((1, 2, 4, 4, 8)), G=rng.randint(1, 16), k=rng.randint(1, 32),
                 len_max=_log_int(rng, 1, 16384))
        c["q_len"] = rng.choice((1, 1, 2, 4)) if c["B"] <= 40 else 1
        c["Hkv"] = min(c["Hkv"], 4) if c["B"] > 40 else c["Hkv"]
        c["k"] = min(c["k"], 16) if c["B"] > 40 else c["k"]
        c["len_min"] = rng.randint(0, c["len_max"])
    elif op == "prefix":
        c.update(layout=rng.choice(("hnd", "nhd")), B=_log_int(rng, 1, 64), Hkv=rng.choice((1, 2, 4, 4)),
                 G=rng.randint(1, 16), prefix=_log_int(rng, 1, 32768), len_max=_log_int(rng, 1, 4096))
        c["q_len"] = rng.choice((1, 1, 2, 4)) if c["B"] <= 16 else 1
        c["len_min"] = rng.randint(0, c["len_max"])
    elif op == "evict":
        c.update(B=_log_int(rng, 1, 256), q_len=rng.choice((1, 2, 4)), Hkv=rng.choice((1, 2, 4)), k=rng.randint(1, 32),
                 cols=_log_int(rng, 4, 8192), sink=rng.randint(0, 1), window=rng.randint(1, 2))
        c["budget"] = rng.randint(3, c["cols"])
        c["len_max"] = c["cols"] * PAGE - rng.randint(0, PAGE)
        c["len_min"] = rng.randint(0, c["len_max"])
    else:
        c.update(dtype=rng.choice(("fp32", "bf16")), B=_log_int(rng, 1, 128), S=rng.randint(0, 5),
                 V=_log_int(rng, 1000, 163840))
        c["greedy"] = rng.randint(0, c["B"] // 4)
    return c


def _lens(c):
    """The batch's lengths: a property of the case, so that work() can count them."""
    r = random.Random(c["seed"])
    v = [r.randint(c["len_min"], c["len_max"]) for _ in range(c["B"])]
    if c["B"] >= 4 and c["len_min"] == 0:  # lengths at which masks leave little or nothing
        v[1], v[2] = 0, 1
    return v


def _n_draft(c):
    r = random.Random(c["seed"])
    return [c["S"] if b % 3 else r.randint(0, c["S"]) for b in range(c["B"])]


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


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


def _spoil_tails(c, lens, table, pools):
    """What lies past a request's last token in its last page is not data: NaN."""
    at = [(int(table[b, n // PAGE]), n % PAGE) for b, n in enumerate(lens) if n % PAGE]
    for page, t in at:
        for p in pools:
            p[page, t:] = 0x7F if p.dtype == torch.uint8 else float("nan")


def _table(g, lens, cols, spare):
    """Pages of the whole batch in a random order, cut into rows; entries past a request's pages are -1."""
    nb = [-(-n // PAGE) for n in lens]
    total = sum(nb)
    perm = torch.randperm(total + spare, device="cuda", generator=g).to(torch.int32).cpu()
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = spare
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[:spare], total + spare


def prepare(case, seed):
    c, g = case, _gen(seed)
    return {"sparse": _prepare_sparse, "prefix": _prepare_prefix, "evict": _prepare_evict,
            "verify": _prepare_verify}[c["op"]](c, g)


def _workspace(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def _prepare_sparse(c, g):
    B, q_len, H, k = c["B"], c["q_len"], c["Hkv"], c["k"]
    lens = _lens(c)
    cols = max(1, -(-c["len_max"] // PAGE))
    table, _, pages = _table(g, lens, cols, 1)
    e4m3 = c["dtype"] == "e4m3"
    kp, ks = _pool(c, g, pages, e4m3)
    vp, vs = _pool(c, g, pages, e4m3)
    _spoil_tails(c, lens, table, (kp, vp))
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # each head's own selection: sink and last two blocks, then others at random; the draft positions of a request
    # agree on all blocks but one, as neighbouring positions do
    nb = (seq + PAGE - 1) // PAGE
    j = torch.arange(cols, device="cuda")
    score = torch.rand(B, H, cols, device="cuda", generator=g)
    n3 = nb[:, None, None]
    score = torch.where((j < 1) | (j >= n3 - 2), score + 1.0, score)
    score = torch.where(j < n3, score, torch.full_like(score, -1.0))
    want = k + q_len - 1
    if want > cols:
        score = torch.cat([score, torch.full((B, H, want - cols), -1.0, device="cuda")], 2)
    top, order = score.sort(dim=2, descending=True)
    order = torch.where(top >= 0, order, torch.full_like(order, -1))
    ids = torch.stack([torch.cat([order[:, :, :k - 1], order[:, :, k - 1 + i:k + i]], 2) for i in range(q_len)], 1)
    pos_nb = (seq[:, None] - (q_len - 1 - torch.arange(q_len, device="cuda")) + PAGE - 1) // PAGE
    ids = torch.where(ids < pos_nb[:, :, None, None], ids, torch.full_like(ids, -1))
    R, Hq = B * q_len, H * c["G"]
    s = dict(case=c, q=_randn(g, R, Hq, D).to(torch.bfloat16), kp=kp, vp=vp, ks=ks, vs=vs,
             table=table.cuda(), seq=seq, ids=ids.reshape(R, H, k).to(torch.int32).contiguous(), scale=D ** -0.5,
             out=torch.empty(R, Hq, D, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(R, Hq, device="cuda"), mass=torch.empty(R, H, k, device="cuda"), ws=_workspace(256))
    return s


def _prepare_prefix(c, g):
    B, q_len, H = c["B"], c["q_len"], c["Hkv"]
    lens = _lens(c)
    cols = max(1, -(-c["len_max"] // PAGE))
    n_prefix = -(-c["prefix"] // PAGE)
    table, prefix, pages = _table(g, lens, cols, n_prefix)
    kp, _ = _pool(c, g, pages, False)
    vp, _ = _pool(c, g, pages, False)
    _spoil_tails(c, lens, table, (kp, vp))
    _spoil_tails(c, [c["prefix"]], prefix[None], (kp, vp))
    R, Hq = B * q_len, H * c["G"]
    s = dict(case=c, q=_randn(g, R, Hq, D).to(torch.bfloat16), kp=kp, vp=vp, prefix=prefix.cuda(),
             prefix_len=torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda"), table=table.cuda(),
             seq=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5,
             out=torch.empty(R, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(R, Hq, device="cuda"))
    if own:
        import sparse_attention_decode_gb300 as msa
        s["ws"] = _workspace(msa.msa_attention_prefix_workspace_bytes(R, Hq, H, n_prefix * PAGE))
    return s


def _prepare_evict(c, g):
    B, q_len, H, k, cols = c["B"], c["q_len"], c["Hkv"], c["k"], c["cols"]
    lens = _lens(c)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nb = (seq + PAGE - 1) // PAGE
    j = torch.arange(cols, device="cuda")
    live = j < nb[:, None]
    # rows of one random order of the pages; entries past a request's pages are -1
    perm = torch.randperm(B * cols, device="cuda", generator=g).to(torch.int32).view(B, cols)
    table = torch.where(live, perm, torch.full_like(perm, -1))
    # accumulated weight has a heavy tail, and blocks that were never selected have none
    w = torch.rand(B, H, cols, device="cuda", generator=g).clamp_min_(1e-4).pow_(-1.2)
    w = torch.where(torch.rand(B, H, cols, device="cuda", generator=g) < 0.4, torch.zeros_like(w), w)
    w = torch.where(live[:, None, :], w, torch.zeros_like(w)).contiguous()
    score = torch.where(live[:, None, None, :], torch.rand(B, q_len, H, cols, device="cuda", generator=g),
                        torch.full((1,), -1.0, device="cuda"))
    top, ids = score.topk(min(k, cols), dim=3)
    ids = torch.where(top >= 0, ids, torch.full_like(ids, -1))
    if k > cols:
        ids = torch.cat([ids, torch.full((B, q_len, H, k - cols), -1, device="cuda")], 3)
    mass = torch.rand(B * q_len, H, k, device="cuda", generator=g)
    mass = torch.where(ids.reshape(B * q_len, H, k) >= 0, mass, torch.zeros_like(mass))
    rows = torch.randint(0, q_len + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    empty = dict(dtype=torch.int32, device="cuda")
    return dict(case=c, table=table, seq=seq, weights=w, mass=mass.contiguous(), n_rows=rows,
                ids=ids.reshape(B * q_len, H, k).to(torch.int32).contiguous(),
                new_table=torch.empty(B, cols, **empty), new_seq=torch.empty(B, **empty),
                new_weights=torch.empty(B, H, cols, device="cuda"), freed=torch.empty(B, cols, **empty),
                n_freed=torch.empty(B, **empty), ws=_workspace(256))


def _prepare_verify(c, g):
    B, S, V = c["B"], c["S"], c["V"]
    # a peaked target; the draft model's logits are near it, its tokens are drawn from its own probabilities
    logits = _randn(g, B, S + 1, V).mul_(2.5)
    draft = torch.empty(B, S, V, device="cuda")
    tokens = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    temp = (0.6 + 0.6 * torch.rand(B, device="cuda", generator=g))
    for i in range(S):
        x = (logits[:, i] + 0.6 * _randn(g, B, V)) / temp[:, None]
        p = (x - x.amax(1, keepdim=True)).exp_()
        draft[:, i] = p / p.sum(1, keepdim=True)
        noise = torch.empty(B, V, device="cuda").exponential_(generator=g)
        tokens[:, i] = (draft[:, i] / noise).argmax(1).to(torch.int32)
        del x, p, noise
    logits = logits.to(torch.bfloat16) if c["dtype"] == "bf16" else logits
    for b in range(c["greedy"]):
        temp[b] = 0.0
        if S and b % 2 == 0:  # a draft that a greedy request accepts
            tokens[b, 0] = logits[b, 0].float().argmax().to(torch.int32)
    return dict(case=c, logits=logits, draft=draft, tokens=tokens, temp=temp,
                u=torch.rand(B, S, device="cuda", generator=g),
                race=torch.empty(B, V, device="cuda").exponential_(generator=g),
                n_draft=torch.tensor(_n_draft(c), dtype=torch.int32, device="cuda"),
                out=torch.empty(B, S + 1, dtype=torch.int32, device="cuda"),
                n=torch.empty(B, dtype=torch.int32, device="cuda"),
                logp=torch.empty(B, S + 1, device="cuda"), ws=_workspace(256))


# ---------------------------------------------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sparse": _own_sparse, "prefix": _own_prefix, "evict": _own_evict, "verify": _own_verify}[op](state)
    return {"sparse": _plain_sparse, "prefix": _plain_prefix, "evict": _plain_evict,
            "verify": _plain_verify}[op](state)


def _own_sparse(s):
    import sparse_attention_decode_gb300 as msa
    q_len = s["case"]["q_len"]
    if s["ks"] is None:
        msa.msa_attention_sparse(s["q"], s["kp"], s["vp"], s["table"], s["seq"], s["ids"], s["out"], s["ws"],
                                 scale=s["scale"], q_len=q_len, out_lse=s["lse"], out_mass=s["mass"])
    else:
        msa.msa_attention_sparse_fp8(s["q"], s["kp"], s["ks"], s["vp"], s["vs"], s["table"], s["seq"], s["ids"],
                                     s["out"], s["ws"], scale=s["scale"], q_len=q_len, out_lse=s["lse"],
                                     out_mass=s["mass"])
    return s["out"], s["lse"], s["mass"]


def _own_prefix(s):
    import sparse_attention_decode_gb300 as msa
    msa.msa_attention_prefix(s["q"], s["kp"], s["vp"], s["prefix"], s["prefix_len"], s["table"], s["seq"], s["out"],
                             s["ws"], scale=s["scale"], q_len=s["case"]["q_len"], out_lse=s["lse"])
    return s["out"], s["lse"]


def _own_evict(s):
    import sparse_attention_decode_gb300 as msa
    c = s["case"]
    msa.msa_cache_accumulate(s["weights"], s["ids"], s["mass"], s["ws"], q_len=c["q_len"], n_rows=s["n_rows"])
    msa.msa_cache_evict(s["table"], s["seq"], s["weights"], c["budget"], c["sink"], c["window"], s["new_table"],
                        s["new_seq"], s["new_weights"], s["freed"], s["n_freed"], s["ws"])
    return s["new_table"], s["new_seq"], s["new_weights"], s["freed"], s["n_freed"]


def _own_verify(s):
    import sparse_attention_decode_gb300 as msa
    msa.msa_verify_draft(s["logits"], s["draft"], s["tokens"], s["u"], s["race"], s["out"], s["n"], s["ws"],
                         temperature=s["temp"], n_draft=s["n_draft"], out_logprobs=s["logp"])
    return s["out"], s["n"], s["logp"]


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


def _plain_sparse(s):
    c = s["case"]
    B, q_len, H, G, k = c["B"], c["q_len"], c["Hkv"], c["G"], c["k"]
    R = B * q_len
    row = torch.arange(R, device="cuda")
    length = s["seq"][row // q_len] - (q_len - 1 - row % q_len)
    ids = s["ids"].long()
    at = ids.clamp_min(0)
    pages = s["table"].long()[(row // q_len)[:, None, None], at].clamp_min(0)
    token = at[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    valid = (ids[..., None] >= 0) & (token < length[:, None, None, None])  # [R, H, k, 128]
    head = torch.arange(H, device="cuda")[None, :, None]
    keys = _values(s["kp"], s["ks"], pages, head).view(R, H, k * PAGE, D)
    x = (s["q"].float().view(R, H, G, D) @ keys.transpose(2, 3)) * s["scale"]
    del keys
    valid = valid.view(R, H, 1, k * PAGE)
    e, l, m = _softmax(torch.where(valid, x, torch.full_like(x, -math.inf)))
    vals = _values(s["vp"], s["vs"], pages, head).view(R, H, k * PAGE, D)
    vals = torch.where(valid.transpose(2, 3), vals, torch.zeros_like(vals))
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    out = (p @ vals).view(R, H * G, D).to(torch.bfloat16)
    return out, (m + l.log()).view(R, H * G), p.view(R, H, G, k, PAGE).sum((2, 4))


def _plain_prefix(s):
    c = s["case"]
    B, q_len, H, G, Lp = c["B"], c["q_len"], c["Hkv"], c["G"], c["prefix"]
    R = B * q_len
    q = s["q"].float().view(R, H, G, D)
    by_head = q.permute(1, 0, 2, 3).reshape(H, R * G, D)
    head = torch.arange(H, device="cuda")
    shared = s["prefix"].long()
    pre = lambda pool: _values(pool, None, shared[None, :], head[:, None]).reshape(H, -1, D)[:, :Lp]  # noqa: E731
    x1 = (by_head @ pre(s["kp"]).transpose(1, 2)) * s["scale"]  # [H, R * G, Lp]
    x1 = x1.view(H, R, G, Lp).permute(1, 0, 2, 3)
    row = torch.arange(R, device="cuda")
    length = s["seq"][row // q_len] - (q_len - 1 - row % q_len)
    cols = s["table"].shape[1]
    pages = s["table"].long().clamp_min(0)
    own_rows = lambda pool: _values(pool, None, pages[:, None, :], head[None, :, None]).view(  # noqa: E731
        B, H, cols * PAGE, D)
    x2 = (q.view(B, q_len, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, q_len * G, D)
          @ own_rows(s["kp"]).transpose(2, 3)) * s["scale"]
    x2 = x2.view(B, H, q_len, G, cols * PAGE).permute(0, 2, 1, 3, 4).reshape(R, H, G, cols * PAGE)
    token = torch.arange(cols * PAGE, device="cuda")
    x2 = torch.where(token < length[:, None, None, None], x2, torch.full_like(x2, -math.inf))
    e, l, m = _softmax(torch.cat([x1, x2], 3))
    o1 = (e[..., :Lp].permute(1, 0, 2, 3).reshape(H, R * G, Lp) @ pre(s["vp"])).view(H, R, G, D).permute(1, 0, 2, 3)
    vals = own_rows(s["vp"])
    vals = torch.where(token[None, None, :, None] < s["seq"][:, None, None, None], vals, torch.zeros_like(vals))
    e2 = e[..., Lp:].reshape(B, q_len, H, G, cols * PAGE).permute(0, 2, 1, 3, 4).reshape(B, H, q_len * G, -1)
    o2 = (e2 @ vals).view(B, H, q_len, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, G, D)
    out = (o1 + o2) / torch.where(l > 0, l, torch.ones_like(l))
    return out.reshape(R, H * G, D).to(torch.bfloat16), (m + l.log()).reshape(R, H * G)


def _plain_evict(s):
    c = s["case"]
    B, q_len, H, cols, budget = c["B"], c["q_len"], c["Hkv"], c["cols"], c["budget"]
    w = s["weights"]
    ids, mass = s["ids"].long().view(B, q_len, H, -1), s["mass"].view(B, q_len, H, -1)
    for i in range(q_len):  # the accepted positions, in order; a row's ids are distinct
        use = (ids[:, i] >= 0) & (i < s["n_rows"][:, None, None])
        w.scatter_add_(2, ids[:, i].clamp_min(0), torch.where(use, mass[:, i], torch.zeros_like(mass[:, i])))
    total = w[:, 0]
    for h in range(1, H):  # the definition's order of the sum
        total = total + w[:, h]
    seq = s["seq"]
    nb = ((seq + PAGE - 1) // PAGE)[:, None]
    j = torch.arange(cols, device="cuda")[None]
    rank_by = torch.where((j < c["sink"]) | (j >= nb - c["window"]), torch.full_like(total, math.inf), total)
    rank_by = torch.where(j < nb, rank_by, torch.full_like(total, -math.inf))
    order = rank_by.sort(dim=1, descending=True, stable=True).indices
    kept = torch.zeros(B, cols, dtype=torch.bool, device="cuda")
    kept.scatter_(1, order[:, :budget], True)
    kept &= j < nb
    n_kept = kept.sum(1, keepdim=True)
    first = (~kept).to(torch.int8).sort(dim=1, stable=True).indices  # kept ones first, in order
    live = j < n_kept
    none = torch.full_like(s["table"], -1)
    table = torch.where(live, s["table"].gather(1, first), none)
    weights = torch.where(live[:, None], w.gather(2, first[:, None].expand(B, H, cols)), torch.zeros_like(w))
    gone = (~kept) & (j < nb)
    freed_first = (~gone).to(torch.int8).sort(dim=1, stable=True).indices
    n_freed = gone.sum(1, keepdim=True)
    freed = torch.where(j < n_freed, s["table"].gather(1, freed_first), none)
    n_freed = n_freed[:, 0].to(torch.int32)
    return table, seq - PAGE * n_freed, weights, freed, n_freed


def _first_max(x):
    """The lowest index of the last axis's largest value."""
    i = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), i, torch.full_like(i, x.shape[-1])).amin(-1)


def _plain_verify(s):
    c = s["case"]
    B, S, V = c["B"], c["S"], c["V"]
    temp = s["temp"]
    x = s["logits"].float() / torch.where(temp > 0, temp, torch.ones_like(temp))[:, None, None]
    e, l, m = _softmax(x)
    p = e / l
    logp = x - m - l.log()
    del e, x
    if c["greedy"]:
        top = _first_max(s["logits"][:c["greedy"]].float())
        hot = torch.arange(V, device="cuda") == top[..., None]
        p[:c["greedy"]] = hot.float()
        logp[:c["greedy"]] = torch.where(hot, torch.zeros_like(logp[:1]), torch.full_like(logp[:1], -math.inf))
    tokens = s["tokens"].long()
    p_x = p[:, :S].gather(2, tokens[..., None])[..., 0]
    q_x = s["draft"].gather(2, tokens[..., None])[..., 0]
    i = torch.arange(S, device="cuda")
    ok = (s["u"] * q_x < p_x) & (i < s["n_draft"][:, None])
    n = ok.to(torch.int32).cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    target = p[b, n]
    refused = n < s["n_draft"]
    rest = target
    if S:
        less = (target - s["draft"][b, n.clamp_max(S - 1)]).clamp_min(0)
        use = refused & (less > 0).any(1)
        rest = torch.where(use[:, None], less, target)
    last = _first_max(rest / s["race"])
    at = torch.arange(S + 1, device="cuda")[None]
    padded = torch.cat([tokens, torch.zeros(B, 1, dtype=torch.long, device="cuda")], 1)
    out = torch.where(at < n[:, None], padded, torch.where(at == n[:, None], last[:, None], torch.full_like(padded, -1)))
    lp = logp.gather(2, out.clamp_min(0)[..., None])[..., 0]
    return out.to(torch.int32), n.to(torch.int32), torch.where(out >= 0, lp, torch.zeros_like(lp))


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def _tokens(c):
    """Tokens of each request that the sparse attention reads: its distinct selected blocks' valid ones."""
    want = c["k"] + c["q_len"] - 1
    got = []
    for n in _lens(c):
        nb = -(-n // PAGE)
        got.append(n if nb <= want else want * PAGE - (-n) % PAGE)
    return got


def work(case):
    c = case
    if c["op"] == "sparse":
        R, Hq = c["B"] * c["q_len"], c["Hkv"] * c["G"]
        a_token = 2 * D + 8 if c["dtype"] == "e4m3" else 4 * D
        each = [min(t, c["k"] * PAGE) for t in _tokens(c)]
        return dict(bytes=sum(_tokens(c)) * c["Hkv"] * a_token + R * Hq * (4 * D + 4) + 8 * R * c["Hkv"] * c["k"],
                    flops=4 * D * Hq * c["q_len"] * sum(each))
    if c["op"] == "prefix":
        R, Hq = c["B"] * c["q_len"], c["Hkv"] * c["G"]
        return dict(bytes=(c["prefix"] + sum(_lens(c))) * c["Hkv"] * 4 * D + R * Hq * (4 * D + 4),
                    flops=4 * D * Hq * c["q_len"] * (c["B"] * c["prefix"] + sum(_lens(c))))
    if c["op"] == "evict":
        B, cols, H = c["B"], c["cols"], c["Hkv"]
        nb = [-(-n // PAGE) for n in _lens(c)]
        kept = sum(min(n, c["budget"]) for n in nb)
        # weights read and the new ones written in full; the table read, the new one and the freed list written
        return dict(bytes=4 * H * (sum(nb) + B * cols) + 4 * (sum(nb) + 2 * B * cols) + 8 * B * c["q_len"] * H * c["k"],
                    flops=H * sum(nb) + kept)
    B, S, V = c["B"], c["S"], c["V"]
    size = 2 if c["dtype"] == "bf16" else 4
    rows = sum(1 + n for n in _n_draft(c))
    return dict(bytes=rows * V * size + sum(4 * V * (2 if n else 1) for n in _n_draft(c)), flops=4 * rows * V)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"sparse": _exact_sparse, "prefix": _exact_prefix, "evict": _exact_evict, "verify": _exact_verify}[
        case["op"]](s)


def _attend64(q, keys, vals, scale):
    """q [n, D], keys and vals [t, D] in 64 bits: out, lse and the weights."""
    if keys.shape[0] == 0:
        return q * 0, torch.full(q.shape[:1], -math.inf, device="cuda", dtype=torch.float64), None
    x = (q @ keys.T) * scale
    lse = x.logsumexp(1)
    w = (x - lse[:, None]).exp()
    return w @ vals, lse, w


def _token64(pool, scale, page, h, n):
    x = pool[page, :n, h]
    return x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale[page, h, :n, None].double()


def _exact_sparse(s):
    c = s["case"]
    q_len, H, G, k = c["q_len"], c["Hkv"], c["G"], c["k"]
    R = c["B"] * q_len
    out = torch.zeros(R, H, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, H, G), -math.inf, dtype=torch.float64, device="cuda")
    mass = torch.zeros(R, H, k, dtype=torch.float64, device="cuda")
    ids, table, lens = s["ids"].tolist(), s["table"].tolist(), _lens(c)
    for r in range(R):
        b, length = r // q_len, lens[r // q_len] - (q_len - 1 - r % q_len)
        for h in range(H):
            sel = [(i, j, min(PAGE, length - i * PAGE)) for j, i in enumerate(ids[r][h]) if i >= 0]
            sel = [(i, j, n) for i, j, n in sel if n > 0]
            if not sel:
                continue
            keys = torch.cat([_token64(s["kp"], s["ks"], table[b][i], h, n) for i, _, n in sel])
            vals = torch.cat([_token64(s["vp"], s["vs"], table[b][i], h, n) for i, _, n in sel])
            q = s["q"][r, h * G:(h + 1) * G].double()
            out[r, h], lse[r, h], w = _attend64(q, keys, vals, s["scale"])
            at = torch.tensor([j for _, j, n in sel for _ in range(n)], device="cuda")
            mass[r, h].index_add_(0, at, w.sum(0))
    return out.view(R, H * G, D), lse.view(R, H * G), mass


def _exact_prefix(s):
    c = s["case"]
    q_len, H, G, Lp = c["q_len"], c["Hkv"], c["G"], c["prefix"]
    R = c["B"] * q_len
    out = torch.zeros(R, H, G, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(R, H, G, dtype=torch.float64, device="cuda")
    table, lens, prefix = s["table"].long(), _lens(c), s["prefix"].long()
    for h in range(H):
        pk = s["kp"][prefix][:, :, h].reshape(-1, D)[:Lp].double()
        pv = s["vp"][prefix][:, :, h].reshape(-1, D)[:Lp].double()
        q = s["q"].view(R, H, G, D)[:, h].double()
        o1, l1, _ = _attend64(q.reshape(R * G, D), pk, pv, s["scale"])
        o1, l1 = o1.view(R, G, D), l1.view(R, G)
        for r in range(R):
            n = lens[r // q_len] - (q_len - 1 - r % q_len)
            rows = table[r // q_len, :max(0, -(-n // PAGE))]
            ok = s["kp"][rows][:, :, h].reshape(-1, D)[:max(n, 0)].double()
            ov = s["vp"][rows][:, :, h].reshape(-1, D)[:max(n, 0)].double()
            o2, l2, _ = _attend64(q[r], ok, ov, s["scale"])
            both = torch.logaddexp(l1[r], l2)
            out[r, h] = o1[r] * (l1[r] - both).exp()[:, None] + o2 * (l2 - both).exp()[:, None]
            lse[r, h] = both
    return out.view(R, H * G, D), lse.view(R, H * G)


def _exact_evict(s):
    import numpy as np
    c = s["case"]
    B, q_len, H, cols, budget = c["B"], c["q_len"], c["Hkv"], c["cols"], c["budget"]
    w, ids, mass = (s[n].cpu().numpy() for n in ("weights", "ids", "mass"))
    table, lens, n_rows = s["table"].cpu().numpy(), _lens(c), s["n_rows"].cpu().numpy()
    w64 = w.astype(np.float64)
    for b in range(B):
        for i in range(int(n_rows[b])):
            for h in range(H):
                row = ids[b * q_len + i, h]
                use = row >= 0
                w64[b, h, row[use]] += mass[b * q_len + i, h, use]
                w[b, h, row[use]] += mass[b * q_len + i, h, use]
    new_t, freed = np.full((B, cols), -1, np.int32), np.full((B, cols), -1, np.int32)
    new_w, new_n, n_freed = np.zeros((B, H, cols)), np.array(lens, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(lens):
        nb = -(-n // PAGE)
        total = w[b, 0, :nb].copy()  # which pages stay goes by the sum in 32 bits, in this order, by definition
        for h in range(1, H):
            total = total + w[b, h, :nb]
        pinned = [j for j in range(nb) if j < c["sink"] or j >= nb - c["window"]]
        rest = sorted(set(range(nb)) - set(pinned), key=lambda j: (-total[j], j))
        keep = np.array(sorted((pinned + rest)[:budget] if nb > budget else range(nb)), dtype=np.int64)
        gone = np.setdiff1d(np.arange(nb), keep)
        new_t[b, :len(keep)], freed[b, :len(gone)] = table[b, keep], table[b, gone]
        new_w[b, :, :len(keep)] = w64[b][:, keep]
        n_freed[b] = len(gone)
        new_n[b] = n - PAGE * len(gone)
    return new_t, new_n, new_w, freed, n_freed


def _exact_verify(s):
    c = s["case"]
    B, S, V = c["B"], c["S"], c["V"]
    out = torch.full((B, S + 1), -1, dtype=torch.int32)
    got, lp = torch.zeros(B, dtype=torch.int32), torch.zeros(B, S + 1, dtype=torch.float64)
    tokens, n_draft, temp, u = s["tokens"].tolist(), _n_draft(c), s["temp"].tolist(), s["u"].tolist()

    def probabilities(b, i):
        z = s["logits"][b, i].double()
        if temp[b] > 0:
            z = z / temp[b]
            z = z - z.logsumexp(0)
            return z, z.exp()
        p = torch.zeros(V, dtype=torch.float64, device="cuda")
        p[int((z == z.max()).nonzero()[0])] = 1.0
        return p.log(), p

    for b in range(B):
        i = 0
        while True:
            z, p = probabilities(b, i)
            if i < n_draft[b]:
                x = tokens[b][i]
                if u[b][i] * float(s["draft"][b, i, x]) < float(p[x]):
                    out[b, i], lp[b, i] = x, float(z[x])
                    i += 1
                    continue
                rest = (p - s["draft"][b, i].double()).clamp_min(0)
                p = rest if bool((rest > 0).any()) else p
            x = int((p / s["race"][b].double()).argmax())
            out[b, i], lp[b, i] = x, float(z[x])
            got[b] = i
            break
    return out, got, lp
