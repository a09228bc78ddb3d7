"""The example's decode step, stage by stage against plain forms."""

import os
import sys

import numpy as np
import pytest
import torch

import attention_ref as ref
from test_gpu_cache_evict import plain_evict
from test_gpu_verify_draft import plain as plain_verify

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_step():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_step as ex
    lens = [700, 130, 2900]
    s = ex.make_step(lens, prompt=300, vocab=500, seed=3)
    table, weights = s["table"].clone(), s["weights"].clone()
    r = ex.step(s, budget=12)
    assert r["faults"] == 0
    q_len, cols = ex.DRAFTS + 1, table.shape[1]
    cpu = {n: s[n].cpu() for n in ("q", "k", "v", "prompt_table", "logits", "draft", "tokens", "uniforms", "race",
                                   "temperature")}
    ids = r["ids"].cpu()
    want = ref.sparse(cpu["q"], cpu["k"], None, cpu["v"], None, table.cpu(), lens, ids, ex.D ** -0.5, q_len)
    ref.check(r["sparse"], want[0], "sparse")
    ref.check(r["mass"], want[2], "mass")
    # the layer with full attention: the prompt, then the request's own tokens
    H, G = ex.KV_HEADS, ex.GROUP
    for row in (0, 5, 11):
        b, n = row // q_len, lens[row // q_len] - (q_len - 1 - row % q_len)
        for h in range(H):
            pages = [(int(p), min(ex.PAGE, 300 - j * ex.PAGE)) for j, p in enumerate(cpu["prompt_table"].tolist())]
            pages += [(int(table[b, j]), min(ex.PAGE, n - j * ex.PAGE)) for j in range(-(-n // ex.PAGE))]
            keys, vals = (torch.cat([ref.gather(x, None, p, h, m) for p, m in pages]) for x in (cpu["k"], cpu["v"]))
            out, lse, _, tol, lse_tol = ref.row(cpu["q"][row, h * G:(h + 1) * G].double(), keys, vals, ex.D ** -0.5)
            ref.check(r["full"][row, h * G:(h + 1) * G], (out, tol), "full")
            ref.check(r["lse"][row, h * G:(h + 1) * G], (lse, lse_tol), "lse")
    out, acc, _, margin = plain_verify(cpu["logits"], cpu["draft"], cpu["tokens"], cpu["uniforms"], cpu["race"],
                                       cpu["temperature"], torch.full((3,), ex.DRAFTS))
    assert margin > 1e-5 and torch.equal(r["tokens"].cpu(), out) and torch.equal(r["accepted"].cpu(), acc)
    # weights of the positions that count, then the pages that stay
    w, mass = weights.cpu().numpy(), r["mass"].cpu().numpy()
    for b in range(3):
        for i in range(int(acc[b]) + 1):
            for h in range(H):
                for j, x in enumerate(ids[b * q_len + i, h].tolist()):
                    if x >= 0:
                        w[b, h, x] += mass[b * q_len + i, h, j]
    left = [n - (ex.DRAFTS - int(a)) for n, a in zip(lens, acc)]
    kept = plain_evict(table.cpu().numpy(), left, w, 12, ex.SINK, ex.WINDOW)
    for got, x in zip((s["table"], s["seq"], s["weights"], r["freed"], r["n_freed"]), kept):
        np.testing.assert_array_equal(got.cpu().numpy(), x)
    again = ex.step(s, budget=12)  # the shrunk cache serves the next step
    assert again["faults"] == 0 and bool(torch.isfinite(again["sparse"].float()).all())
    assert cols == table.shape[1]
