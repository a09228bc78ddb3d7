"""One decode step of a sparse-attention server with drafted tokens, from block scores to the pages that leave.

    python examples/serve_step.py

A batch of requests, each with three drafted tokens (four query positions), goes through what a serving loop does with
this library, on synthetic tensors:

1. the indexer scores every block of the paged index-K cache and picks k of them for each position and KV group;
2. attention over the picked blocks of the K/V cache, with the mass each block received;
3. a layer with full attention, whose requests share a system prompt: the prompt's K/V is read once for all of them;
4. the drafted tokens are verified against the target's probabilities;
5. the mass of the accepted positions is added to the pages' weights, and requests over their budget of pages give the
   lightest ones back.  The block table is shared by the index-K and the K/V cache, so both shrink together.
"""

from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_attention_decode_gb300 as msa  # noqa: E402

PAGE, D = 128, 128
DRAFTS = 3  # drafted tokens a request; DRAFTS + 1 positions a step
KV_HEADS, GROUP, K = 4, 16, 16
SINK, WINDOW = 1, 2


def make_step(lens, prompt, vocab, seed=0):
    """Synthetic state of a server between two steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    B, q_len = len(lens), DRAFTS + 1
    cols = max(-(-n // PAGE) for n in lens)
    prompt_pages = -(-prompt // PAGE)
    pages = prompt_pages + B * cols
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    held = torch.tensor([[j < -(-n // PAGE) for j in range(cols)] for n in lens], device="cuda")
    table = torch.where(held, order[prompt_pages:].view(B, cols), torch.full((1,), -1, dtype=torch.int32, device="cuda"))
    s = dict(
        seq=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        table=table,
        prompt_table=order[:prompt_pages].contiguous(),
        prompt_len=torch.tensor([prompt], dtype=torch.int32, device="cuda"),
        # head-major pages: a page's tile of one KV head is contiguous
        index_k=randn(pages, PAGE, D).to(torch.bfloat16),
        k=randn(pages, KV_HEADS, PAGE, D).to(torch.bfloat16).permute(0, 2, 1, 3),
        v=randn(pages, KV_HEADS, PAGE, D).to(torch.bfloat16).permute(0, 2, 1, 3),
        index_q=randn(B * q_len, 4, D).to(torch.bfloat16),
        q=randn(B * q_len, KV_HEADS * GROUP, D).to(torch.bfloat16),
        weights=torch.zeros(B, KV_HEADS, cols, device="cuda"),
        logits=2.5 * randn(B, q_len, vocab))
    draft = torch.softmax(s["logits"][:, :DRAFTS] + 0.6 * randn(B, DRAFTS, vocab), 2)
    noise = torch.empty_like(draft).exponential_(generator=g)
    s.update(draft=draft, tokens=(draft / noise).argmax(2).to(torch.int32),
             uniforms=torch.rand(B, DRAFTS, device="cuda", generator=g),
             race=torch.empty(B, vocab, device="cuda").exponential_(generator=g),
             temperature=torch.full((B,), 1.0, device="cuda"))
    return s


def step(s, budget):
    """One step; the table, lengths and weights in `s` are updated in place."""
    B, cols = s["table"].shape
    q_len, rows = DRAFTS + 1, B * (DRAFTS + 1)
    limit = cols * PAGE
    empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731

    # 1. blocks: [B, positions, KV heads, K]
    ids, scores = empty(B, q_len, 4, K, dtype=torch.int32), empty(B, q_len, 4, K)
    ws = torch.zeros(msa.msa_indexer_workspace_bytes_mq(B, limit, K, q_len=q_len), dtype=torch.uint8, device="cuda")
    msa.msa_indexer_decode_mq(s["index_q"].view(B, q_len, 4, D), s["index_k"], s["table"], s["seq"], K, SINK, WINDOW,
                              ids, scores, ws, max_model_len=limit)

    # 2. attention over them, and what each received
    ids = ids.view(rows, KV_HEADS, K)
    sparse, mass = torch.empty_like(s["q"]), empty(rows, KV_HEADS, K)
    msa.msa_attention_sparse(s["q"], s["k"], s["v"], s["table"], s["seq"], ids, sparse, ws, scale=D ** -0.5,
                             q_len=q_len, out_mass=mass)

    # 3. a layer with full attention over the shared prompt and each request's own tokens
    full, lse = torch.empty_like(s["q"]), empty(rows, KV_HEADS * GROUP)
    pws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(rows, KV_HEADS * GROUP, KV_HEADS,
                                                               PAGE * s["prompt_table"].numel()),
                      dtype=torch.uint8, device="cuda")
    msa.msa_attention_prefix(s["q"], s["k"], s["v"], s["prompt_table"], s["prompt_len"], s["table"], s["seq"], full,
                             pws, scale=D ** -0.5, q_len=q_len, out_lse=lse)

    # 4. which drafts stand, and the token behind them
    out, accepted, logp = empty(B, q_len, dtype=torch.int32), empty(B, dtype=torch.int32), empty(B, q_len)
    msa.msa_verify_draft(s["logits"], s["draft"], s["tokens"], s["uniforms"], s["race"], out, accepted, ws,
                         temperature=s["temperature"], out_logprobs=logp)

    # 5. the mass of the positions that count (the one before the first draft, then the accepted drafts); the refused
    # drafts' tokens leave the cache's end, the lightest pages of requests over their budget its middle (a page that held
    # refused drafts alone leaves the table unlisted: a server takes its number from the table before this call)
    msa.msa_cache_accumulate(s["weights"], ids, mass, ws, q_len=q_len, n_rows=accepted + 1)
    s["seq"] -= DRAFTS - accepted
    freed, n_freed = torch.empty_like(s["table"]), empty(B, dtype=torch.int32)
    msa.msa_cache_evict(s["table"], s["seq"], s["weights"], budget, SINK, WINDOW, s["table"], s["seq"], s["weights"],
                        freed, n_freed, ws)

    faults = msa.msa_indexer_get_error(ws) | msa.msa_indexer_get_error(pws)
    return dict(ids=ids, sparse=sparse, mass=mass, full=full, lse=lse, tokens=out, accepted=accepted, logp=logp,
                freed=freed, n_freed=n_freed, faults=faults)


def main():
    s = make_step(lens=[5000, 700, 12000, 3333], prompt=2500, vocab=32000)
    for i in range(2):
        r = step(s, budget=24)
        print(f"step {i}: accepted {r['accepted'].tolist()}, tokens {r['tokens'].tolist()}, pages freed "
              f"{r['n_freed'].tolist()}, lengths {s['seq'].tolist()}, faults {r['faults']}")


if __name__ == "__main__":
    main()
