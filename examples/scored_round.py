"""One MTP round with log probabilities: the residual stream is normed (add_rmsnorm), three tokens are drafted from
the candidate table, the target verifies them against the full head, and the tokens that the round emits are scored
(head_logprobs: log probability, entropy and the five best alternatives of each position).  Then one training step of
the scored positions: log probabilities from logits, their gradient, and the norm's gradient.

    python examples/scored_round.py            # random weights, needs a GPU and the built library
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import verify_head_gb300 as vh

B, K, H, V, VC, TOP = 4, 3, 1024, 32_000, 8_192, 5


def main():
    vh.build()
    g = torch.Generator("cuda").manual_seed(0)
    bf16 = torch.bfloat16

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(bf16)

    W = randn(V, H, scale=0.05)                                           # full head
    cand = torch.sort(torch.randperm(V, generator=g, device="cuda")[:VC]).values.int()
    W_cand = W[cand.long()].contiguous()                                  # candidate table
    embed = randn(V, H)
    weight = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(bf16)
    stream = randn(B, H, scale=2.0)                                       # residual stream after the last verified token
    layer_out = randn(B, H)

    # Draft: norm, candidate head, next token's embedding into the stream.
    ws = vh.workspace(B)
    drafts, x, h = [], layer_out, stream
    for _ in range(K):
        hidden, h = vh.add_rmsnorm(x, h, weight)
        ids, _ = vh.mtp_draft_head_argmax(hidden, W_cand, cand, ws=ws)
        drafts.append(ids.clone())
        x = embed[ids.long()]
    draft_ids = torch.stack(drafts, 1).contiguous()                       # [B, K]

    # Verify: the target's hidden rows of the K + 1 positions (random here, in place of the target model).
    rows = B * (K + 1)
    target_x, target_stream = randn(rows, H), randn(rows, H, scale=2.0)
    hidden, h = vh.add_rmsnorm(target_x, target_stream, weight)
    accept_len, next_ids, _ = vh.spec_verify_greedy(hidden, W, draft_ids, B, K)

    # Score the target's token of every position; padding (-1) past the emitted ones.
    pos = torch.arange(K + 1, device="cuda")[None, :]
    emitted = torch.where(pos <= accept_len[:, None], next_ids.view(B, K + 1), -1).int().reshape(-1)
    logprob, entropy, lse, top_ids, top_lp = vh.head_logprobs(hidden, W, emitted, TOP)
    assert torch.equal(top_ids[:, 0], next_ids)  # the first alternative is the verify kernel's argmax
    for b in range(B):
        n = int(accept_len[b]) + 1
        for j in range(n):
            r = b * (K + 1) + j
            print(f"sequence {b} token {int(emitted[r])}: logprob {float(logprob[r]):.3f} entropy {float(entropy[r]):.3f}"
                  f" alternatives {top_ids[r].tolist()}")

    # Train: the same positions from logits in memory, the gradient of -mean(logprob) - 0.01 mean(entropy), back
    # through the head (a plain product) and the norm.
    logits = hidden @ W.t()
    lp, ent, lse, _, _ = vh.logits_logprobs(logits, emitted)
    count = (emitted >= 0).sum()
    dlogits = vh.logits_logprobs_grad(logits, emitted, lse, ent, (-1.0 / count).expand(rows).contiguous().float(),
                                      torch.full((rows,), -0.01 / rows, device="cuda"), dlogits=logits)
    dhidden = dlogits @ W
    dx, dweight = vh.add_rmsnorm_grad(dhidden, h, weight)
    print(f"scored again from bf16 logits: largest difference {float((lp - logprob).abs().max()):.4f};"
          f" |dx| {float(dx.float().norm()):.4f} |dweight| {float(dweight.norm()):.4f}")

    # The stream in 8 bits, for a layer that takes them.
    q, scales, _ = vh.add_rmsnorm_q8(target_x, target_stream, weight)
    off = (q.float() * scales[:, None] - hidden.float()).abs().max() / hidden.float().abs().max()
    print(f"int8 rows: largest error {float(off):.4f} of the largest value")


if __name__ == "__main__":
    main()
