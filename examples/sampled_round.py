"""One MTP round that samples from a 4-bit target head: the hidden rows go to 4 bits with a scale for each row, are multiplied with
the 4-bit head, and the logits of the K + 1 positions are processed (a bias, penalties for tokens of the history and of the draft
before each position, a grammar mask, temperature).  A token is drawn from each row, its log probability kept.  Then the gradient of
a policy's loss, through the processing and the head.

    python examples/sampled_round.py            # random weights, needs a GPU and the built library
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import verify_head_gb300 as vh

B, K, H, V, L = 4, 3, 1024, 32_000, 200


def main():
    vh.build()
    g = torch.Generator("cuda").manual_seed(0)
    rows = B * (K + 1)
    ints = lambda hi, *shape: torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731

    # Once: the head in 4 bits, and its tiled copy for the product.
    W = torch.randn(V, H, generator=g, device="cuda").mul_(0.05).bfloat16()
    g_head = float(W.abs().max()) / 2688
    codes, scales, _ = vh.nvfp4_quantize(W, g_head)
    table = vh.nvfp4_tile(codes, scales)
    print(f"head: {W.numel() * 2 / 1e6:.0f} MB in bf16, {table.numel() / 1e6:.0f} MB in 4 bits")

    # The round: hidden rows of the last verified token and the K drafted ones (random, in place of the target model).
    hidden = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    x, x_scales = vh.nvfp4_quantize_tiles(hidden)
    logits = vh.nvfp4_matmul(x, x_scales, table, g_head, rows, V, H)
    rules = dict(history=ints(V, B, L), history_len=torch.tensor([200, 150, 20, 0], dtype=torch.int32, device="cuda"),
                 prompt_len=torch.full((B,), 20, dtype=torch.int32, device="cuda"), draft_ids=ints(V, B, K),
                 repetition=torch.full((B,), 1.1, device="cuda"), frequency=torch.full((B,), 0.2, device="cuda"),
                 presence=torch.full((B,), 0.1, device="cuda"), temperature=torch.tensor([0.7, 1.0, 1.3, 0.0], device="cuda"),
                 bias_ids=ints(V, B, 2), bias=torch.tensor([[5.0, -5.0]] * B, device="cuda"),
                 allowed=ints(2 ** 31 - 1, rows, V // 32))
    out = vh.logits_process(logits, **rules)
    tokens = torch.multinomial(torch.softmax(out.float(), 1), 1, generator=g)[:, 0].int()
    words = rules["allowed"].gather(1, (tokens // 32).long()[:, None])[:, 0]
    assert bool(((words >> (tokens % 32)) & 1).all())  # nothing that the grammar forbids
    logprob, entropy, lse, best, _ = vh.logits_logprobs(out, tokens, 1)
    greedy = best.view(B, K + 1)[3]  # the last sequence's temperature is 0
    print(f"tokens {tokens.view(B, K + 1)[:3].tolist()}, greedy {greedy.tolist()}; mean log probability {float(logprob.mean()):.3f}")

    # Train: -mean(advantage * logprob), back through the processing and the head.
    advantage = torch.randn(rows, generator=g, device="cuda")
    d = vh.logits_logprobs_grad(out, tokens, lse, entropy, -advantage / rows)
    d = vh.logits_process_grad(d, logits, **rules)  # (dlogits=d saves the buffer, and takes longer)
    dhidden = d @ vh.nvfp4_dequantize(codes, scales, g_head)
    print(f"|dlogits| {float(d.float().norm()):.4f} |dhidden| {float(dhidden.float().norm()):.4f}")
    assert bool(torch.isfinite(dhidden).all())


if __name__ == "__main__":
    main()
