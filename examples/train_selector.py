"""Train a candidate selector on the GPU: every training operator in the order of a step.

    python examples/train_selector.py [--steps 60] [--state-bits 8]

The task is synthetic: a table says how well each class of token follows each predecessor,
and the right token of a position is the candidate that follows best.  The unary logits
do not know the table; the codebooks can learn it.  A step is

    h       = embedding(E, context)                     rows of the embedding by token id
    ids, u, G = unary_topk(h, W_lm, K, W_H)             the candidates, their logits, h W_H^T
    loss, dscores, dG, dA, dBc = selector_loss_grad(...)
    dW_H    = dG^T h,  dh = dG W_H                      (plain matrix products)
    dE      = embedding_grad(dh, context)
    AdamW over E, W_H, A and Bc: bf16 weights with fp32 masters, states in 8 or 32 bits
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dflash2_draft_block_gb300 as df2  # noqa: E402


def train(steps=60, positions=2048, vocab=4096, hidden=256, rank=64, top_k=16, state_bits=8, seed=0):
    """The mean loss of every step (rows whose right token is a candidate)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def weights(*shape, std):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    E, W_lm = weights(vocab, hidden, std=0.5) + 1.0, weights(vocab, hidden, std=0.05)
    W_H, A, Bc = weights(rank, hidden, std=1.0), weights(vocab, rank, std=0.3), weights(vocab, rank, std=0.3)
    classes = 64
    follows = torch.randn(classes, classes, generator=gen, device="cuda")
    params = [E, W_H, A, Bc]
    grads = [torch.zeros_like(p, dtype=torch.float32) for p in params]
    opt = df2.AdamW(params, grads, lr=[1e-3, 3e-3, 3e-2, 3e-2], weight_decay=0.0, state_bits=state_bits,
                    master_weights=True)
    scale = hidden ** -0.5
    losses = []
    for _ in range(steps):
        context = torch.randint(0, vocab, (positions,), generator=gen, device="cuda", dtype=torch.int32)
        context[:: 16] = -1                                      # padding
        pred = torch.randint(0, classes, (positions,), generator=gen, device="cuda", dtype=torch.int32)
        h = df2.embedding(E, context, scale=scale)
        ids, vals, G = df2.unary_topk(h, W_lm, top_k, W_H)
        column = follows[pred.long()].gather(1, ids.long() % classes).argmax(dim=1)
        targets = ids.gather(1, column[:, None])[:, 0]
        targets = torch.where(context < 0, torch.full_like(targets, -1), targets)
        loss, label, dscores, dG, _, _ = df2.selector_loss_grad(pred, targets, ids, vals, G, A, Bc,
                                                                dA=grads[2], dBc=grads[3])
        grads[1].copy_(dG.t() @ h.float())
        df2.embedding_grad(dG @ W_H.float(), context, vocab, scale=scale, out=grads[0])
        # gradients of the sum so far: the mean's by the optimiser (no counted row: no step)
        counted = (label >= 0).sum()
        opt.step(grad_scale=(1.0 / counted.float()).reshape(1))
        losses.append(torch.where(label >= 0, loss, torch.zeros_like(loss)).sum() / counted)
    return [float(x) for x in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    losses = train(a.steps, state_bits=a.state_bits)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
