"""A small language model on the library's vocabulary-side operators: trained, quantised to a 4-bit head, and served.

The model predicts a token's successor: h = sqrt(D) * table[token], z = h W, logits = z table^T with one table for both
ends (tied embeddings). It learns a synthetic chain in which every token has four possible successors.

* training: ``vsamp_embed`` -> z, logits (library products) -> ``vsamp_score_tokens`` (loss: minus the mean
  log-probability of the targets minus a small entropy bonus) -> ``vsamp_score_tokens_backward`` into the logits' own
  buffer -> gradients of W and the table, the lookup's part added by ``vsamp_embed_backward``;
* serving: the table in 4 bits (``vsamp_head_pack``), one decode step captured as a CUDA graph: ``vsamp_embed`` ->
  ``vsamp_head_logits`` -> ``vsamp_sample`` -> ``vsamp_score_tokens`` (log-probability, rank and alternatives of the
  drawn token).

    python -m examples.tied_lm
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

import top_sampling_gb300 as ts


class Chain:
    """Four equally likely successors for every token."""

    def __init__(self, V: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.V = V
        self.next = torch.stack([torch.randperm(V, generator=g) for _ in range(4)], dim=1)

    def batch(self, n: int, gen: torch.Generator, dev):
        tok = torch.randint(0, self.V, (n,), generator=gen)
        target = self.next[tok, torch.randint(0, 4, (n,), generator=gen)]
        # every eighth position stands for a prompt token: it is not scored
        target[::8] = ts.VSAMP_TOKEN_IGNORE
        return tok.to(dev, torch.int32), target.to(dev, torch.int32)

    def is_successor(self, tok, nxt):
        return (self.next.to(tok.device)[tok.long()] == nxt.long()[:, None]).any(dim=1)


class Model(NamedTuple):
    table: torch.Tensor    # [V, D] fp32
    W: torch.Tensor        # [D, D] fp32


def gradients(model: Model, tok, target, entropy_bonus: float = 0.0):
    """Loss and gradients of the mean over the scored positions."""
    table, W = model
    V, D = table.shape
    scored = (target != ts.VSAMP_TOKEN_IGNORE).sum()
    t16, w16 = table.bfloat16(), W.bfloat16()
    h, _ = ts.vsamp_embed(tok, t16, scale=math.sqrt(D))
    z = h @ w16
    logits = z @ t16.t()
    lp, ent, _, _, _, m, logsum, status = ts.vsamp_score_tokens(logits, target)
    loss = -(lp.sum() + entropy_bonus * ent.sum()) / scored
    g = (-1.0 / scored).expand(tok.numel()).contiguous()
    dlogits, _ = ts.vsamp_score_tokens_backward(logits, target, g, m, logsum, entropy=ent, dentropy=entropy_bonus * g,
                                                dlogits=logits)
    dz = dlogits @ t16
    dtable = (dlogits.t() @ z).float()
    dW = (h.t() @ dz).float()
    dh = dz @ w16.t()
    ts.vsamp_embed_backward(tok, dh, V, scale=math.sqrt(D), dtable=dtable, accumulate=True)
    return loss, status, Model(dtable, dW)


def train(chain: Chain, D: int = 256, steps: int = 400, batch: int = 4096, lr: float = 3e-3, seed: int = 1,
          device="cuda"):
    """Adam on the model's two matrices. Returns the model and the losses."""
    dev = torch.device(device)
    gen = torch.Generator().manual_seed(seed)
    model = Model((torch.randn((chain.V, D), generator=gen) * D ** -0.5).to(dev),
                  (torch.eye(D) + torch.randn((D, D), generator=gen) * 0.02).to(dev))
    first = Model(*(torch.zeros_like(p) for p in model))
    second = Model(*(torch.zeros_like(p) for p in model))
    losses = []
    for step in range(1, steps + 1):
        tok, target = chain.batch(batch, gen, dev)
        loss, status, grad = gradients(model, tok, target, entropy_bonus=0.01)
        losses.append(loss)
        for p, d, a, b in zip(model, grad, first, second):
            a.mul_(0.9).add_(d, alpha=0.1)
            b.mul_(0.99).addcmul_(d, d, value=0.01)
            p.addcdiv_(a / (1 - 0.9 ** step), (b / (1 - 0.99 ** step)).sqrt_().add_(1e-8), value=-lr)
    return model, torch.stack(losses).tolist()


def quantise(weight: torch.Tensor, group: int = 64):
    """4-bit codes (even elements in the low nibble), bf16 scales and zero points of [V, D] weights, by the range of
    every group."""
    V, D = weight.shape
    w = weight.float().view(V, D // group, group)
    lo, hi = w.amin(dim=2).clamp(max=0), w.amax(dim=2).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
    zero = torch.round(-lo / scale.float()).clamp(0, 15)
    q = torch.round(w / scale.float()[:, :, None] + zero[:, :, None]).clamp(0, 15).to(torch.uint8).view(V, D)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


class Server:
    """A decode step for a fixed batch, captured once and replayed."""

    def __init__(self, model: Model, batch: int, n_alt: int = 4, temperature: float = 0.8, top_k: int = 20):
        dev = model.table.device
        D = model.table.shape[1]
        codes, scale, zero = quantise(model.table)
        self.head = ts.vsamp_head_pack(codes, scale, zeros=zero, group=64)
        self.table, self.W = model.table.bfloat16(), model.W.bfloat16()
        self.token = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.step = torch.zeros(batch, dtype=torch.int64, device=dev)
        self.seed = torch.arange(batch, dtype=torch.int64, device=dev)
        self.temperature = torch.full((batch,), temperature, device=dev)
        self.top_k = torch.full((batch,), top_k, dtype=torch.int32, device=dev)

        def decode():
            h, _ = ts.vsamp_embed(self.token, self.table, scale=math.sqrt(D))
            logits = ts.vsamp_head_logits(h @ self.W, self.head)
            token, _, status, _ = ts.vsamp_sample(logits, temperature=self.temperature, top_k=self.top_k, seed=self.seed,
                                                  step=self.step)
            scores = ts.vsamp_score_tokens(logits, token, temperature=self.temperature, n_alt=n_alt)
            self.token.copy_(token)
            self.step += 1
            return token, status, scores

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            decode()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = decode()

    def generate(self, first: torch.Tensor, n: int):
        """n tokens after `first` [batch]. Returns tokens [n, batch], log-probabilities and ranks of the same shape."""
        self.token.copy_(first)
        self.step.zero_()
        rows = []
        for _ in range(n):
            self.graph.replay()
            token, status, scores = self.out
            rows.append((token.clone(), scores[0].clone(), scores[2].clone(), status.clone()))
        token, lp, rank, status = (torch.stack(c) for c in zip(*rows))
        if status.any():
            raise RuntimeError(f"rows failed: {status.unique().tolist()}")
        return token, lp, rank


def main(V: int = 2000, steps: int = 400, n: int = 32, batch: int = 16):
    chain = Chain(V)
    model, losses = train(chain, steps=steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} (the chain's entropy is {math.log(4):.3f})")
    server = Server(model, batch)
    first = torch.arange(batch, dtype=torch.int32, device=model.table.device)
    token, lp, rank = server.generate(first, n)
    before = torch.cat([first[None], token[:-1]])
    legal = chain.is_successor(before.reshape(-1), token.reshape(-1)).float().mean()
    print(f"{n} tokens for {batch} sequences: {100 * float(legal):.1f}% legal successors, mean log-probability "
          f"{float(lp.mean()):.3f}, largest rank {int(rank.max())}")
    return losses, float(legal), lp, rank


if __name__ == "__main__":
    main()
