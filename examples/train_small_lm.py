"""Train a small language model with every step of libmuon: the norms between
its blocks, the head's cross entropy with its gradient, the global gradient
norm, Muon on the matrices of the blocks and AdamW on the embedding, the head
and the gains; then look at what it has learnt: how likely it finds the words
of a held-out text, how sure it is and what else it expects.

    python examples/train_small_lm.py [--steps 60]

The text is synthetic: every word has a few likely successors. The inside of
the model's two blocks (over the last two words) is plain torch; weights that
AdamW owns are 32-bit with the 16-bit copies that the model computes with.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import muon_newton_schulz_update_amd as mu  # noqa: E402

VOCAB, WIDTH, BLOCKS, TOKENS = 4096, 256, 2, 2048
BF = torch.bfloat16


class Model:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        normal = lambda *s, sd: torch.randn(*s, generator=g, device="cuda") * sd
        # Muon's: the blocks' matrices, 16-bit
        self.matrices = [normal(*s, sd=0.02).to(BF) for _ in range(BLOCKS)
                         for s in ((4 * WIDTH, 2 * WIDTH), (WIDTH, 4 * WIDTH))]
        self.momenta = [torch.zeros(w.shape, device="cuda") for w in self.matrices]
        # AdamW's: embedding, head, gains
        self.masters = [normal(VOCAB, WIDTH, sd=1.0), normal(VOCAB, WIDTH, sd=0.02)] + [
            torch.ones(WIDTH, device="cuda") for _ in range(BLOCKS + 1)]
        self.copies = [w.to(BF) for w in self.masters]
        self.firsts = [torch.zeros_like(w) for w in self.masters]
        self.seconds = [torch.zeros_like(w) for w in self.masters]
        for p in self.matrices + self.copies:
            p.requires_grad_()

    def hidden(self, words: torch.Tensor) -> torch.Tensor:
        embedding, gains = self.copies[0], self.copies[2:]
        x = embedding[words]
        h = mu.rms_norm(x, gains[0])
        for b in range(BLOCKS):
            y = torch.cat((h, torch.roll(h, 1, 0)), 1)
            y = torch.relu(y @ self.matrices[2 * b].t()).square()
            # the block's end and the next one's start (or the head's)
            x, h = mu.residual_norm(x, y @ self.matrices[2 * b + 1].t(), post_norm=False, pre_gain=gains[b + 1])
        return h

    def score(self, words: torch.Tensor, targets: torch.Tensor, top: int = 4) -> mu.LogProbs:
        """Log probabilities of the targets, the distributions' entropies and their likeliest words."""
        with torch.no_grad():
            return mu.linear_logprobs(self.hidden(words), self.copies[1], targets, top=top)

    def step(self, words: torch.Tensor, targets: torch.Tensor, number: int) -> tuple[torch.Tensor, torch.Tensor]:
        """One training step; (loss, gradient norm), both still on the device."""
        loss = mu.linear_cross_entropy(self.hidden(words), self.copies[1], targets)
        loss.backward()
        matrix_grads = [p.grad for p in self.matrices]
        other_grads = [p.grad for p in self.copies]
        norm, coef = mu.grad_norm(matrix_grads + other_grads, max_norm=1.0)
        with torch.no_grad():
            mu.scale(matrix_grads, coef)
            mu.muon_update(matrix_grads, self.momenta, self.matrices, mu.make_config(lr=0.01))
            mu.adamw_update(other_grads, self.firsts, self.seconds, self.masters, step=number, lr=0.01, eps=1e-8,
                            grad_scale=coef, copies=self.copies)
        for p in self.matrices + self.copies:
            p.grad = None
        return loss.detach(), norm


def text(seed: int, likely: torch.Tensor) -> torch.Tensor:
    """TOKENS + 1 words, each one of the four likely successors of the one before."""
    g = torch.Generator()
    g.manual_seed(seed)
    choice = torch.randint(0, likely.shape[1], (TOKENS,), generator=g).tolist()
    table, words = likely.tolist(), [seed % VOCAB]
    for c in choice:
        words.append(table[words[-1]][c])
    return torch.tensor(words, device="cuda")


def language() -> torch.Tensor:
    """Each word's four likely successors; an eighth of the words occur."""
    g = torch.Generator()
    g.manual_seed(1)
    return torch.randint(0, VOCAB // 8, (VOCAB, 4), generator=g)


def train(steps: int, say=print, model: Model | None = None) -> list[float]:
    model, likely, losses = model or Model(), language(), []
    for k in range(1, steps + 1):
        words = text(k, likely)
        targets = words[1:].clone()
        targets[::64] = -100                      # positions that are no part of the loss
        losses.append(model.step(words[:-1], targets, k))
        if say and (k == 1 or k % 10 == 0):
            say(f"step {k:4d}  loss {float(losses[-1][0]):.3f}  gradient norm {float(losses[-1][1]):.3f}", flush=True)
    return [float(x) for x, _ in losses]


def look(model: Model, say=print) -> dict[str, float]:
    """A held-out text: mean log probability and entropy, and how often the next word is among the four likeliest."""
    words = text(0, language())
    out = model.score(words[:-1], words[1:])
    among = (out.top_tokens == words[1:, None]).any(1).float().mean()
    found = dict(logprob=float(out.logprobs.mean()), entropy=float(out.entropy.mean()), among_four=float(among))
    if say:
        say("held out  " + "  ".join(f"{k} {v:.3f}" for k, v in found.items()), flush=True)
    return found


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    trained = Model()
    train(ap.parse_args().steps, model=trained)
    look(trained)
