"""A small model trained on packed updates, from the packer to the weights.

One process, one GPU: ``Packer.step`` assembles an update's rows, and the model's
operators take its arrays as they are:

    tokens -> embedding -> gated_scan (pos, doc) -> route (doc) -> experts
           -> logits -> distill_loss (mask) -> gradients

The corpus is the synthetic two-source one, the weights are random, and the
teacher is a stand-in that knows the next token: what is shown is how the parts
fit.  The corpus's tokens are random, so there is nothing to learn from one update
for another: the model is trained on the first one again and again, whose loss
falls as it is memorised.

    python examples/packed_training_step.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import deterministic_packed_assembly_gb300 as nsp  # noqa: E402
from corpus import make_preset  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab: int, width: int = 256, experts: int = 8, chosen: int = 2):
        super().__init__()
        self.chosen = chosen
        self.embed = torch.nn.Embedding(vocab, width)
        self.mix = torch.nn.Linear(width, 2 * width)
        self.forget = torch.nn.Parameter(torch.linspace(0.0, 5.0, width))  # short memories to long
        self.router = torch.nn.Linear(width, experts, bias=False)
        self.experts = torch.nn.Parameter(torch.randn(experts, width, width) * width**-0.5)
        self.head = torch.nn.Linear(width, vocab, bias=False)

    def forward(self, tokens, pos, doc):
        B, T = tokens.shape
        x = self.embed(tokens)
        z, f = self.mix(x).chunk(2, dim=-1)  # halves of one projection, taken as they lie
        y, _ = nsp.gated_scan(z, f, self.forget, pos=pos, doc=doc)
        x = (x + y).reshape(B * T, -1)
        r = nsp.route(self.router(x), self.chosen, doc=doc.reshape(-1))
        # the few small experts are all computed; a large model would gather by r.ids
        share = torch.zeros(B * T, self.experts.shape[0], device=x.device)
        share = share.scatter_add(1, r.ids.clamp(min=0).long(), r.weights)
        x = x + torch.einsum("ne,nd,edk->nk", share, x, self.experts).tanh()
        return self.head(x), r


def targets(tokens, pos, mask):
    """Each position's next token, and whether it is learned: the next position is,
    and it goes on with the same document."""
    nxt = torch.roll(tokens, -1, dims=1)
    learned = torch.roll(mask, -1, dims=1) * (torch.roll(pos, -1, dims=1) != 0)
    learned[:, -1] = 0
    return nxt.reshape(-1), learned.reshape(-1).to(torch.uint8)


def teacher(nxt, vocab: int, k: int = 16):
    """Top logits of a teacher that gives the next token most of its probability."""
    others = (nxt[:, None] + torch.arange(k, device=nxt.device) * 977) % vocab
    logits = torch.linspace(0.0, -3.0, k, device=nxt.device).expand(nxt.numel(), k).clone()
    logits[:, 0] = 3.0
    return logits, others.int()


def train(steps: int = 8, seed: int = 0, device: str = "cuda:0"):
    """Losses of the steps."""
    torch.manual_seed(seed)
    corpus = make_preset("c1")
    packer = nsp.Packer.from_corpus(corpus, device=device)
    model = Model(corpus.vocab).to(device)
    optimizer = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for k in range(steps):
        out = packer.step(0)
        tokens, pos, doc, mask = (out[n][0] for n in ("tokens", "pos", "doc", "mask"))
        nxt, learned = targets(tokens, pos, mask)
        top, ids = teacher(nxt, corpus.vocab)
        logits, routing = model(tokens, pos, doc)
        each = nsp.distill_loss(logits, top, ids, mask=learned)
        loss = each.sum() / learned.sum().clamp(min=1)
        optimizer.zero_grad(set_to_none=True)
        (loss + 0.01 * routing.loss).backward()
        optimizer.step()
        losses.append(float(loss.detach()))
        print(f"step {k}: loss {losses[-1]:.4f}  balance {float(routing.loss.detach()):.3f}  "
              f"learned {int(learned.sum())} of {learned.numel()}  "
              f"experts' tokens {routing.counts.tolist()}")
    packer.check()
    packer.close()
    return losses


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
