"""Text from a model of two tokens, through the library from end to end.

    python examples/generate.py [--corpus FILE] [--merges N] [--rows R] [--tokens T]

A vocabulary is trained on a corpus, the corpus encoded with it, and the ids that follow each id are
counted.  The model's hidden state after an id is the row of log-probabilities of what follows it; the
stream that is added to it is the log-probability of each token alone; its head is the identity, in 8
bits.  Each step then runs as a decoding step of any model does: norm, logits, draw, and at the end the
ids become bytes.  The steps are captured in a CUDA graph and replayed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bpe_trie_encode_gb300 as bt  # noqa: E402


class Bigrams:
    """Counts of pairs of neighbouring ids, as hidden states [n_tok, n_tok] and the stream [n_tok] added to them."""

    def __init__(self, ctx: bt.Context, ids: torch.Tensor, n_tok: int):
        ids = ids.long()
        pairs = torch.bincount(ids[:-1] * n_tok + ids[1:], minlength=n_tok * n_tok).view(n_tok, n_tok).float() + 1e-3
        alone = torch.bincount(ids, minlength=n_tok).float() + 1e-3
        self.hidden = (pairs / pairs.sum(1, keepdim=True)).log().bfloat16()
        self.alone = 0.05 * (alone / alone.sum()).log().bfloat16()
        self.weight = torch.ones(n_tok, device=ids.device)
        # the norm divides a state by its root mean square; the head gives that back on average
        rms = (self.hidden.float() + self.alone.float()).square().mean(1).sqrt()
        self.head = ctx.head_quantize(rms.mean() * torch.eye(n_tok, device=ids.device))


def generate(ctx: bt.Context, model: Bigrams, first: torch.Tensor, n_tokens: int, u: torch.Tensor, **filters):
    """Ids int32 [rows, n_tokens] after the ids ``first`` [rows], drawn by u [n_tokens, rows], and their
    log-probabilities."""
    rows = first.numel()
    ids, logprob = first.clone(), torch.empty(rows, device=first.device)
    draw = torch.empty(rows, device=first.device)
    stream = model.alone.expand(rows, -1).contiguous()

    def step():
        x8, xs, _ = ctx.head_norm(model.hidden[ids.long()], model.weight, stream)
        ctx.head_sample(ctx.head_logits(x8, xs, *model.head), draw, ids=ids, logprob=logprob, **filters)

    draw.copy_(u[0])
    step()   # what a first call sets up is set up outside the graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(first)
    out, logprobs = [], []
    for t in range(n_tokens):
        draw.copy_(u[t])
        graph.replay()
        out.append(ids.clone())
        logprobs.append(logprob.clone())
    torch.cuda.synchronize()
    ctx.head_check()   # a replayed product reports nothing by itself
    return torch.stack(out, 1), torch.stack(logprobs, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--corpus", help="a text file (default: the generator's tiny corpus)")
    ap.add_argument("--merges", type=int, default=256)
    ap.add_argument("--rows", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    if a.corpus:
        with open(a.corpus, "rb") as f:
            text = torch.frombuffer(bytearray(f.read()), dtype=torch.uint8)
    else:
        import synth
        text = torch.from_numpy(synth.corpus("tiny").copy())
    ctx = bt.Context()
    text = text.cuda()
    merges, _ = ctx.train(ctx.pretokenize(text), a.merges, final=False)
    trie = ctx.trie_build(*bt.vocab_from_merges(merges))
    ids, _ = ctx.encode(trie, text)
    model = Bigrams(ctx, ids, trie.n_tok)
    u = torch.rand(a.tokens, a.rows, generator=torch.Generator().manual_seed(a.seed)).cuda()
    out, logprob = generate(ctx, model, ids[:a.rows].clone(), a.tokens, u, temperature=0.9, top_k=100, top_p=0.95)
    texts = [bytes(ctx.decode(merges, row.contiguous()).cpu().tolist()) for row in out]
    for t, p in zip(texts, logprob.mean(1).tolist()):
        print(f"{p:8.3f}  {t.decode('utf-8', 'replace')!r}")
    return out, logprob, texts, merges


if __name__ == "__main__":
    main()
