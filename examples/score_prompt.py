"""A prompt scored in whole, and a token after it, through one decoder layer and the head on random weights: the
norm, the 8-bit products, the keys rotated into the cache, the attention and the log probabilities as a serving
loop calls them.

The prompt's tokens go through the layer together, which the products over PN weights (up to 16 tokens) do
in pieces:
  1. the norm of the embeddings, as 8-bit rows, and q, k and v by one 8-bit product,
  2. q and k rotated by their positions, k and v quantised into the microscaled cache,
  3. attention of every token over itself and those before it, from the cache,
  4. the output product over 8-bit rows, the residual's addition and the next norm in one,
  5. the head by another 8-bit product, and of its logits the log probability of each next token, its
     rank, the entropy and the likeliest tokens.
A decode step is the same with one token.

  python3 examples/score_prompt.py [--tokens 77] [--format mxfp4]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_quantized_weight_pn3t_amd as pn  # noqa: E402

HIDDEN, HEADS, GROUP, DIM, ROT, VOCAB, PAGE, EPS = 1280, 2, 4, 128, 64, 4001, 32, 1e-6


class Layer:
    """Random weights of one layer and a head, 8-bit rows, and a cache of `most` tokens of one sequence."""

    def __init__(self, most, format, seed=0, dev="cuda:0"):
        self.dev = torch.device(dev)
        g = self.gen = torch.Generator(device=self.dev)
        g.manual_seed(seed)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=self.dev)
        self.norms = [1.0 + 0.2 * torch.randn(HIDDEN, generator=g, device=self.dev) for _ in range(2)]
        self.wqkv = self.weights(HEADS * (GROUP + 2) * DIM, HIDDEN)
        self.wo = self.weights(HIDDEN, HEADS * GROUP * DIM)
        self.head = self.weights(VOCAB, HIDDEN)
        angle = torch.arange(most, device=self.dev).double()[:, None] * 10000.0 ** (
            -torch.arange(0, ROT, 2, device=self.dev).double() / ROT)
        self.rotation = torch.cat([angle.cos(), angle.sin()], 1).float()
        pages = -(-most // PAGE)
        self.table = torch.randperm(pages, generator=g, device=self.dev).int()[None]
        self.cache = pn.Cache(format, HEADS, DIM, PAGE, torch.empty(
            pages * pn.cache_page_bytes(format, HEADS, DIM, PAGE), dtype=torch.uint8, device=self.dev))
        self.length = 0  # tokens in the cache

    def weights(self, rows, K):
        return self.rows8(torch.randn(rows, K, generator=self.gen, device=self.dev) / K ** 0.5)

    def rows8(self, x):
        """The rows of x as 8-bit integers and their scales."""
        codes = torch.empty(x.shape, dtype=torch.int8, device=self.dev)
        scales = torch.empty(x.shape[0], device=self.dev)
        pn.int8_quantize_rows(x, codes, scales)
        return codes, scales

    def norm8(self, x, weight, residual=None):
        """8-bit rows of the norm of x + residual, and the sum."""
        codes = torch.empty(x.shape, dtype=torch.int8, device=self.dev)
        scales = torch.empty(x.shape[0], device=self.dev)
        total = None if residual is None else torch.empty_like(x)
        pn.add_norm(x, weight, EPS, codes=codes, scales=scales, residual=residual, sum=total)
        return (codes, scales), total

    def project(self, x, w):
        (a, a_scales), (w, w_scales) = x, w
        out = torch.empty(a.shape[0], w.shape[0], device=self.dev)
        work = torch.empty(pn.gemm_int8_workspace_bytes(a.shape[0], w.shape[0], a.shape[1]), dtype=torch.uint8,
                           device=self.dev)
        pn.gemm_int8(a, a_scales, w, w_scales, out, work)
        return out

    def logits(self, tokens):
        """The logits [T, VOCAB] at tokens [T] after those that are in the cache, which takes them in."""
        T, dev = len(tokens), self.dev
        x = self.embed[tokens]
        y, _ = self.norm8(x, self.norms[0])
        qkv = self.project(y, self.wqkv).view(T, HEADS * (GROUP + 2), DIM)
        q, k, v = qkv.split([HEADS * GROUP, HEADS, HEADS], 1)
        place = torch.arange(self.length, self.length + T, device=dev)
        slots = self.table[0].long()[place // PAGE] * PAGE + place % PAGE
        pn.cache_append(self.cache, k, v, slots, self.rotation, positions=place, q=q, q_out=q)
        self.length += T
        lens = torch.tensor([self.length], dtype=torch.int32, device=dev)
        query = q[None]
        out = torch.empty(query.shape, device=dev)
        work = torch.empty(pn.attend_workspace_bytes(self.cache, query, self.table), dtype=torch.uint8, device=dev)
        pn.attend(self.cache, query, self.table, lens, out, workspace=work)
        o = self.project(self.rows8(out.view(T, -1)), self.wo)
        z, _ = self.norm8(o, self.norms[1], residual=x)
        return self.project(z, self.head)

    def score(self, tokens, top):
        """Of each token after the first: log probability, rank; of each place: entropy, likeliest tokens and their
        log probabilities."""
        logits = self.logits(tokens)
        T, dev = len(tokens), self.dev
        after = torch.full((T,), -1, dtype=torch.int32, device=dev)  # none after the last
        after[:-1] = tokens[1:].int()
        got = dict(logprob=torch.empty(T, device=dev), rank=torch.empty(T, dtype=torch.int32, device=dev),
                   entropy=torch.empty(T, device=dev), top_ids=torch.empty(T, top, dtype=torch.int32, device=dev),
                   top_logprobs=torch.empty(T, top, device=dev))
        work = torch.empty(pn.logprobs_workspace_bytes(T, VOCAB, top), dtype=torch.uint8, device=dev)
        pn.logprobs(logits, after, workspace=work, **got)
        return got


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=77)
    ap.add_argument("--format", choices=("mxfp8", "mxfp4"), default="mxfp8")
    a = ap.parse_args()
    layer = Layer(a.tokens + 4, pn.MXFP8 if a.format == "mxfp8" else pn.MXFP4)
    prompt = torch.randint(0, VOCAB, (a.tokens,), generator=layer.gen, device=layer.dev)
    got = layer.score(prompt, 3)
    print(f"{a.tokens} tokens: log probability {got['logprob'].sum().item():.3f}, mean rank "
          f"{got['rank'][:-1].float().mean().item():.0f}, mean entropy {got['entropy'].mean().item():.3f}", flush=True)
    last = got["top_ids"][-1:, 0].long()
    for n in range(4):
        got = layer.score(last, 3)
        print(f"token {last.item()}: likeliest next {got['top_ids'][0].tolist()}, log probabilities "
              f"{[round(p, 3) for p in got['top_logprobs'][0].tolist()]}", flush=True)
        last = got["top_ids"][:, 0].long()


if __name__ == "__main__":
    main()
