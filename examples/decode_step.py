"""Steps of drafted tokens through one decoder layer and the head, on random weights: the products, the
cache, the attention and the verification as a serving loop calls them.

A batch of sequences shares a prompt. Each step takes every sequence's last token and its drafts
(at most 16 tokens in all, what one pn_gemv takes), and
  1. q, k and v of all tokens by one grouped product over PN weights,
  2. k and v quantised into the microscaled cache,
  3. attention over the shared prompt and each sequence's own tokens, from the cache,
  4. the output product, and the row-scaled E4M3 head, which gives the target's logits,
  5. the drafts verified against the target's probabilities; the own lengths grow by the accepted
     drafts and the token after them, so what the refused drafts left in the cache is written over.

  python3 examples/decode_step.py [--steps 4] [--format mxfp4]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_quantized_weight_pn3t_amd as pn  # noqa: E402

HIDDEN, HEADS, GROUP, DIM, VOCAB, PAGE = 1280, 2, 4, 128, 4001, 32


class Layer:
    """Random weights of one layer and a head, and the buffers of a step of B sequences of Q tokens."""

    def __init__(self, B, Q, format, prompt, steps, seed=0, dev="cuda:0"):
        self.B, self.Q, self.dev = B, Q, torch.device(dev)
        g = self.gen = torch.Generator(device=self.dev)
        g.manual_seed(seed)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=self.dev)
        self.wq = self.weights(pn.PN3T, HEADS * GROUP * DIM, HIDDEN)
        self.wk = self.weights(pn.PN4T, HEADS * DIM, HIDDEN)
        self.wv = self.weights(pn.PN4T, HEADS * DIM, HIDDEN)
        self.wo = self.weights(pn.PN4T, HIDDEN, HEADS * GROUP * DIM)
        # E4M3 words of magnitude 0.25 .. 3.75, one bf16 multiplier a row
        self.head = torch.randint(0x28, 0x48, (VOCAB, HIDDEN), generator=g, device=self.dev, dtype=torch.uint8)
        self.head += 128 * torch.randint(0, 2, (VOCAB, HIDDEN), generator=g, device=self.dev, dtype=torch.uint8)
        self.head_scale = torch.full((VOCAB,), 0.04, device=self.dev).bfloat16()
        # the shared prompt's pages first, then each sequence's own
        self.prompt = prompt
        own = -(-(1 + steps * Q) // PAGE)
        self.prefix_table = torch.arange(-(-prompt // PAGE), dtype=torch.int32, device=self.dev)
        self.table = (self.prefix_table.numel() + torch.arange(B * own, dtype=torch.int32, device=self.dev)).view(B, own)
        pages = self.prefix_table.numel() + B * own
        self.cache = pn.Cache(format, HEADS, DIM, PAGE, torch.empty(
            pages * pn.cache_page_bytes(format, HEADS, DIM, PAGE), dtype=torch.uint8, device=self.dev))
        self.own = torch.zeros(B, dtype=torch.int32, device=self.dev)  # own tokens in the cache

    def weights(self, type_, rows, K):
        w = torch.randn(rows, K, generator=self.gen, device=self.dev) / K ** 0.5
        W = torch.empty(rows, pn.row_bytes(type_, K), dtype=torch.uint8, device=self.dev)
        pn.quantize_rows(type_, w, W)
        return type_, W, rows

    def project(self, x, parts):
        """One grouped product of the parts' weights with x [M, K]."""
        ys = [torch.empty(x.shape[0], rows, device=self.dev) for _, _, rows in parts]
        pn.gemv_group([(t, W, rows, y) for (t, W, rows), y in zip(parts, ys)], x.shape[1], x)
        return ys

    def fill_prompt(self, tokens):
        """The prompt's keys and values into the shared pages, 16 tokens a product."""
        for at in range(0, len(tokens), 16):
            x = self.embed[tokens[at:at + 16]]
            k, v = self.project(x, (self.wk, self.wv))
            place = torch.arange(at, at + len(x), device=self.dev)
            slots = self.prefix_table.long()[place // PAGE] * PAGE + place % PAGE
            pn.cache_write(self.cache, k.view(-1, HEADS, DIM), v.view(-1, HEADS, DIM), slots)

    def logits(self, tokens):
        """The target's logits [B, Q, VOCAB] at the last token and the drafts, tokens [B, Q]; their keys and
        values enter the cache at the own lengths, which are left to the verification to move."""
        B, Q = self.B, self.Q
        x = self.embed[tokens.view(-1)]
        q, k, v = self.project(x, (self.wq, self.wk, self.wv))
        place = self.own[:, None].long() + torch.arange(Q, device=self.dev)
        slots = self.table.long().gather(1, place // PAGE) * PAGE + place % PAGE
        pn.cache_write(self.cache, k.view(-1, HEADS, DIM), v.view(-1, HEADS, DIM), slots.view(-1))
        query = q.view(B, Q, HEADS * GROUP, DIM)
        out = torch.empty_like(query)
        work = torch.empty(pn.attend_workspace_bytes(self.cache, query, self.table, self.prompt),
                           dtype=torch.uint8, device=self.dev)
        pn.attend(self.cache, query, self.table, self.own + Q, out, workspace=work,
                  prefix_table=self.prefix_table, prefix_len=self.prompt)
        y, = self.project(out.view(B * Q, -1), (self.wo,))
        x = x + y
        logits = torch.empty(B * Q, VOCAB, device=self.dev)
        for at in range(0, B * Q, pn.MAX_TOKENS):  # the head takes up to four tokens a call
            pn.gemv_fp8row(self.head, self.head_scale, VOCAB, HIDDEN, x[at:at + pn.MAX_TOKENS],
                           logits[at:at + pn.MAX_TOKENS])
        return logits.view(B, Q, VOCAB)

    def step(self, last, draft, draft_probs):
        """One step: last int32[B], draft int32[B, Q - 1]. The tokens that stand and how many drafts did."""
        B, K = draft.shape
        p = torch.softmax(self.logits(torch.cat([last[:, None], draft], 1).long()), -1)
        tokens = torch.empty(B, K + 1, dtype=torch.int32, device=self.dev)
        accepted = torch.empty(B, dtype=torch.int32, device=self.dev)
        work = torch.empty(pn.verify_workspace_bytes(B, VOCAB), dtype=torch.uint8, device=self.dev)
        pn.verify(p, draft_probs, draft, torch.rand(B, K, generator=self.gen, device=self.dev),
                  torch.rand(B, generator=self.gen, device=self.dev), tokens, accepted, work)
        self.own += 1 + accepted  # the last token and the drafts that stand
        return tokens, accepted


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--format", choices=("mxfp8", "mxfp4"), default="mxfp8")
    a = ap.parse_args()
    B, K = 4, 3
    layer = Layer(B, K + 1, pn.MXFP8 if a.format == "mxfp8" else pn.MXFP4, prompt=77, steps=a.steps)
    prompt = torch.randint(0, VOCAB, (layer.prompt,), generator=layer.gen, device=layer.dev)
    layer.fill_prompt(prompt)
    last = torch.randint(0, VOCAB, (B,), generator=layer.gen, device=layer.dev, dtype=torch.int32)
    for n in range(a.steps):
        # drafts of a stand-in for a draft model: flat probabilities with one token made likelier
        guess = torch.randn(B, K, VOCAB, generator=layer.gen, device=layer.dev).softmax(-1)
        draft = torch.multinomial(guess.view(B * K, VOCAB), 1, generator=layer.gen).view(B, K).int()
        tokens, accepted = layer.step(last, draft, guess)
        last = tokens.gather(1, accepted[:, None].long())[:, 0]
        print(f"step {n}: accepted {accepted.tolist()}, own tokens {layer.own.tolist()}, next {last.tolist()}",
              flush=True)


if __name__ == "__main__":
    main()
