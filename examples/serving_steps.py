"""Serving steps of one attention layer with LoRA adapters, from prompts to checked drafts.

Several sequences share a batch, each with its own adapter. A step takes some new tokens of every
sequence: a chunk of its prompt, or its last token and a few drafted ones behind it. The layer

  1. projects the tokens' activations to queries, keys and values and adds each token's adapter
     (sgmv_lora_delta_ids, one call for q, k and v together);
  2. writes keys and values into the paged cache, quantised (sgmv_kv_write);
  3. attends over the cache (sgmv_kv_attention);
  4. turns outputs into probabilities, and checks the drafts against them (sgmv_verify_drafts).
     Rejected drafts leave the cache by leaving the sequence's length: the next write takes
     their places.

The drafter looks a sequence's last token up in its past and proposes what followed (its drafts are
certain, so it has no probabilities of its own). Weights are random; the point is the calls. Every step,
that of the prompts too, is compared with plain attention in torch, in 64 bits on the CPU, over the values
that the cache holds.

    python examples/serving_steps.py [--cache e4m3|i8|bf16] [--steps 12]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_gemv_amd as sg  # noqa: E402

WIDTH, HEADS, KV_HEADS, DIM, VOCAB = 512, 8, 2, 64, 24
PAGE, RANK, ADAPTERS, DRAFTS = 16, 16, 3, 3
FORMATS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


class Layer:
    def __init__(self, device, seed=0):
        g = torch.Generator().manual_seed(seed)
        bf16 = lambda *s, std: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).to(device)
        n = (HEADS + 2 * KV_HEADS) * DIM
        self.embed = bf16(VOCAB, WIDTH, std=1.0)
        self.qkv = bf16(n, WIDTH, std=WIDTH ** -0.5)
        self.out = bf16(VOCAB, HEADS * DIM, std=0.3)
        self.pool = sg.sgmv_pool_pack(bf16(ADAPTERS, RANK, WIDTH, std=WIDTH ** -0.5),
                                      bf16(ADAPTERS, n, RANK, std=0.3 * RANK ** -0.5),
                                      [RANK] * ADAPTERS, [float(RANK)] * ADAPTERS)

    def project(self, tokens, adapters):
        """Queries, keys and values of the tokens, as views of one projection."""
        x = self.embed[tokens.long()]
        y = x @ self.qkv.T
        seg = sg.sgmv_segments_alloc(x.shape[0], ADAPTERS, 0, x.device)
        sg.sgmv_lora_delta_ids(adapters, x, self.pool, seg, y)
        q, k, v = y.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1)
        return q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM))

    def probabilities(self, attended):
        return torch.softmax((attended.flatten(1) @ self.out.T).float(), 1)


class Sequence:
    def __init__(self, prompt, adapter, pages):
        self.tokens, self.adapter, self.pages = list(prompt), adapter, pages
        self.cached = 0  # tokens whose keys and values are in the cache

    def drafts(self):
        last = self.tokens[-1]
        for i in range(len(self.tokens) - 2, -1, -1):
            if self.tokens[i] == last:
                return self.tokens[i + 1:i + 1 + DRAFTS]
        return []


def step(layer, cache, seqs, new, device):
    """One step: new[b] tokens of sequence b. Returns the outputs and the batch."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    start = [0]
    for n in new:
        start.append(start[-1] + len(n))
    table = torch.full((len(seqs), max(len(s.pages) for s in seqs)), -1, dtype=torch.int32)
    for b, s in enumerate(seqs):
        table[b, :len(s.pages)] = torch.tensor(s.pages)
    lens = [s.cached + len(n) for s, n in zip(seqs, new)]
    batch = sg.sgmv_kv_batch(i32(start), i32(lens), table.to(device), start[-1], max(map(len, new)), max(lens))
    adapters = [s.adapter for s, n in zip(seqs, new) for _ in n]
    q, k, v = layer.project(i32([t for n in new for t in n]), i32(adapters))
    sg.sgmv_kv_write(k, v, batch, cache)
    out, _ = sg.sgmv_kv_attention(q, batch, cache)
    return q, out, batch, lens


def check(q, out, batch, lens, cache):
    """Largest difference of a step's outputs from plain attention over what the cache holds; NaN where
    one is not a number."""
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    k, v = sg.sgmv_kv_read(batch, cache, torch.tensor(start, dtype=torch.int32, device=q.device), start[-1],
                           torch.float32 if cache.dtype != torch.bfloat16 else torch.bfloat16)
    k, v, q64, o64 = (t.double().cpu() for t in (k, v, q, out))
    first, worst = batch.q_start.tolist(), torch.zeros((), dtype=torch.float64)
    for b, n in enumerate(lens):
        rows = first[b + 1] - first[b]
        kb, vb = (t[start[b]:start[b + 1]].repeat_interleave(HEADS // KV_HEADS, 1) for t in (k, v))
        s = torch.einsum("qhd,thd->hqt", q64[first[b]:first[b + 1]], kb) / math.sqrt(DIM)
        pos = torch.arange(n - rows, n)[:, None]
        s = s.masked_fill(torch.arange(n) > pos, -math.inf)
        ref = torch.einsum("hqt,thd->qhd", torch.softmax(s, 2), vb)
        if rows:  # (Python's max would lose NaN)
            worst = torch.maximum(worst, (ref - o64[first[b]:first[b + 1]]).abs().max())
    return worst


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--cache", choices=sorted(FORMATS), default="e4m3")
    parser.add_argument("--steps", type=int, default=12)
    args = parser.parse_args(argv)
    if args.steps < 1:
        parser.error("--steps must be at least 1")
    device = torch.device("cuda:0")
    layer = Layer(device)
    g = torch.Generator().manual_seed(1)
    free = torch.randperm(64, generator=g).tolist()
    cache = sg.sgmv_kv_init(64, PAGE, KV_HEADS, DIM, FORMATS[args.cache], device)
    seqs = []
    for b, n in enumerate((40, 7, 90)):
        prompt = torch.randint(0, 12, (n,), generator=g).tolist()
        seqs.append(Sequence(prompt, b % ADAPTERS if b != 1 else -1, [free.pop() for _ in range(16)]))
    # the prompts; the last token of each waits for its first step with drafts
    worst = check(*step(layer, cache, seqs, [s.tokens[:-1] for s in seqs], device), cache)
    for s in seqs:
        s.cached = len(s.tokens) - 1
    taken = 0
    for _ in range(args.steps):
        drafts = [s.drafts() for s in seqs]
        new = [[s.tokens[-1]] + d for s, d in zip(seqs, drafts)]
        q, out, batch, lens = step(layer, cache, seqs, new, device)
        worst = torch.maximum(worst, check(q, out, batch, lens, cache))
        target = layer.probabilities(out)
        flat = [t for d in drafts for t in d]
        first = [0]
        for d in drafts:
            first.append(first[-1] + len(d))
        tokens, accepted = sg.sgmv_verify_drafts(
            target, None, torch.tensor(flat, dtype=torch.int32, device=device),
            torch.tensor(first, dtype=torch.int32, device=device),
            torch.rand(len(flat), generator=g).to(device), torch.rand(len(seqs), generator=g).to(device),
            max(map(len, drafts)))
        for s, row, n in zip(seqs, tokens.tolist(), accepted.tolist()):
            s.cached += 1 + n  # the token before the drafts, and those that were taken
            s.tokens += row[:n + 1]
            taken += n
    for b, s in enumerate(seqs):
        print(f"sequence {b} (adapter {s.adapter}): {len(s.tokens)} tokens, last {s.tokens[-8:]}")
    print(f"{taken} drafts taken in {args.steps} steps; outputs off by at most {float(worst):.2e}")
    # output and probabilities are rounded to bf16, over values below 8
    return 0 if worst <= 2 * 2.0 ** -8 * 8 else 1


if __name__ == "__main__":
    sys.exit(main())
