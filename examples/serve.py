"""Continuous batching of a small random transformer on the library's operators:
requests of unlike prompts share steps, pages are handed out and taken back on the
GPU (plan_step, release_pages), the norms around each block write the next
product's int8 activations (residual_norm), attention reads the pages whose bounds
promise the most (cache_bounds, select_pages, tree_attention), and each request
samples with settings of its own (sample).  Weights are random, so the text means
nothing; the calls, their order and their buffers are those of a serving loop.  The
host looks at the sampled tokens alone.

    python examples/serve.py [requests] [new tokens of each]
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_quantized_matmul_repack_amd as tq  # noqa: E402
from examples.speculative_decode import (D, HEADS, HIDDEN, KV_HEADS, LAYERS, PAGE, VOCAB,  # noqa: E402
                                         Model)

BATCH, PAGES, WIDTH = 4, 64, 24                  # requests at a time, pages, pages of one
CHUNK = 48                                       # rows of a step
KEEP = 4                                         # pages read beside the first and the newest


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    """Where each request's pages are, and the bounds of what they hold."""

    def __init__(self):
        self.lens, self.owned = int32([0] * BATCH), int32([0] * BATCH)
        self.table = torch.full((BATCH, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free, self.count = int32(list(range(PAGES))), int32([PAGES])
        n = tq.cache_bytes(tq.Q8_0, PAGES, PAGE, KV_HEADS, D)
        self.layers = []
        for _ in range(LAYERS):
            codes = torch.zeros((PAGES, KV_HEADS, D // 32, 2, 32), dtype=torch.int8, device="cuda")
            scales = torch.zeros((PAGES, KV_HEADS, D // 32), dtype=torch.float16, device="cuda")
            self.layers.append([torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "kv"]
                               + [codes, scales])


def forward(m, s, tokens, new, most):
    """Logits after each request's last new token.  tokens int32 [CHUNK]: the new
    tokens, request by request; new int32 [BATCH]: how many of each."""
    begin = s.lens
    starts, pos, slots, s.lens, s.owned, s.count = tq.plan_step(
        s.lens, new, s.owned, s.table, s.free, s.count, PAGE, CHUNK)
    x = m.embed[tokens.long()]
    norm, gate = m.ones, m.gate
    x, act = tq.residual_norm(torch.zeros_like(x), x, norm, quantize=True)
    for layer, (kc, vc, codes, scales) in zip(m.layers, s.layers):
        qkv = tq.matmul(*layer["qkv"].args, *act).bfloat16()
        q = qkv[:, :HEADS * D].unflatten(1, (HEADS, D))
        k, v = qkv[:, HEADS * D:].unflatten(1, (2, KV_HEADS, D)).unbind(1)
        q, k = tq.qk_norm_rope(q, k, pos, m.freq, m.norm, m.norm)
        tq.cache_write(tq.Q8_0, k, v, kc, vc, slots, PAGE)
        tq.cache_bounds(tq.Q8_0, kc, s.table, begin, s.lens, KV_HEADS, D, PAGE, codes, scales,
                        max_new=most)
        tables, ctx = tq.select_pages(q, codes, scales, s.table, begin, starts, PAGE, KEEP,
                                      max_nodes=most)
        o = torch.zeros_like(q)                  # rows of no request stay zeros
        tq.tree_attention(tq.Q8_0, q, kc, vc, tables, ctx, starts, KV_HEADS, PAGE, max_nodes=most,
                          out=o)
        x, act = tq.residual_norm(layer["out"](o.flatten(1)), x, norm, post_weight=norm, gate=gate,
                                  quantize=True)
        y = layer["down"](torch.nn.functional.silu(tq.matmul(*layer["up"].args, *act)))
        x, act = tq.residual_norm(y, x, norm, post_weight=norm, gate=gate, quantize=True)
    last = (starts[1:] - 1).clamp(min=0).long()
    return tq.matmul(*m.head.args, *(a[last] for a in act))


def serve(requests=9, new_tokens=24, quiet=False):
    """The texts of random prompts, each with sampling settings of its own; and how
    many steps they took."""
    m, s = Model(), State()
    m.ones = torch.ones(HIDDEN, device="cuda")
    m.gate = torch.full((1,), 0.1, device="cuda")
    rng = np.random.default_rng(3)
    waiting = [(i, rng.integers(0, VOCAB, int(rng.integers(1, 200))).tolist())
               for i in range(requests)]
    temp = [0.0 if i % 3 == 0 else 0.5 + 0.1 * i for i in range(requests)]
    texts, running, steps = {}, [None] * BATCH, 0
    draws = torch.Generator(device="cuda").manual_seed(5)
    done = int32([0] * BATCH)
    while waiting or any(running):
        for b in range(BATCH):                   # a free place takes the next request
            if running[b] is None and waiting:
                i, prompt = waiting.pop(0)
                running[b], texts[i] = [i, prompt], []
        room, new, rows = CHUNK, [], []
        for r in running:                        # single tokens, and prompts in chunks
            n = min(len(r[1]), room) if r else 0
            rows += r[1][:n] if r else []
            new.append(n)
            room -= n
        tokens = int32(rows + [0] * room)
        logits = forward(m, s, tokens, int32(new), max(new))
        set_ = [temp[r[0]] if r else 1.0 for r in running]
        drawn = tq.sample(logits, torch.rand(BATCH, device="cuda", generator=draws),
                          temperature=torch.tensor(set_, device="cuda"),
                          top_k=int32([40] * BATCH),
                          top_p=torch.full((BATCH,), 0.95, device="cuda")).tolist()
        steps += 1
        ended = [0] * BATCH
        for b, r in enumerate(running):
            if r is None or new[b] == 0:
                continue
            r[1] = r[1][new[b]:]
            if r[1]:
                continue                         # more of its prompt to come
            texts[r[0]].append(drawn[b])
            r[1] = [drawn[b]]
            if len(texts[r[0]]) == new_tokens:
                ended[b], running[b] = 1, None
        if any(ended):
            done = int32(ended)
            s.owned, s.count = tq.release_pages(done, s.owned, s.table, s.free, s.count)
            s.lens = s.lens * (1 - done)
        if not quiet:
            print(f"step {steps}: {CHUNK - room} rows, {int(s.count)} pages free, "
                  f"requests {[r[0] if r else None for r in running]}")
    return [texts[i] for i in range(requests)], steps, s


if __name__ == "__main__":
    args = [int(a) for a in sys.argv[1:]]
    out, took, _ = serve(*args[:2])
    for i, text in enumerate(out):
        print(i, text)
    print(f"{sum(map(len, out))} tokens in {took} steps")
