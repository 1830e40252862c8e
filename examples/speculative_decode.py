"""Greedy speculative decoding of a small random transformer, end to end on the
library's operators: block-quantized weights (matmul_x), per-head norm and
rotation (qk_norm_rope), a Q8_0 cache in pages (cache_write), attention of a
tree of drafted tokens over it (tree_attention) and their verification
(verify_draft).  Drafts are looked up: what followed the last token when it
came before.  Weights are random, so the text means nothing; the calls, their
order and their buffers are those of a serving loop.

    python examples/speculative_decode.py [new tokens] [drafted tokens a step]
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_quantized_matmul_repack_amd as tq  # noqa: E402
import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, D, FFN, VOCAB, LAYERS = 256, 8, 2, 64, 512, 997, 2
PAGE = 16


class Weight:
    """A Q4_0 or Q8_0 matrix as tiles."""

    def __init__(self, qtype, K, N, seed):
        w = synth.Workload("w", qtype, K, N, 1, "uniform" if qtype == synth.Q4_0 else "absnormal",
                           seed=seed)
        flat = torch.from_numpy(synth.make_inputs(w).flat).cuda()
        self.args = (qtype, tq.repack_tiles(qtype, flat, K, N), K, N)

    def __call__(self, x):
        return tq.matmul_x(*self.args, x)


def rms(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self):
        g = torch.Generator().manual_seed(0)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=g).cuda()
        self.layers = [{
            "qkv": Weight(synth.Q4_0, HIDDEN, (HEADS + 2 * KV_HEADS) * D, 10 * i),
            "out": Weight(synth.Q4_0, HEADS * D, HIDDEN, 10 * i + 1),
            "up": Weight(synth.Q4_0, HIDDEN, FFN, 10 * i + 2),
            "down": Weight(synth.Q4_0, FFN, HIDDEN, 10 * i + 3)} for i in range(LAYERS)]
        self.head = Weight(synth.Q8_0, HIDDEN, VOCAB, 99)
        self.freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).float().cuda()
        self.norm = torch.ones(D, dtype=torch.bfloat16, device="cuda")


class Sequence:
    """One sequence's pages in every layer's cache."""

    def __init__(self, most):
        self.pages = -(-most // PAGE)
        n = tq.cache_bytes(tq.Q8_0, self.pages, PAGE, KV_HEADS, D)
        self.caches = [[torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "kv"]
                       for _ in range(LAYERS)]
        # any order of pages will do
        self.table = torch.from_numpy(np.random.default_rng(1).permutation(self.pages)
                                      .astype(np.int32))[None].cuda()

    def slots(self, positions):
        p = torch.as_tensor(positions, device="cuda")
        return (self.table[0, p // PAGE] * PAGE + p % PAGE).int()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def forward(m, s, ctx, tokens, depth, mask):
    """Logits of new tokens, whose keys and values go to positions ctx, ctx +
    1, ...; depth: their distance from the last cached one."""
    T = len(tokens)
    x = m.embed[torch.tensor(tokens, device="cuda")]
    pos, slots = int32([ctx + d for d in depth]), s.slots(range(ctx, ctx + T))
    lens, starts = int32([ctx]), int32([0, T])
    for layer, (kc, vc) in zip(m.layers, s.caches):
        qkv = layer["qkv"](rms(x)).bfloat16()
        q = qkv[:, :HEADS * D].unflatten(1, (HEADS, D))
        k, v = qkv[:, HEADS * D:].unflatten(1, (2, KV_HEADS, D)).unbind(1)
        q, k = tq.qk_norm_rope(q, k, pos, m.freq, m.norm, m.norm)
        tq.cache_write(tq.Q8_0, k, v, kc, vc, slots, PAGE)
        o = tq.tree_attention(tq.Q8_0, q, kc, vc, s.table, lens, starts, KV_HEADS, PAGE,
                              max_nodes=T, max_ctx=ctx, mask=mask)
        x = x + 0.1 * rms(layer["out"](o.flatten(1)))
        x = x + 0.1 * rms(layer["down"](torch.nn.functional.silu(layer["up"](rms(x)))))
    return m.head(rms(x))


def look_up(text, drafted):
    """A tree of drafted tokens: parents and tokens of its nodes, node 0 the
    last token of the text.  What followed the last token's latest two
    occurrences, as two branches from the root."""
    parents, tokens = [-1], [text[-1]]
    seen = [i for i in range(len(text) - 1) if text[i] == text[-1]][::-1][:2]
    for n, i in enumerate(seen):
        at = 0
        for t in text[i + 1:i + 1 + (drafted if n == 0 else 1)]:
            if len(tokens) > drafted:
                break
            parents.append(at)
            tokens.append(t)
            at = len(tokens) - 1
    return parents, tokens


def generate(new_tokens=64, prompt=32, drafted=4, quiet=False):
    """Text after a random prompt, and how many steps it took."""
    m, s = Model(), Sequence(prompt + new_tokens + 2 * drafted + 4)
    rng = np.random.default_rng(7)
    draws = torch.Generator(device="cuda").manual_seed(5)
    text = rng.integers(0, VOCAB, prompt).tolist()
    logits = forward(m, s, 0, text, range(prompt), None)          # the prompt: one chain
    ctx, steps = prompt, 0
    text.append(int(logits[-1].argmax()))
    while len(text) < prompt + new_tokens:
        parents, tokens = look_up(text, drafted)
        T = len(tokens)
        depth, rows = [0] * T, [1] * T
        for i in range(1, T):
            depth[i] = depth[parents[i]] + 1
            rows[i] = rows[parents[i]] | 1 << i                   # itself and its ancestors
        logits = forward(m, s, ctx, tokens, depth, int32(rows)[:, None])
        # greedy: all of the target's probability on its likeliest token
        target = torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()
        count, out, path = tq.verify_draft(
            target, int32(tokens), int32([0, T]), torch.rand(T, device="cuda", generator=draws),
            torch.rand(1, device="cuda", generator=draws), parents=int32(parents), max_nodes=T)
        n = int(count)
        text += out[0, :n + 1].tolist()
        # the accepted nodes' keys and values move up behind the root's
        took = path[0, :n].tolist()
        if took != list(range(1, n + 1)):
            src, dst = s.slots([ctx + i for i in took]), s.slots(range(ctx + 1, ctx + 1 + n))
            for kc, vc in s.caches:
                k, v = tq.cache_read(tq.Q8_0, kc, vc, src, KV_HEADS, D, PAGE)
                tq.cache_write(tq.Q8_0, k, v, kc, vc, dst, PAGE)  # the same blocks again
        ctx, steps = ctx + 1 + n, steps + 1
        if not quiet:
            print(f"step {steps}: {T - 1} drafted, {n} accepted, next {text[-1]}")
    return text[prompt:], steps


if __name__ == "__main__":
    args = [int(a) for a in sys.argv[1:]]
    out, steps = generate(*(args[:1] or [64]), drafted=args[1] if len(args) > 1 else 4)
    print(f"{len(out)} tokens in {steps} steps: {out}")
