"""The example's loop with drafts that are known to be right or wrong: drafted
tokens are accepted on a second branch, their cache entries move up, and the
text and the cache are those of decoding token by token."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

NEW, PROMPT = 40, 40


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import speculative_decode
    finally:
        sys.path.pop(0)
    return speculative_decode


def run(example, monkeypatch, look_up):
    """Text, steps, the sequence with its cache, and how often entries moved."""
    kept, moves = [], []

    class Sequence(example.Sequence):
        def __init__(self, most):
            super().__init__(most)
            kept.append(self)

    read = example.tq.cache_read
    with monkeypatch.context() as m:
        m.setattr(example, "Sequence", Sequence)
        m.setattr(example, "look_up", look_up)
        m.setattr(example.tq, "cache_read", lambda *a, **k: moves.append(1) or read(*a, **k))
        text, steps = example.generate(new_tokens=NEW, prompt=PROMPT, drafted=5, quiet=True)
    return text[:NEW], steps, kept[0], len(moves) // example.LAYERS


def cached(example, s, n):
    """Keys and values of positions 0 .. n - 1 in every layer."""
    out = []
    for kc, vc in s.caches:
        k, v = example.tq.cache_read(example.tq.Q8_0, kc, vc, s.slots(range(n)), example.KV_HEADS,
                                     example.D, example.PAGE)
        out += [k.flatten(1), v.flatten(1)]
    return torch.stack(out)


def forced(plain, shape):
    """Drafts from the text that is to come: shape(right) gives (parent,
    token) of nodes 1, 2, ...; right(i) is the token i places on."""
    def look_up(text, drafted):
        at = len(text) - PROMPT
        right = lambda i: plain[at + i] if at + i < len(plain) else 1       # noqa: E731
        nodes = shape(right)
        return [-1] + [p for p, _ in nodes], [text[-1]] + [t for _, t in nodes]
    return look_up


def wrong(example, t):
    return (t + 1) % example.VOCAB


@pytest.mark.parametrize("case", ["chain", "second branch", "deep in the second branch", "wrong"])
def test_speculation_changes_nothing(example, monkeypatch, case):
    only_root = lambda text, drafted: ([-1], [text[-1]])                    # noqa: E731
    plain, steps, alone, moved = run(example, monkeypatch, only_root)
    assert steps == NEW - 1 and moved == 0
    bad = lambda t: wrong(example, t)                                       # noqa: E731
    shape = {
        "chain": lambda r: [(0, r(0)), (1, r(1)), (2, r(2)), (3, bad(r(3)))],
        "second branch": lambda r: [(0, bad(r(0))), (0, r(0)), (1, r(1)), (2, r(1))],
        "deep in the second branch": lambda r: [(0, r(0)), (1, bad(r(1))), (1, r(1)),
                                                (2, r(2)), (3, r(2)), (5, bad(r(3)))],
        "wrong": lambda r: [(0, bad(r(0))), (1, r(1)), (0, bad(bad(r(0))))],
    }[case]
    most = {"chain": 3, "second branch": 2, "deep in the second branch": 3, "wrong": 0}[case]
    text, steps, s, moved = run(example, monkeypatch, forced(plain, shape))
    assert text == plain
    assert steps == -(-(NEW - 1) // (most + 1))
    # the last step's drafts may run past the known text
    assert moved >= steps - 1 if "second" in case else moved <= 1
    n = PROMPT + NEW - 1
    a, b = cached(example, alone, n), cached(example, s, n)
    # the same tokens at the same places: equal but for the products' rounding;
    # another token's keys and values would be as far off as they are long
    far = (a - b).norm(dim=-1) / a.norm(dim=-1)
    assert float(far.max()) < 0.25, float(far.max())
