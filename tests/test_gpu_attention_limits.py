"""tq_tree_attention where scores leave the ordinary range."""
import pytest
import torch

import decode_ref as ref
from test_gpu_attention import KINDS, Setup, pack, tq, tree_masks  # noqa: F401

pytestmark = pytest.mark.gpu


def alike(s, masks=None):
    """Outputs where all keys are equal: the plain mean of the values seen.
    Every probability is the same number, so only its rounding (2^-11), the
    values' (2^-11), the sums' and the output's count."""
    out, row = [], 0
    for b, (c, n) in enumerate(s.seqs):
        see = s.see(b, None if masks is None else masks[b]).double()
        w = (see / see.sum(1, keepdim=True)).repeat_interleave(s.Hq, 0)
        v = s.v[b].repeat_interleave(s.Hq // s.Hkv, 1)                # [L, Hq, D]
        o, mag = (torch.stack([w.view(n, s.Hq, -1)[:, h] @ x[:, h] for h in range(s.Hq)], 1)
                  for x in (v, v.abs()))
        h = ref.half_step(s.q.dtype)
        tol = h * o.abs() + (2 * 2.0 ** -11 + (c + n + 64) * 2.0 ** -24) * mag * 1.01 + 2.0 ** -24
        out.append((o, tol))
    return torch.cat([o for o, _ in out]), torch.cat([t for _, t in out])


def check_alike(s, out, masks=None):
    want, tol = alike(s, masks)
    out = out.cpu().double()
    assert bool(torch.isfinite(out).all())
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() - tol).max())
    assert float((want.abs() > 4 * tol).double().mean()) > 0.8      # zeros would not pass


def equal_keys(seqs, Hq, Hkv, D, dt, kind, value, seed=1):
    return lambda tq: Setup(tq, kind, seqs, Hq, Hkv, D, 16, dt, seed=seed,
                            k=lambda b, L: torch.full((L, Hkv, D), value))


# codes of the largest magnitude with a scale that is a power of two: exact in
# both types and in fp16
FULL = {"q8_0": 127.0, "q4_0": -128.0}
SHAPES = [([(70, 1), (300, 1)], 4, 2), ([(150, 5), (0, 9)], 8, 2), ([(90, 40)], 4, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("seqs,Hq,Hkv", SHAPES)
def test_scores_of_many_millions(tq, kind, dt, sign, seqs, Hq, Hkv):
    """Scores of 10^9 and more whose fp32 neighbours are over a hundred apart:
    equal scores still share the weight equally, and one larger score takes
    it all."""
    D = 128
    s = equal_keys(seqs, Hq, Hkv, D, dt, kind, sign * FULL[kind])(tq)
    s.q = (3e3 + 1e4 * torch.rand(s.q.shape, generator=torch.Generator().manual_seed(2))).to(
        s.q.dtype).cuda()
    for scale in (3.1, 77.7):
        check_alike(s, s.run(scale=scale))

    def one_loud(b, L):
        k = torch.zeros((L, Hkv, D))
        k[L // 3] = abs(FULL[kind]) if kind == "q8_0" else FULL[kind]
        return k
    s = Setup(tq, kind, seqs, Hq, Hkv, D, 16, dt, seed=3, k=one_loud)
    s.q = (float(FULL[kind] > 0) * 2 - 1) * (3e3 + torch.zeros_like(s.q))
    out, row = s.run(scale=50.0).cpu().double(), 0
    for b, (c, n) in enumerate(seqs):
        j = (c + n) // 3
        for i in range(n):
            if j >= c + i + 1:
                continue                         # that token does not see it
            v = s.v[b][j].repeat_interleave(Hq // Hkv, 0)
            tol = (2 * 2.0 ** -11 + ref.half_step(s.q.dtype)) * v.abs() + 2.0 ** -24
            assert bool(((out[row + i] - v).abs() <= tol).all())
        row += n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,Hq,Hkv", SHAPES)
def test_scores_far_below_zero(tq, kind, seqs, Hq, Hkv):
    """All scores of a row near -10^32: it sees keys all the same."""
    s = equal_keys(seqs, Hq, Hkv, 128, "bf16", kind, FULL[kind] / 8)(tq)
    s.q = torch.full_like(s.q, -2.0 ** 100 if FULL[kind] > 0 else 2.0 ** 100)
    check_alike(s, s.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,Hq,Hkv", SHAPES)
def test_scores_below_fp32(tq, kind, seqs, Hq, Hkv):
    """Scores that are zero in fp32, beside keys that a mask hides."""
    s = equal_keys(seqs, Hq, Hkv, 128, "bf16", kind, FULL[kind])(tq)
    s.q = torch.full_like(s.q, 2.0 ** -120)
    masks = tree_masks(seqs, 6)
    check_alike(s, s.run(scale=1e-12, mask=pack(masks)), masks)


@pytest.mark.parametrize("n", [4, 40])
def test_infinite_query_leaves_the_others_alone(tq, n):
    """A row whose scores are infinite shares a wave with ordinary ones: those
    keep their bits."""
    s = Setup(tq, "q8_0", [(3000, n)], 4, 2, 128, 32, seed=4)
    want = s.run()
    q = s.q.clone()
    q[1, 2] = float("inf")
    q[n - 1, 1, 3] = -float("inf")
    out = s.run(q=q)
    keep = torch.ones((n, 4), dtype=torch.bool)
    keep[1, 2] = keep[n - 1, 1] = False
    assert torch.equal(out[keep.cuda()], want[keep.cuda()])
