"""tq_tree_attention on keys whose blocks have powers of two as scales, so that
code * scale is exact in fp16 and a sharp softmax can be held to a bound far
below its outputs; the kernels of four waves in fp16; and long runs of new
tokens."""
import pytest
import torch

import decode_ref as ref
from test_gpu_attention import KINDS, Setup, pack, tq, tree_masks  # noqa: F401

pytestmark = pytest.mark.gpu


def rising_keys(kind, Hkv, D, top):
    """Whole numbers, one of the largest magnitude in every block, times 2^n
    with n rising to `top` along the sequence."""
    def k(b, L):
        g = torch.Generator().manual_seed(100 + b)
        most = 127 if kind == "q8_0" else 8
        low = 127 if kind == "q8_0" else 7
        x = torch.randint(-low, low + 1, (L, Hkv, D // 32, 32), generator=g).float()
        at = torch.randint(0, 32, (L, Hkv, D // 32, 1), generator=g)
        x.scatter_(-1, at, -float(most))
        n = top - 8 + torch.div(9 * torch.arange(L), max(L, 1), rounding_mode="floor")
        return (x * torch.exp2(n.float())[:, None, None, None]).view(L, Hkv, D)
    return k


def bound(s, out, mag, span, keys, vsum):
    """Half a step of the output's type; 2^-11 for each value and, with bf16
    outputs, for each probability (with fp16 outputs two operands hold it: 2^-21);
    a score is a sum of D products in fp32 and three more roundings, each at
    most 2^-24 of sum |q||k|, and moves the weighted mean by twice its error
    at most; sums over the keys; below fp16's normal numbers the absolute
    steps of values and of probabilities times 2^10."""
    h = 2.0 ** -11
    p = h if s.q.dtype is torch.bfloat16 else 2.0 ** -21
    rel = h + p + 2 * (s.D + 8) * 2.0 ** -24 * span + (keys + 64) * 2.0 ** -24
    return ref.half_step(s.q.dtype) * out.abs() + rel * mag * 1.01 + 2.0 ** -25 + 2.0 ** -35 * vsum


def check(s, got, masks=None):
    row, apart, all_ = 0, 0.0, 0
    for b, (c, n) in enumerate(s.seqs):
        if n == 0:
            continue
        see = s.see(b, None if masks is None else masks[b])
        o, mag, span = ref.attention(s.q[row:row + n].cpu(), s.k[b], s.v[b], see, s.D ** -0.5)
        vsum = s.v[b].abs().sum(0).repeat_interleave(s.Hq // s.Hkv, 0)
        tol = bound(s, o, mag, span, c + n, vsum)
        err = (got[row:row + n].cpu().double() - o).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()))
        apart += float((o.abs() > 8 * tol).sum())
        all_ += o.numel()
        row += n
    # zeros, or an output off by an eighth, would not pass
    assert apart > 0.8 * all_, apart / all_


SEQS = [([(2500, 1), (400, 5)], 4, 2), ([(0, 1), (17, 1), (9000, 1)], 8, 2),
        ([(3000, 7)], 6, 2), ([(2000, 20), (333, 17)], 4, 2), ([(1500, 40)], 4, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("seqs,Hq,Hkv", SEQS)
def test_rising_scores(tq, kind, dt, D, seqs, Hq, Hkv):
    """The largest score keeps rising along the keys, to about 100 above the
    others: sums are rescaled again and again, and most weight lies on few keys."""
    s = Setup(tq, kind, seqs, Hq, Hkv, D, 32, dt, seed=D + Hq,
              k=rising_keys(kind, Hkv, D, -2 if kind == "q8_0" else 2))
    check(s, s.run())
    masks = tree_masks(seqs, 5)
    check(s, s.run(mask=pack(masks)), masks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [18, 40])
def test_many_short_trees(tq, kind, dt, D, n):
    """More heads and row blocks than compute units: workgroups of four waves."""
    seqs = [(i * 7 % 90, n - i % 3) for i in range(66)]
    s = Setup(tq, kind, seqs, 8, 4, D, 16, dt, seed=n + D,
              k=rising_keys(kind, 4, D, -3 if kind == "q8_0" else 1))
    masks = tree_masks(seqs, n)
    check(s, s.run(mask=pack(masks)), masks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (256, 1), (64, 20), (96, 40), (128, 34),
                                 (256, 20)])
def test_workgroup_for_each_head(tq, kind, D, n):
    """fp16 with so many heads and row blocks that none is cut."""
    seqs = [(i * 5 % 200, n - i % min(n, 3)) for i in range(130)]
    s = Setup(tq, kind, seqs, 16, 16, D, 16, "fp16", seed=n + D,
              k=rising_keys(kind, 16, D, -3 if kind == "q8_0" else 1))
    check(s, s.run())


@pytest.mark.parametrize("kind,dt,D,Hq,Hkv", [("q8_0", "bf16", 128, 4, 2), ("q4_0", "fp16", 64, 4, 1),
                                              ("q8_0", "fp16", 96, 2, 2), ("q4_0", "bf16", 256, 4, 2)])
@pytest.mark.parametrize("seqs", [[(0, 1100)], [(100, 1500)], [(7, 700), (0, 1), (300, 1025)]])
def test_a_prompt(tq, kind, dt, D, Hq, Hkv, seqs):
    """Chains of a thousand tokens and more, some over keys that were there."""
    s = Setup(tq, kind, seqs, Hq, Hkv, D, 32, dt, seed=D)
    s.check(s.run())
