"""Sampling and its distributions against whole-number weights on the host.

Tokens are whole numbers and equal: the weights of both sides differ by a unit
of 2^-45 at most here and there (exp in fp64), so a draw that falls between
them has a chance of about V * 2^-45.  A probability is a quotient of two such sums
rounded once to fp32: 2^-24 relative, and 2^-40 for the units."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from decode_ref import DTYPES

pytestmark = pytest.mark.gpu
INF = float("inf")


def tq():
    import block_quantized_matmul_repack_amd as m
    return m


def settings(N, **kw):
    out = {}
    for k, v in kw.items():
        if v is not None:
            t = torch.int32 if k == "top_k" else torch.float32
            out[k] = torch.tensor(v if isinstance(v, list) else [v] * N, dtype=t, device="cuda")
    return out


def pick(v, r):
    return v[r] if isinstance(v, list) else v


def check(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    N, V = logits.shape
    kw = settings(N, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    tokens = tq().sample(logits, torch.tensor(u, dtype=torch.float32, device="cuda"), **kw)
    probs = tq().sample_probs(logits, **kw).double().cpu().numpy()
    x = logits.double().cpu().numpy()
    u = np.float32(u)
    for r in range(N):
        t = pick(temperature, r)
        w = ref.kept(x[r], 1.0 if t is None else float(np.float32(t)), pick(top_k, r),
                     pick(top_p, r), pick(min_p, r))
        assert tokens[r].item() == ref.sample(w, u[r]), r
        p = w / w.sum() if w.any() else w.astype(float)
        assert ((p > 0) == (probs[r] > 0)).all(), (r, np.nonzero((p > 0) != (probs[r] > 0)))
        assert (abs(probs[r] - p) <= 2.0 ** -24 * p * 1.01 + 2.0 ** -40).all(), r
    return tokens, probs


def rows(N, V, dtype="fp32", scale=2.5, seed=0):
    g = torch.Generator().manual_seed(V * 31 + N + seed)
    return (scale * torch.randn((N, V), generator=g)).to(DTYPES[dtype]).cuda(), \
        torch.rand(N, generator=g).tolist()


@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 255, 1000, 1024, 1025, 8191, 8193, 50257,
                               128001, 262144])
def test_vocabularies(V):
    x, u = rows(4, V)
    check(x, u, [0.8, 1.0, 0.5, 1.7], [0, 40, 3, 1], [0.95, 1.0, 0.5, 0.9], [0.0, 0.02, 0.0, 0.1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [777, 20001])
@pytest.mark.parametrize("which", range(8))
def test_settings(dtype, V, which):
    x, u = rows(7, V, dtype, seed=which)
    kw = [dict(), dict(temperature=0.7), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05),
          dict(top_k=200, top_p=0.8), dict(temperature=1.5, top_p=0.99, min_p=0.01),
          dict(temperature=0.3, top_k=20, top_p=0.95, min_p=0.2)][which]
    check(x, u, **kw)


@pytest.mark.parametrize("V", [5, 300, 4097, 40000])
def test_ties(V):
    """Equal logits: the lower index first, whatever cuts them."""
    x = torch.zeros((10, V), device="cuda")
    x[5:] = torch.randint(0, 3, (5, V), generator=torch.Generator().manual_seed(V)).cuda().float()
    u = [0.0, 0.3, 0.5, 0.9, 0.999] * 2
    check(x, u, top_k=[1, 3, V // 2, V, V + 5] * 2)
    check(x, u, top_p=[0.0, 0.001, 0.5, 0.9, 1.0] * 2)
    check(x, u, top_k=[0, 2, V // 2, V - 1, V] * 2, top_p=[0.1, 0.6, 0.5, 0.3, 0.999] * 2)
    check(x, u, temperature=[2.0, 0.5, 0.01, 100.0, 1e-3] * 2, min_p=[0.1, 0.5, 1.0, 0.2, 7.0] * 2)


def test_few_values_over_a_long_row():
    """bf16 logits of few values: thousands of ties at the cut."""
    x, u = rows(6, 128001, "bf16", 0.05)
    check(x, u, top_k=[1000, 0, 20000, 100, 0, 70000], top_p=[1.0, 0.5, 0.7, 0.3, 0.01, 0.999])


def test_values_close_together_over_a_long_row():
    """fp32 logits within a thousandth: many different keys at the cut."""
    x, u = rows(5, 128001, "fp32", 1e-3)
    check(x, u, top_k=[1000, 0, 20000, 0, 77777], top_p=[1.0, 0.5, 0.7, 0.01, 0.999])
    check(x + 1000.0, u, [1e-3, 1.0, 0.1, 1e-2, 1e-4], [9, 0, 5000, 0, 600], [1.0, 0.6, 0.9, 0.3, 0.5])


@pytest.mark.parametrize("V", [70, 9000])
def test_borders(V):
    """Numbers that are none, masks, empty rows, and settings at their ends."""
    lo = torch.finfo(torch.float32).min
    x, _ = rows(12, V)
    x[0] = -INF                                  # nothing
    x[1] = float("nan")
    x[2, 3:] = -INF                              # three
    x[3, ::2] = float("nan")
    x[4, 7] = x[4, 11] = INF                     # two share the row
    x[5] = lo                                    # masked all alike
    x[6, 5:] = lo
    x[7, :] = -INF
    x[7, V - 1] = -1e30                          # one, far down
    x[8] = 3e38
    x[8, 1] = -3e38
    x[9] *= 1e-30
    u = [0.0, 0.5, 0.99999994, 0.25] * 3
    tokens, probs = check(x, u)
    assert tokens[:2].tolist() == [-1, -1] and (probs[:2] == 0).all()
    assert tokens[7].item() == V - 1
    check(x, u, 0.6, 2, 0.9, 0.3)
    check(x, u, [0.0, -1.0, INF, 1e-30, 1e30, 0.1] * 2, [0, -5, 1, 2, 2 ** 31 - 1, 4] * 2,
          [0.0, -1.0, 2.0, 1e-9, 0.999999, 0.5] * 2, [0.0, -1.0, 2.0, 1e-9, 1.0, 0.5] * 2)


def test_greedy_takes_the_first_of_the_largest():
    x = torch.zeros((3, 9001), device="cuda")
    x[0, [4000, 8999]] = 1.0
    x[1, 9000] = 1.0
    tokens, probs = check(x, [0.999, 0.5, 0.999], temperature=0.0)
    assert tokens.tolist() == [4000, 9000, 0] and probs[0, 4000] == 1.0


def test_numbers_outside_the_unit_interval():
    """u at 1 and past it: the last token that is kept; below 0, NaN: the first."""
    x, _ = rows(1, 5000)
    x = x.repeat(4, 1)
    tokens, _ = check(x[:1], [0.0], top_k=30)
    keep = tq().sample_probs(x[:1], top_k=settings(1, top_k=30)["top_k"])[0].nonzero()[:, 0]
    got = tq().sample(x, torch.tensor([1.0, 7.0, -1.0, float("nan")], device="cuda"),
                      top_k=settings(4, top_k=30)["top_k"])
    assert got.tolist() == [keep[-1], keep[-1], keep[0], keep[0]] and tokens[0] == keep[0]


def test_strides_and_rows():
    """Rows of a wider tensor at odd places; probabilities beside others."""
    x, u = rows(9, 1001, "bf16")
    wide = torch.full((9, 1100), 50.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 13:1014] = x
    ud = torch.tensor(u, device="cuda")
    kw = settings(9, top_k=30, top_p=0.9)
    assert torch.equal(tq().sample(wide[:, 13:1014], ud, **kw), tq().sample(x, ud, **kw))
    out = torch.full((9, 1010), 3.0, device="cuda")
    tq().sample_probs(wide[:, 13:1014], **kw, out=out[:, 4:1005])
    assert torch.equal(out[:, 4:1005], tq().sample_probs(x, **kw))
    assert (out[:, :4] == 3).all() and (out[:, 1005:] == 3).all()
    assert tq().sample(x[:0], ud).shape == (0,)


def test_many_rows():
    x, u = rows(3000, 130)
    check(x, u, top_k=20, top_p=0.8)


def test_draws_follow_the_distribution():
    """Each token as often as evenly spread numbers say: off by two at most (the
    ends of its stretch)."""
    x, _ = rows(1, 40)
    n = 4096
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = tq().sample(x.expand(n, 40), u, top_p=settings(n, top_p=0.9)["top_p"])
    p = tq().sample_probs(x, top_p=settings(1, top_p=0.9)["top_p"])[0]
    assert ((torch.bincount(got.long(), minlength=40) - n * p).abs() <= 2).all()


def test_refusals():
    x, u = rows(3, 50)
    u = torch.tensor(u, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=x.t()), dict(logits=x.double()), dict(uniforms=u[:2]),
                dict(uniforms=u.double()), dict(top_k=u), dict(top_p=i), dict(min_p=u[:1]),
                dict(temperature=u.cpu()), dict(logits=x[0])):
        with pytest.raises(tq().TiledqError):
            tq().sample(**{**dict(logits=x, uniforms=u), **bad})
    with pytest.raises(tq().TiledqError):
        tq().sample_probs(x, out=x[:2])


@pytest.mark.parametrize("scale", [0.0, 1e-3, 0.02, 0.1, 0.5])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nearly_even_rows(scale, dtype):
    """Thousands to all of a long row's elements near the cut."""
    x, u = rows(5, 60001, dtype, scale)
    check(x, u, [1.0, 2.0, 0.5, 3.0, 1.0], [0, 0, 30000, 7, 0], [0.95, 0.5, 0.9, 1.0, 0.02])


def test_more_rows_than_a_launch_takes():
    """Hundreds of rows of several tiles, their settings each their own."""
    x, u = rows(700, 17000)
    k = [(i * 7) % 50 for i in range(700)]
    p = [0.5 + 0.0007 * i for i in range(700)]
    check(x, u, [0.5 + 0.001 * i for i in range(700)], k, p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [524288, 524289, 600001, 1048577])
def test_the_longest_rows(V, dtype):
    """Tiles twice as large, and rows of more tiles than are kept apart."""
    x, u = rows(3, V, dtype)
    x[2, ::3] = -INF
    check(x, u, [0.8, 1.0, 0.0], [0, 40, 3], [0.95, 1.0, 0.5], [0.0, 0.02, 0.1])
    check(x[:2], u[:2], [1.0, 0.6], [100000, 0], [0.5, 0.05])


@pytest.mark.parametrize("V", [3000, 8192, 40000, 530000])
def test_thousands_of_equal_logits_at_the_cut(V):
    """Which of the equal ones are kept, wherever they lie: evenly, all at one end, or
    among others close by."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((6, V), -9.0)
    x[0, torch.randperm(V, generator=g)[:2000]] = 1.0
    x[1, :2000] = 1.0
    x[2, V - 2000:] = 1.0
    x[3] = 1.0 + 2.0 ** -9 * torch.randint(0, 3, (V,), generator=g)
    x[4] = 1.0 + 1e-5 * torch.rand(V, generator=g)
    x[4, ::3] = 1.0
    x[5, :7] = 3.0
    x[5, V - 2500:] = 1.0
    x, u = x.cuda(), [0.0, 0.2, 0.4, 0.6, 0.8, 0.999]
    check(x, u, top_k=[1, 500, 1999, 900, 1500, 2000])
    check(x, u, top_p=[0.3, 0.5, 0.9, 0.2, 0.05, 0.7])
    check(x, u, top_k=[1700, 1500, 1999, 2500, 900, 2000], top_p=[0.3, 0.9, 0.5, 0.99, 0.6, 0.7])
