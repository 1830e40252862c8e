"""Sampling from more rows than one launch takes: the rows of the second launch and
a short last one, each with its own settings, are the same as in a call by themselves."""
import pytest
import torch

from test_gpu_sample import check, tq

pytestmark = pytest.mark.gpu


def rows_a_launch(V):
    """The number of rows from which on the workspace no longer grows."""
    size = tq().lib().tq_sample_workspace_bytes
    lo, hi = 1, 1 << 12                          # (rows * V stays in the domain)
    assert size(hi, V) == size(2 * hi, V) > size(1, V) > 0
    while lo < hi:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if size(mid, V) == size(1 << 12, V) else (mid + 1, hi)
    return lo


def spread(N, lo, hi, dtype):
    return (lo + (hi - lo) * torch.rand(N, generator=torch.Generator().manual_seed(N))).to(dtype).cuda()


# rows behind the full launches: few tiles, whose bins are apart, and many, which share them
@pytest.mark.parametrize("V,launches,more", [(8193, 1, 1), (8193, 2, 300), (17000, 1, 5),
                                             (17000, 1, 600), (60001, 1, 3), (524289, 1, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_several_launches(V, launches, more, dtype):
    most = rows_a_launch(V)
    N = launches * most + more
    g = torch.Generator(device="cuda").manual_seed(V + N)
    wide = torch.empty((N, V + 9), dtype=dtype, device="cuda")
    for a in range(0, N, 64):
        part = wide[a:a + 64]
        part.copy_(2.5 * torch.randn(part.shape, device="cuda", generator=g))
    x, u = wide[:, 4:V + 4], torch.rand(N, device="cuda", generator=g)
    kw = dict(temperature=spread(N, 0.3, 1.5, torch.float32), top_k=spread(N, -20, 60, torch.int32),
              top_p=spread(N, 0.3, 1.1, torch.float32), min_p=spread(N, -0.1, 0.1, torch.float32))
    kw["temperature"][[1, most + 1 if more > 1 else 2]] = 0.0
    x[3] = -float("inf")
    tokens = tq().sample(x, u, **kw)
    out = torch.full((N, V + 2), 7.0, device="cuda")
    probs = tq().sample_probs(x, **kw, out=out[:, 1:V + 1])
    assert (out[:, 0] == 7).all() and (out[:, V + 1] == 7).all()
    assert tokens[3] == -1 and (probs[3] == 0).all()
    for a in range(0, N, 100):                   # a hundred rows take one launch
        part = slice(a, a + 100)
        own = {k: v[part] for k, v in kw.items()}
        assert torch.equal(tq().sample(x[part], u[part], **own), tokens[part]), a
        assert torch.equal(tq().sample_probs(x[part], **own), probs[part]), a
    at = [0, most - 1, most, N - 1]
    own = {k: v[at].tolist() for k, v in kw.items()}
    own["top_k"] = [int(k) for k in own["top_k"]]
    got, _ = check(x[at], u[at].tolist(), **own)
    assert torch.equal(got, tokens[at])


def test_one_row_for_several_launches():
    """Row stride 0: every launch begins at the same logits."""
    V = 9000
    N = rows_a_launch(V) + 40
    x = 2.5 * torch.randn((1, V), generator=torch.Generator().manual_seed(3)).cuda()
    p = spread(N, 0.05, 1.0, torch.float32)
    probs = tq().sample_probs(x.expand(N, V), top_p=p)
    for a in range(0, N, 200):
        part = p[a:a + 200]
        assert torch.equal(tq().sample_probs(x.expand(part.shape[0], V), top_p=part),
                           probs[a:a + 200]), a
