"""tq_tree_attention with bounds on the new tokens that are far above what a
sequence has, starts that are not in order, and more workgroups than one grid
dimension holds."""
import numpy as np
import pytest
import torch

import decode_ref as ref
from test_gpu_attention import Setup, ctype, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,D", [("q8_0", 64), ("q4_0", 128)])
def test_many_sequences_with_the_default_bound(tq, kind, D):
    """512 sequences of 256 tokens, with max_nodes left at all rows of q: the
    launch goes by the rows there are."""
    n, B, Hkv, G = 256, 512, 8, 4
    g = torch.Generator().manual_seed(4)
    P, per = 64, 5
    ct = ctype(tq, kind)
    pages = per
    nb = tq.cache_bytes(ct, pages, P, Hkv, D)
    kc, vc = (torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(per * P, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((per * P, Hkv, D), generator=g).bfloat16().cuda() for _ in range(2))
    tq.cache_write(ct, k, v, kc, vc, slots, P)
    table = torch.arange(per, dtype=torch.int32, device="cuda").repeat(B, 1)   # shared pages
    q = torch.randn((n, Hkv * G, D), generator=g).bfloat16().cuda().repeat(B, 1, 1)
    ctx = torch.full((B,), 17, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    out = tq.tree_attention(ct, q, kc, vc, table, ctx, starts, Hkv, P)
    one = tq.tree_attention(ct, q[:n], kc, vc, table[:1], ctx[:1], starts[:2], Hkv, P)
    assert bool((out.view(B, n, Hkv * G, D) == out[:n]).all())
    assert float((out[:n].float() - one.float()).abs().max()) < 0.02   # another cut of the sums
    kr, vr = (x.cpu().double() for x in tq.cache_read(ct, kc, vc, slots[:17 + n], Hkv, D, P))
    see = torch.ones((n, 17 + n), dtype=torch.bool).tril(17)
    o, mag, span = ref.attention(q[:n].cpu(), kr, vr, see, D ** -0.5)
    tol = ref.attention_bound(o, mag, span, 17 + n, q.dtype, vr.abs().sum(0).repeat_interleave(G, 0))
    assert bool(((out[:n].cpu().double() - o).abs() <= tol).all())


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 4), (128, 6, 2), (256, 4, 2)])
def test_ragged_sequences_with_the_default_bound(tq, D, Hq, Hkv):
    """Empty, short and long sequences among many, starts not at row 0, and
    rows behind the last sequence: each token once, in its place."""
    rng = np.random.default_rng(D)
    seqs = [(int(rng.integers(0, 90)), int(rng.choice([0, 1, 1, 2, 3, 17, 60])))
            for _ in range(700)]
    seqs[5], seqs[699] = (3, 300), (20, 0)
    s = Setup(tq, "q8_0", seqs, Hq, Hkv, D, 16, seed=D)
    head, tail = 7, 9
    T = s.T
    q = torch.cat([torch.zeros_like(s.q[:head]), s.q, torch.zeros_like(s.q[:tail])])
    out = torch.full_like(q, 7.0)
    s.run(q=q, starts=s.starts + head, out=out, max_nodes=q.shape[0])
    assert bool((out[:head] == 7).all()) and bool((out[head + T:] == 7).all())
    s.check(out[head:head + T])
    tight = s.run()
    assert float((out[head:head + T].float() - tight.float()).abs().max()) < 0.05


def test_starts_out_of_order(tq):
    """Starts that go back or leave the rows: every access stays inside, rows
    of the sequences before them are right."""
    seqs = [(10, 1)] * 300
    s = Setup(tq, "q8_0", seqs, 16, 16, 64, 16, seed=3)
    starts = s.starts.clone()
    starts[200:] = torch.tensor([5, -3, 2, -2 ** 31] * 26, dtype=torch.int32)[:101]
    out = torch.zeros_like(s.q)
    s.run(starts=starts, out=out, max_nodes=s.T)
    s.run(starts=torch.full_like(starts, 2 ** 31 - 1), out=out, max_nodes=s.T)
    s.run(starts=torch.full_like(starts, -1), out=out, max_nodes=s.T)
    want = s.run()
    assert torch.equal(out[6:150], want[6:150])


def test_more_workgroups_than_one_dimension_holds(tq):
    """65535 sequences of one token, 272 key heads: 17.8 million units of 256
    threads."""
    B, H, D, P = 65535, 272, 64, 16
    g = torch.Generator().manual_seed(8)
    nb = tq.cache_bytes(tq.Q8_0, 1, P, H, D)
    kc, vc = (torch.zeros(nb, dtype=torch.uint8, device="cuda") for _ in range(2))
    k, v = (torch.randn((P, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    slots = torch.arange(P, dtype=torch.int32, device="cuda")
    tq.cache_write(tq.Q8_0, k, v, kc, vc, slots, P)
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    ctx = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    one = torch.randn((1, H, D), generator=g).bfloat16().cuda()
    q = one.expand(B, H, D)
    out = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    tq.tree_attention(tq.Q8_0, q, kc, vc, table, ctx, starts, H, P, max_nodes=1, max_ctx=3, out=out)
    kr, vr = (x.cpu().double() for x in tq.cache_read(tq.Q8_0, kc, vc, slots[:4], H, D, P))
    o, mag, span = ref.attention(one.cpu(), kr, vr, torch.ones((1, 4), dtype=torch.bool), D ** -0.5)
    tol = ref.attention_bound(o, mag, span, 4, q.dtype, vr.abs().sum(0))
    assert bool(((out[0].cpu().double() - o[0]).abs() <= tol[0]).all())
    assert bool((out == out[:1]).all())
