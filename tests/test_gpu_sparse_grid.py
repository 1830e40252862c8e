"""The choice of pages and attention over them where there are so many heads that
each has a workgroup to itself: from 128 on the choice, from 512 on the attention."""
import numpy as np
import pytest
import torch

from decode_ref import DTYPES, attention, attention_bound
from test_gpu_sparse import Cache, check_select, dev, mask_words, queries, starts_of, tq, trees

pytestmark = pytest.mark.gpu


def ragged(B, most, nodes, seed):
    """Contexts 0 .. most, those at whole pages of 16 among them, and new tokens 1 .. nodes."""
    rng = np.random.default_rng(seed)
    ctx = [int(c) for c in rng.integers(0, most + 1, B)]
    n = [int(c) for c in rng.integers(1, nodes + 1, B)]
    ctx[:6] = [0, 1, 16, 15, most, 160]
    n[5], n[0] = nodes, nodes
    return ctx, n


def check_attention(c, q, ctx, nodes, keep, tree, **kw):
    see = trees(nodes, len(nodes)) if tree else [np.tri(n, dtype=bool) for n in nodes]
    mask = mask_words(see) if tree else None
    tables, ctx_out = check_select(c, q, ctx, nodes, keep, **kw)
    starts = starts_of(nodes)

    def run():
        return tq().tree_attention(c.ctype, q, c.kc, c.vc, tables, ctx_out, dev(starts), c.H, c.page,
                                   mask=mask, out=torch.full_like(q, 5.0), **kw)

    out = run()
    assert torch.equal(run(), out)
    G, D, qd = q.shape[1] // c.H, c.D, q.double().cpu()
    pages, cached = tables.cpu().long(), ctx_out.tolist()
    got = out.double().cpu()
    for b, n in enumerate(nodes):
        for h in range(c.H if n else 0):
            cx = cached[b]
            slots = (pages[b, h][:, None] * c.page + torch.arange(c.page)).flatten()[:cx + n]
            k, v = c.k[slots, h:h + 1], c.v[slots, h:h + 1]
            sees = torch.ones((n, cx + n), dtype=torch.bool)
            sees[:, cx:] = torch.from_numpy(see[b])
            rows, heads = slice(starts[b], starts[b + 1]), slice(h * G, (h + 1) * G)
            o, mag, span = attention(qd[rows, heads], k, v, sees, D ** -0.5)
            tol = attention_bound(o, mag, span, cx + n, q.dtype, v.abs().sum(0)[None])
            assert ((got[rows, heads] - o).abs() <= tol).all(), (b, h)


@pytest.mark.parametrize("kind,D,dtype", [("q8_0", 64, "bf16"), ("q8_0", 128, "fp16"),
                                          ("q4_0", 128, "bf16"), ("q4_0", 96, "fp16")])
@pytest.mark.parametrize("B", [63, 64, 70])
def test_one_token_of_many_sequences(kind, D, dtype, B):
    """504, 512 and 560 heads with tables of their own, on both sides of the rule."""
    ctx, _ = ragged(B, 300, 1, B + D)
    nodes = [1] * B
    c = Cache(kind, B, 20, 16, 8, D, [a + 1 for a in ctx], seed=D + B)
    c.bounds([0] * B, c.lens)
    check_attention(c, queries(c, nodes, 2, dtype), ctx, nodes, 3, False, max_nodes=1, max_ctx=300)


@pytest.mark.parametrize("D,G,dtype", [(64, 4, "bf16"), (128, 4, "fp16"), (256, 1, "bf16")])
@pytest.mark.parametrize("bound", ["tight", "rows"])
def test_trees_of_many_sequences(D, G, dtype, bound):
    """512 heads with up to 20 and 80 query rows; max_nodes as it is, or all rows of q."""
    ctx, nodes = ragged(64, 200, 20, D)
    c = Cache("q8_0", 64, 16, 16, 8, D, [a + n for a, n in zip(ctx, nodes)], seed=D)
    c.bounds([0] * 64, c.lens)
    q = queries(c, nodes, G, dtype)
    kw = dict(max_nodes=20 if bound == "tight" else sum(nodes), max_ctx=200)
    check_attention(c, q, ctx, nodes, 2, True, **kw)


@pytest.mark.parametrize("D,G,nodes", [(64, 4, 40), (128, 5, 33), (256, 4, 20)])
@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
def test_choice_with_more_query_rows_than_a_workgroup_holds(kind, D, G, nodes):
    """128 heads, each chosen for by one workgroup, which takes the query rows 128 (64 with
    256 channels) at a time."""
    ctx, n = ragged(64, 290, nodes, D + G)
    c = Cache(kind, 64, 22, 16, 2, D, [a + b for a, b in zip(ctx, n)], seed=G)
    c.bounds([0] * 64, c.lens)
    q = queries(c, n, G, "bf16")
    check_select(c, q, ctx, n, 4, max_nodes=nodes, max_ctx=290)
    check_select(c, q, ctx, n, 1, first=0, last=0, max_nodes=nodes, max_ctx=0)


def test_sequences_without_tokens_among_many():
    """They keep pages inside their tables, their neighbours' choice and outputs do not
    change, and rows behind the last sequence stay as they were."""
    B, H, G = 80, 8, 2
    ctx, _ = ragged(B, 250, 1, 1)
    none = [3, 17, 79]
    nodes = [0 if b in none else 1 for b in range(B)]
    c = Cache("q8_0", B, 16, 16, H, 64, [a + 1 for a in ctx], seed=5)
    c.bounds([0] * B, c.lens)
    q = queries(c, nodes + [4], G, "bf16")       # four rows of no sequence behind
    table, starts = c.table.cuda(), dev(starts_of(nodes))
    args = (c.codes, c.scales, table, dev(ctx), starts, 16, 3)
    tables, ctx_out = tq().select_pages(q, *args, max_nodes=1, max_ctx=250)
    out = tq().tree_attention(c.ctype, q, c.kc, c.vc, tables, ctx_out, starts, H, 16, max_nodes=1,
                              out=torch.full_like(q, 5.0))
    assert (out[B - 3:] == 5).all() and not (out[:B - 3] == 5).all(-1).any()
    live = [b for b in range(B) if nodes[b]]
    st = dev(starts_of([1] * len(live)))
    t2, c2 = tq().select_pages(q[:len(live)], c.codes, c.scales, table[live], dev([ctx[b] for b in live]),
                               st, 16, 3, max_nodes=1, max_ctx=250)
    assert torch.equal(t2, tables[live]) and torch.equal(c2, ctx_out[live])
    o2 = tq().tree_attention(c.ctype, q[:len(live)], c.kc, c.vc, t2, c2, st, H, 16, max_nodes=1)
    assert torch.equal(o2, out[:len(live)])
    for b in none:
        own = set(c.table[b].tolist())
        assert all(int(e) in own or int(e) == -1 for e in tables[b].cpu().flatten())
