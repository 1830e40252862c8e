"""Bounds of pages, the choice of pages, and attention over them.

Bounds and choices are whole numbers of steps that both sides take in fp32 or
exactly, so they are equal; attention has decode_ref's bound."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from decode_ref import DTYPES, attention, attention_bound

pytestmark = pytest.mark.gpu


def tq():
    import block_quantized_matmul_repack_amd as m
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    def __init__(self, kind, B, width, page, H, D, lens, seed=0, spare=2):
        self.kind, self.page, self.H, self.D, self.lens = kind, page, H, D, lens
        self.ctype = tq().Q8_0 if kind == "q8_0" else tq().Q4_0
        g = torch.Generator().manual_seed(seed)
        per = [-(-n // page) for n in lens]
        self.n_pages = sum(per) + spare
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        slots = self.n_pages * page
        # pages differ, and some channels are loud
        k = torch.randn((slots, H, D), generator=g) + 2 * torch.randn(
            (self.n_pages, H, D), generator=g).repeat_interleave(page, 0)
        k *= 1 + 6 * (torch.rand(D, generator=g) > 0.9)
        v = torch.randn((slots, H, D), generator=g)
        n = tq().cache_bytes(self.ctype, self.n_pages, page, H, D)
        self.kc, self.vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "kv")
        all_slots = torch.arange(slots, dtype=torch.int32, device="cuda")
        tq().cache_write(self.ctype, k.bfloat16().cuda(), v.bfloat16().cuda(), self.kc, self.vc,
                         all_slots, page)
        self.k, self.v = (t.double().cpu() for t in
                          tq().cache_read(self.ctype, self.kc, self.vc, all_slots, H, D, page))
        self.codes = torch.full((self.n_pages, H, D // 32, 2, 32), 99, dtype=torch.int8, device="cuda")
        self.scales = torch.full((self.n_pages, H, D // 32), 9.0, dtype=torch.float16, device="cuda")

    def bounds(self, begin, end, max_new=None, table=None):
        tq().cache_bounds(self.ctype, self.kc, (self.table if table is None else table).cuda(),
                          dev(begin), dev(end), self.H, self.D, self.page, self.codes, self.scales,
                          max_new=max_new)

    def page_keys(self, e, h):
        return self.k[e * self.page:(e + 1) * self.page, h].numpy()

    def check_bounds(self, begin, end):
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        want_c, want_s = np.full_like(codes, 99), np.full_like(scales, 9.0)
        for b in range(len(begin)):
            lo, hi = max(begin[b], 0), min(end[b], self.table.shape[1] * self.page)
            for j in range(lo // self.page, -(-hi // self.page)) if lo < hi else ():
                e = int(self.table[b, j])
                if not 0 <= e < self.n_pages:
                    continue
                for h in range(self.H):
                    c, s = ref.bounds(self.page_keys(e, h), min(hi - j * self.page, self.page))
                    want_c[e, h], want_s[e, h] = c, s
        assert (scales.view(np.int16) == want_s.view(np.int16)).all()
        assert (codes == want_c).all()


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_bounds(kind, D, page):
    lens = [page, 3 * page + 5, 1, 0, 2 * page - 1]
    c = Cache(kind, 5, 6, page, 3, D, lens, seed=D + page)
    begin = [0, page + 1, 0, 0, 2 * page - 2]
    c.bounds(begin, lens)
    c.check_bounds(begin, lens)


def test_bounds_leave_the_rest_alone():
    """Pages outside the ranges, entries that name no page, ranges that are
    empty, backwards, or past the table; and max_new, which only bounds the work."""
    c = Cache("q8_0", 6, 5, 32, 2, 64, [160, 100, 70, 64, 33, 90], seed=5)
    c.table[1, 1] = -1
    c.table[2, 0] = c.n_pages
    c.table[5, 2] = 2 ** 31 - 1
    begin, end = [40, 0, 0, 64, 50, -7], [4000, 100, 70, 64, 20, 90]
    c.bounds(begin, end, max_new=128)
    c.check_bounds(begin, end)
    before = c.codes.clone()
    c.bounds(begin, end, max_new=0)
    assert torch.equal(before, c.codes)


def test_bounds_grow_with_the_page():
    """A page filled token by token has the bounds of what it holds."""
    c = Cache("q8_0", 1, 2, 16, 1, 64, [32])
    for n in range(1, 33):
        c.bounds([n - 1], [n], max_new=1)
    c.check_bounds([0], [32])


def test_bounds_of_zeros():
    c = Cache("q4_0", 1, 1, 16, 2, 64, [16])
    c.kc.zero_()                                 # scale 0: all keys are 0
    c.bounds([0], [16])
    e = int(c.table[0, 0])
    assert (c.codes[e] == 0).all() and (c.scales[e] == 0).all()


def queries(c, nodes, G, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 77)
    return torch.randn((sum(nodes), c.H * G, c.D), generator=g).to(DTYPES[dtype]).cuda()


def starts_of(nodes):
    out = [0]
    for n in nodes:
        out.append(out[-1] + n)
    return out


def check_select(c, q, ctx, nodes, keep, first=1, last=1, **kw):
    starts = starts_of(nodes)
    tables, ctx_out = tq().select_pages(q, c.codes, c.scales, c.table.cuda(), dev(ctx), dev(starts),
                                        c.page, keep, first=first, last=last, **kw)
    codes, scales = c.codes.cpu().numpy().astype(np.float64), c.scales.cpu().numpy()
    G, qf = q.shape[1] // c.H, q.float().cpu().numpy()
    for b, n in enumerate(nodes):
        n = min(n, kw.get("max_nodes") or n)
        want, want_ctx = ref.select(qf[starts[b]:starts[b] + n], codes, scales, c.table[b].tolist(),
                                    c.n_pages, ctx[b], n, c.page, first, last, keep, G,
                                    tables.shape[2])
        assert (tables[b].cpu().numpy() == want).all(), b
        assert ctx_out[b].item() == want_ctx
    return tables, ctx_out


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [1, 3, 8, 17])
def test_select(D, dtype, G):
    page, nodes = 16, [1, 1, 4, 2]
    ctx = [700, 33, 511, 0]
    c = Cache("q8_0", 4, 50, page, 2, D, [a + n for a, n in zip(ctx, nodes)], seed=D + G)
    c.bounds([0] * 4, c.lens)
    q = queries(c, nodes, G, dtype)
    check_select(c, q, ctx, nodes, 7)
    check_select(c, q, ctx, nodes, 7, max_nodes=4, max_ctx=700)


@pytest.mark.parametrize("first,last,keep", [(0, 0, 0), (0, 0, 1), (0, 0, 5), (3, 2, 0), (1, 0, 6),
                                             (0, 4, 3), (50, 1, 2), (1, 50, 2), (2, 2, 500)])
def test_select_budgets(first, last, keep):
    ctx, nodes = [640, 639, 20, 5, 641], [1, 1, 1, 1, 3]
    c = Cache("q4_0", 5, 41, 16, 2, 64, [a + n for a, n in zip(ctx, nodes)], seed=4)
    c.bounds([0] * 5, c.lens)
    check_select(c, queries(c, nodes, 4, "bf16"), ctx, nodes, keep, first, last)


@pytest.mark.parametrize("pages", [1030, 2500])
def test_select_from_many_pages(pages):
    ctx, nodes = [pages * 16 + 3], [2]
    c = Cache("q4_0", 1, pages + 7, 16, 1, 64, [ctx[0] + 2], seed=6)
    c.bounds([0], c.lens)
    q = queries(c, nodes, 5, "bf16")
    for keep in (1, 100, pages - 3, pages):
        check_select(c, q, ctx, nodes, keep)


@pytest.mark.parametrize("pages,heads", [(8300, 1), (60, 2)])
def test_select_from_tables_wider_than_a_workgroup_holds(pages, heads):
    """More than 8192 entries a row: scored and chosen in two launches."""
    ctx, nodes = [pages * 16 - 5, 100], [3, 1]
    c = Cache("q4_0", 2, 8320, 16, heads, 64, [ctx[0] + 3, 101], seed=pages)
    c.bounds([0, 0], c.lens)
    q = queries(c, nodes, 3, "fp16")
    for keep in (1, 40):
        check_select(c, q, ctx, nodes, keep)
        check_select(c, q, ctx, nodes, keep, max_nodes=3, max_ctx=64)    # a bound too small


@pytest.mark.parametrize("G", [4, 17])
def test_select_reads_queries_wherever_they_are(G):
    """Any token and head strides, and rows that begin on an odd element."""
    ctx, nodes = [700, 30], [2, 3]
    c = Cache("q8_0", 2, 50, 16, 2, 96, [702, 33], seed=G)
    c.bounds([0, 0], c.lens)
    q = queries(c, nodes, G, "bf16")
    want = check_select(c, q, ctx, nodes, 6)
    heads = 2 * G
    wide = torch.full((5, heads, 2 * 96 + 3), float("nan"), dtype=q.dtype, device="cuda")
    turned = torch.full((heads, 5, 96), float("nan"), dtype=q.dtype, device="cuda")
    odd = torch.full((5 * heads * 96 + 1,), float("nan"), dtype=q.dtype, device="cuda")
    for view in (wide[:, :, 1:97], turned.transpose(0, 1), odd[1:].view(5, heads, 96)):
        view.copy_(q)
        got = check_select(c, view, ctx, nodes, 6)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    # one query row for all
    one = q[:1, :1].expand(5, heads, 96)
    check_select(c, one, ctx, nodes, 6)


@pytest.mark.parametrize("nodes", [1, 40])
def test_select_with_a_bound_too_small(nodes):
    """max_ctx shapes the launch: the pages past it are scored all the same."""
    ctx = [1000 * 16 + 7]
    c = Cache("q8_0", 1, 1100, 16, 2, 64, [ctx[0] + nodes], seed=12)
    c.bounds([0], c.lens)
    q = queries(c, [nodes], 4, "bf16")
    for most in (0, 300, ctx[0]):
        check_select(c, q, ctx, [nodes], 9, max_nodes=nodes, max_ctx=most)


def test_select_takes_the_earlier_of_equal_pages():
    """Equal scores, zero scores, queries of zeros, and pages that are not there."""
    ctx, nodes = [320, 320], [1, 1]
    c = Cache("q8_0", 2, 22, 16, 2, 64, [321, 321], seed=8)
    c.bounds([0, 0], c.lens)
    c.codes[:] = c.codes[0].clone()
    c.scales[:] = c.scales[0].clone()
    q = queries(c, nodes, 2, "bf16")
    check_select(c, q, ctx, nodes, 5)
    check_select(c, torch.zeros_like(q), ctx, nodes, 5)
    c.table[0, [3, 4, 9]] = torch.tensor([-1, c.n_pages, 2 ** 31 - 1], dtype=torch.int32)
    check_select(c, q, ctx, nodes, 16)
    check_select(c, q, ctx, nodes, 5)


def test_select_with_queries_that_are_no_numbers():
    ctx, nodes = [400], [3]
    c = Cache("q8_0", 1, 30, 16, 1, 64, [403], seed=9)
    c.bounds([0], c.lens)
    q = queries(c, nodes, 2, "bf16")
    q[0, 0, 5], q[1, 1, 40], q[2, 0, 3] = float("nan"), float("inf"), -float("inf")
    q[0, 1] *= 1e-35
    check_select(c, q, ctx, nodes, 6)


def test_select_sequences_without_tokens():
    """Lengths past the table and sequences of no new tokens stay inside."""
    c = Cache("q8_0", 3, 10, 16, 2, 64, [160, 160, 160], seed=3)
    c.bounds([0] * 3, c.lens)
    q = queries(c, [1, 0, 1], 2, "bf16")
    tables, ctx = tq().select_pages(q, c.codes, c.scales, c.table.cuda(), dev([5000, 90, 159]),
                                    dev([0, 1, 1, 2]), 16, 3)
    t = tables.cpu()
    for b in range(3):
        rows = set(c.table[b].tolist())
        assert all(int(e) in rows or int(e) == -1 for e in t[b].flatten())
    assert ctx.tolist()[2] == 159 - 16 * 4


def trees(nodes, seed):
    rng = np.random.default_rng(seed)
    see = []
    for n in nodes:
        m = np.zeros((n, n), bool)
        for i in range(n):
            if i:
                m[i] = m[rng.integers(0, i)]
            m[i, i] = True
        see.append(m)
    return see


def mask_words(see):
    words = max((len(m) + 31) // 32 for m in see)
    rows = []
    for m in see:
        for r in m:
            v = sum(1 << i for i, x in enumerate(r) if x)
            rows.append([((v >> 32 * w) & 0xFFFFFFFF) - ((1 << 32) if (v >> (32 * w + 31)) & 1 else 0)
                         for w in range(words)])
    return dev(rows)


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("D,G,dtype", [(64, 1, "bf16"), (96, 4, "fp16"), (128, 4, "bf16"),
                                       (256, 8, "fp16"), (128, 16, "bf16")])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_over_selected_pages(kind, D, G, dtype, tree):
    nodes = [7, 1, 40, 3] if tree else [1, 1, 1, 1]
    ctx = [500, 15, 333, 64]
    c = Cache(kind, 4, 40, 16, 2, D, [a + n for a, n in zip(ctx, nodes)], seed=D + G)
    c.bounds([0] * 4, c.lens)
    q = queries(c, nodes, G, dtype)
    see = trees(nodes, D)
    mask = mask_words(see) if tree else None
    kw = dict(max_nodes=max(nodes), max_ctx=max(ctx))
    tables, ctx_out = check_select(c, q, ctx, nodes, 5, **kw)
    starts = starts_of(nodes)
    out = tq().tree_attention(c.ctype, q, c.kc, c.vc, tables, ctx_out, dev(starts), c.H, c.page,
                              mask=mask, **kw)
    qd = q.double().cpu()
    for b, n in enumerate(nodes):
        cx = ctx_out[b].item()
        for h in range(c.H):
            pages = tables[b, h].cpu().long()
            slots = (pages[:, None] * c.page + torch.arange(c.page)).flatten()[:cx + n]
            k, v = c.k[slots, h:h + 1], c.v[slots, h:h + 1]
            sees = torch.ones((n, cx + n), dtype=torch.bool)
            sees[:, cx:] = torch.from_numpy(see[b])
            rows = slice(starts[b], starts[b + 1])
            o, mag, span = attention(qd[rows, h * G:(h + 1) * G], k, v, sees, D ** -0.5)
            tol = attention_bound(o, mag, span, cx + n, DTYPES[dtype], v.abs().sum(0)[None])
            got = out[rows, h * G:(h + 1) * G].double().cpu()
            assert ((got - o).abs() <= tol).all(), (b, h)


def test_one_table_for_each_head_is_the_shared_one():
    """The same pages for every head: the same numbers as with one table."""
    ctx, nodes = [900, 61], [1, 1]
    c = Cache("q8_0", 2, 60, 16, 4, 128, [901, 62], seed=2)
    q = queries(c, nodes, 4, "bf16")
    args = (dev(ctx), dev([0, 1, 2]), 4, 16)
    t = c.table.cuda()
    want = tq().tree_attention(c.ctype, q, c.kc, c.vc, t, *args)
    heads = t[:, None].expand(2, 4, 60)
    assert torch.equal(tq().tree_attention(c.ctype, q, c.kc, c.vc, heads, *args), want)
    assert torch.equal(tq().tree_attention(c.ctype, q, c.kc, c.vc, heads.contiguous(), *args), want)
    # all pages kept: select gives the same table, and the same numbers
    c.bounds([0, 0], c.lens)
    tables, ctx_out = tq().select_pages(q, c.codes, c.scales, t, args[0], args[1], 16, 60)
    assert ctx_out.tolist() == ctx
    assert torch.equal(tq().tree_attention(c.ctype, q, c.kc, c.vc, tables, ctx_out, *args[1:]), want)


def test_refusals():
    c = Cache("q8_0", 2, 4, 16, 2, 64, [33, 20])
    q = queries(c, [1, 1], 2, "bf16")
    t, ctx, starts = c.table.cuda(), dev([32, 19]), dev([0, 1, 2])
    good = dict(q=q, codes=c.codes, scales=c.scales, page_table=t, ctx_lens=ctx, starts=starts,
                page_size=16, keep=2)
    tq().select_pages(**good)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(codes=c.codes[..., :16]),
                dict(codes=c.codes.float()), dict(scales=c.scales[:1]), dict(page_table=t.long()),
                dict(page_table=t[None].expand(2, 2, 4)), dict(starts=starts[:2]), dict(keep=-1),
                dict(page_size=24), dict(first=-1), dict(max_nodes=0), dict(q=q[..., :32])):
        with pytest.raises(tq().TiledqError):
            tq().select_pages(**{**good, **bad})
    good = dict(ctype=c.ctype, k_cache=c.kc, page_table=t, begin=ctx, end=ctx, kv_heads=2, D=64,
                page_size=16, codes=c.codes, scales=c.scales)
    for bad in (dict(ctype=tq().Q4_1), dict(k_cache=c.kc[:-1]), dict(begin=ctx[:1]), dict(kv_heads=4),
                dict(D=96), dict(codes=c.codes[1:], scales=c.scales[1:]), dict(page_table=t.cpu()),
                dict(max_new=-1)):
        with pytest.raises(tq().TiledqError):
            tq().cache_bounds(**{**good, **bad})
    with pytest.raises(tq().TiledqError):
        tq().tree_attention(c.ctype, q, c.kc, c.vc, t[:, None].expand(2, 3, 4), ctx, starts, 2, 16)
