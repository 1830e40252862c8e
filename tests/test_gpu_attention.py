"""tq_tree_attention against its fp64 definition over the values the cache
holds; the bound is decode_ref.attention_bound."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu
KINDS = ("q8_0", "q4_0")


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    tq.lib()
    return tq


def ctype(tq, kind):
    return {"q8_0": tq.Q8_0, "q4_0": tq.Q4_0}[kind]


class Setup:
    """Sequences of (cached, new) tokens in a cache whose other bytes are
    0xFF: scales that are NaN wherever no token was written."""

    def __init__(self, tq, kind, seqs, Hq, Hkv, D, P, dt="bf16", seed=0, k=None, v=None,
                 spare=2, loud=1.0):
        g = torch.Generator().manual_seed(seed)
        self.tq, self.kind, self.seqs = tq, kind, seqs
        self.Hq, self.Hkv, self.D, self.P = Hq, Hkv, D, P
        per = [-(-(c + n) // P) for c, n in seqs]
        self.pages = sum(per) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(max(per), 1)
        table = np.full((len(seqs), width), -1, np.int32)
        n = tq.cache_bytes(ctype(tq, kind), self.pages, P, Hkv, D)
        self.kc = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.vc = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.k, self.v = [], []
        dtype = ref.DTYPES[dt]
        for b, (c, nn) in enumerate(seqs):
            for i in range(per[b]):
                table[b, i] = order.pop()
            L = c + nn
            kk = (torch.randn((L, Hkv, D), generator=g) if k is None else k(b, L)).to(dtype)
            vv = (torch.randn((L, Hkv, D), generator=g) if v is None else v(b, L)).to(dtype)
            pos = np.arange(L)
            slots = torch.from_numpy(table[b, pos // P] * P + pos % P).int().cuda()
            if L:
                tq.cache_write(ctype(tq, kind), kk.cuda(), vv.cuda(), self.kc, self.vc, slots, P)
                a, e = tq.cache_read(ctype(tq, kind), self.kc, self.vc, slots, Hkv, D, P)
            else:
                a = e = torch.zeros((0, Hkv, D))
            self.k.append(a.cpu().double())
            self.v.append(e.cpu().double())
        self.table = torch.from_numpy(table).cuda()
        self.T = sum(n for _, n in seqs)
        self.q = (loud * torch.randn((self.T, Hq, D), generator=g)).to(dtype).cuda()
        self.ctx = torch.tensor([c for c, _ in seqs], dtype=torch.int32).cuda()
        self.starts = torch.tensor(np.concatenate(([0], np.cumsum([n for _, n in seqs]))),
                                   dtype=torch.int32).cuda()

    def run(self, mask=None, **kw):
        kw.setdefault("max_nodes", max(max(n for _, n in self.seqs), 1))
        kw.setdefault("max_ctx", max(c for c, _ in self.seqs))
        return self.tq.tree_attention(ctype(self.tq, self.kind), kw.pop("q", self.q), self.kc,
                                      self.vc, kw.pop("table", self.table), self.ctx,
                                      kw.pop("starts", self.starts), self.Hkv, self.P, mask=mask,
                                      **kw)

    def see(self, b, mask_rows=None, dead=()):
        """[T, L] bool; dead: positions on unmapped pages."""
        c, n = self.seqs[b]
        s = torch.ones((n, c + n), dtype=torch.bool)
        s[:, c:] = torch.tril(torch.ones(n, n, dtype=torch.bool)) if mask_rows is None \
            else mask_rows
        s[:, list(dead)] = False
        return s

    def check(self, out, masks=None, scale=None, dead=None):
        scale = self.D ** -0.5 if scale is None else scale
        row = 0
        for b, (c, n) in enumerate(self.seqs):
            if n == 0:
                continue
            see = self.see(b, None if masks is None else masks[b],
                           () if dead is None else dead[b])
            o, mag, span = ref.attention(self.q[row:row + n].cpu(), self.k[b], self.v[b], see,
                                         scale)
            vsum = self.v[b].abs().sum(0).repeat_interleave(self.Hq // self.Hkv, 0)
            tol = ref.attention_bound(o, mag, span, c + n, self.q.dtype, vsum)
            got = out[row:row + n].cpu().double()
            bad = ~((got - o).abs() <= tol)
            assert not bool(bad.any()), (b, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                         float((got - o).abs().max()))
            row += n


def seeded(seed, shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def pack(masks):
    """Bool rows [T, n] of each sequence -> int32 words for all of them."""
    words = max(1, -(-max(m.shape[1] for m in masks) // 32))
    out = np.zeros((sum(m.shape[0] for m in masks), words), np.uint32)
    row = 0
    for m in masks:
        for i in range(m.shape[0]):
            for j in range(m.shape[1]):
                if m[i, j]:
                    out[row, j // 32] |= np.uint32(1 << (j % 32))
            row += 1
    return torch.from_numpy(out.view(np.int32)).cuda()


def tree_masks(seqs, seed):
    rng = np.random.default_rng(seed)
    masks = []
    for _, n in seqs:
        m = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            if i:
                m[i] = m[int(rng.integers(max(0, i - 4), i))]
            m[i, i] = True
        masks.append(m)
    return masks


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (7, 1), (6, 2)])
def test_decode(tq, kind, dt, D, Hq, Hkv):
    """Single tokens over lengths around every border: none cached, parts of
    a step, whole steps, several workgroups."""
    s = Setup(tq, kind, [(0, 1), (1, 1), (15, 1), (16, 1), (31, 1), (32, 1), (127, 1), (128, 1),
                         (300, 1), (1025, 1)], Hq, Hkv, D, 16, dt, seed=D + Hq)
    s.check(s.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [16, 32, 64, 256, 1024])
def test_page_sizes(tq, kind, P):
    s = Setup(tq, kind, [(700, 3), (P - 1, 2), (P, 1), (3, 5)], 4, 2, 128, P, seed=P)
    s.check(s.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [2, 5, 17, 33, 70])
def test_trees(tq, kind, D, n):
    seqs = [(200, n), (0, n), (37, max(1, n - 3)), (64, 0), (5, 1)]
    s = Setup(tq, kind, seqs, 4, 2, D, 32, seed=n + D)
    masks = tree_masks(seqs, n)
    s.check(s.run(mask=pack(masks)), masks=masks)
    s.check(s.run())                                      # and as chains


@pytest.mark.parametrize("kind", KINDS)
def test_long_split(tq, kind):
    """Long caches cut over many workgroups, ragged beside short ones."""
    seqs = [(9000, 1), (1, 1), (4097, 1)]
    s = Setup(tq, kind, seqs, 8, 2, 128, 64, seed=2)
    s.check(s.run())
    seqs = [(5000, 13), (100, 2)]
    s = Setup(tq, kind, seqs, 8, 2, 128, 64, "fp16", seed=3)
    masks = tree_masks(seqs, 4)
    s.check(s.run(mask=pack(masks)), masks=masks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (128, 9), (256, 3), (96, 40)])
def test_every_key_counts_once(tq, kind, D, n):
    """Keys of zero: every visible key has the same weight, and value element
    d is set only for positions = d mod D, so an output element counts the
    visible ones among them; one too many or too few is 1 / (L / D)."""
    def v(b, L):
        x = torch.zeros((L, 2, D))
        for j in range(L):
            x[j, :, j % D] = 1.0
        return x
    seqs = [(1500 + D, n), (300, n)]
    s = Setup(tq, kind, seqs, 2, 2, D, 16, "fp16", seed=1, v=v,
              k=lambda b, L: torch.zeros((L, 2, D)))
    masks = tree_masks(seqs, 8)
    out = s.run(mask=pack(masks)).cpu().double()
    row = 0
    for b, (c, nn) in enumerate(seqs):
        see = s.see(b, masks[b]).double()
        want = torch.einsum("tl,lhd->thd", see / see.sum(1, keepdim=True), s.v[b])
        tol = want.abs() * (2.0 ** -11 + 2 * 2.0 ** -11 + (c + nn + 64) * 2.0 ** -24) + 2.0 ** -25
        assert bool(((out[row:row + nn] - want).abs() <= tol).all())
        row += nn


def test_rows_that_see_nothing_are_zero(tq):
    seqs = [(0, 6), (40, 3)]
    s = Setup(tq, "q8_0", seqs, 4, 2, 64, 16, seed=5)
    masks = tree_masks(seqs, 1)
    masks[0][2] = False
    masks[0][5] = False
    masks[1][1] = False                                   # still sees its 40 cached keys
    out = s.run(mask=pack(masks))
    assert bool((out[2] == 0).all()) and bool((out[5] == 0).all())
    s.check(out, masks=masks)
    s = Setup(tq, "q4_0", [(0, 70)], 4, 1, 128, 16, seed=5)
    out = s.run(mask=torch.zeros((70, 3), dtype=torch.int32, device="cuda"))
    assert bool((out == 0).all())


def test_mask_rows_shorter_than_the_tree(tq):
    """New tokens past the mask's words are not seen."""
    seqs = [(10, 40)]
    s = Setup(tq, "q8_0", seqs, 2, 2, 64, 16, seed=6)
    masks = tree_masks(seqs, 3)
    wide = pack(masks)
    masks[0][:, 32:] = False
    s.check(s.run(mask=wide[:, :1]), masks=masks)         # a view: rows two words apart


@pytest.mark.parametrize("kind", KINDS)
def test_unmapped_pages_are_not_seen(tq, kind):
    """Page numbers outside the cache, in the middle and at the end; a table
    row that ends before the sequence."""
    P = 16
    s = Setup(tq, kind, [(100, 2), (60, 1), (33, 4)], 4, 2, 64, P, seed=7)
    t = s.table.clone()
    t[0, 2], t[0, 5], t[1, 0], t[2, 1] = -1, s.pages, 2 ** 31 - 1, -2 ** 31
    dead = [[p for p in range(102) if p // P in (2, 5)], list(range(16)),
            [p for p in range(37) if p // P == 1]]
    s.check(s.run(table=t), dead=dead)
    cut = s.table[:, :3].contiguous()
    dead = [list(range(48, 102)), list(range(48, 61)), []]
    s.check(s.run(table=cut), dead=dead)
    none = torch.full_like(s.table, -1)
    assert bool((s.run(table=none) == 0).all())


def test_lengths_beyond_the_hints(tq):
    """A longer cache than max_ctx is still read whole; rows past max_nodes
    and rows outside the sequences stay as they were."""
    s = Setup(tq, "q8_0", [(900, 1), (50, 1)], 4, 2, 128, 32, seed=8)
    s.check(s.run(max_ctx=0))
    s.check(s.run(max_ctx=5000))
    s = Setup(tq, "q8_0", [(20, 40)], 4, 1, 64, 32, seed=8)
    out = torch.full((44, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    s.run(out=out, max_nodes=16)
    assert bool((out[16:] == 7).all())
    s.run(out=out, max_nodes=64)
    assert bool((out[40:] == 7).all())
    s.check(out[:40])
    big = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32).cuda()
    s.check(s.run(starts=big, max_nodes=40))


def test_defaults(tq):
    s = Setup(tq, "q8_0", [(100, 3), (7, 2)], 4, 2, 64, 16, seed=9)
    s.check(tq.tree_attention(tq.Q8_0, s.q, s.kc, s.vc, s.table, s.ctx, s.starts, 2, 16))


@pytest.mark.parametrize("loud,scale", [(30.0, None), (1e-30, None), (1e4, 1e-3), (1.0, 4.0)])
def test_sharp_and_flat_softmax(tq, loud, scale):
    """Scores whose maximum keeps rising; queries near fp16's limits and far
    below them (bf16 has the range)."""
    s = Setup(tq, "q8_0", [(2500, 1), (400, 5)], 4, 2, 128, 32, seed=10, loud=loud,
              k=lambda b, L: seeded(b, (L, 2, 128)) * torch.linspace(0.01, 3, L)[:, None, None])
    s.check(s.run(scale=scale), scale=scale)


def test_large_values(tq):
    """Keys and values at the largest magnitudes a cache holds."""
    s = Setup(tq, "q8_0", [(200, 2)], 2, 1, 64, 16, "bf16", seed=11,
              k=lambda b, L: torch.full((L, 1, 64), 1e-3),
              v=lambda b, L: seeded(b, (L, 1, 64)).sign() * 1e9)
    out = s.run()
    assert bool(torch.isfinite(out).all())
    s.check(out)


def test_query_with_nan_stays_in_its_row(tq):
    s = Setup(tq, "q8_0", [(100, 4)], 4, 2, 64, 16, seed=12)
    q = s.q.clone()
    q[1, 2, 5] = float("nan")
    q[2, 0, 7] = float("inf")
    out, want = s.run(q=q), s.run()
    assert bool(out[1, 2].isnan().all())
    keep = torch.ones((4, 4), dtype=torch.bool)
    keep[1, 2] = keep[2, 0] = False
    assert torch.equal(out[keep.cuda()], want[keep.cuda()])


def test_strides(tq):
    """Queries inside a fused projection, output heads first, table and mask
    as column ranges of larger ones."""
    seqs = [(90, 4), (20, 3)]
    s = Setup(tq, "q8_0", seqs, 6, 2, 64, 16, seed=13)
    masks = tree_masks(seqs, 2)
    want = s.run(mask=pack(masks))
    rows = torch.zeros((7, 6 * 64 + 130), dtype=torch.bfloat16, device="cuda")
    q = rows[:, 130:].unflatten(1, (6, 64))
    q.copy_(s.q)
    out = torch.zeros((6, 7, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    wide = torch.full((2, s.table.shape[1] + 3), -5, dtype=torch.int32, device="cuda")
    wide[:, :-3] = s.table
    s.run(q=q, out=out, table=wide[:, :-3], mask=pack(masks))
    assert torch.equal(out, want)
    s.check(want, masks=masks)


def test_repeats_bitwise_and_on_other_streams(tq):
    s = Setup(tq, "q8_0", [(6000, 1), (300, 1)], 8, 2, 128, 64, seed=14)
    a = s.run()
    assert torch.equal(a, s.run())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = s.run()
    side.synchronize()
    assert torch.equal(a, b)


def test_offsets_past_32_bits(tq):
    """The sequence's pages lie behind the first 4.3 GB of each buffer."""
    H, D, P = 8, 128, 64
    page = tq.cache_bytes(tq.Q8_0, 1, P, H, D)
    first = (1 << 32) // page + 5
    s = Setup(tq, "q8_0", [(300, 2)], 8, H, D, P, seed=15)
    n = s.kc.numel()
    big = [torch.empty(first * page + n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    big[0][first * page:], big[1][first * page:] = s.kc, s.vc
    s.kc, s.vc = big
    s.check(s.run(table=torch.where(s.table >= 0, s.table + first, s.table)))


def test_empty(tq):
    s = Setup(tq, "q8_0", [(10, 1)], 2, 2, 64, 16)
    out = s.run(q=s.q[:0])
    assert out.shape == (0, 2, 64)
    out = tq.tree_attention(tq.Q8_0, s.q, s.kc, s.vc, s.table[:0], s.ctx[:0], s.starts[:1], 2, 16,
                            out=torch.full_like(s.q, 3.0))
    assert bool((out == 3).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n", [18, 40])
def test_many_short_trees(tq, kind, D, n):
    """More heads and row blocks than compute units, with more than 32 and 64
    rows each: the workgroups of four waves."""
    seqs = [(i * 7 % 90, n - i % 3) for i in range(66)]
    s = Setup(tq, kind, seqs, 8, 4, D, 16, seed=n + D)
    masks = tree_masks(seqs, n)
    s.check(s.run(mask=pack(masks)), masks=masks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,c,n", [(1, 3001, 1), (3, 2000, 1), (7, 1111, 6), (5, 900, 20),
                                   (2, 2500, 45), (64, 130, 1), (65, 130, 1)])
def test_lengths_alike(tq, kind, D, B, c, n):
    """As many keys in every sequence: each head is cut by itself, or many
    are in one line; bounds that are met and bounds far above."""
    s = Setup(tq, kind, [(c, n)] * B, 6, 3, D, 32, seed=B + D)
    s.check(s.run())
    s.check(s.run(max_ctx=8 * c))


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_far_above(tq, kind):
    """Lengths that fill a small part of the line that the bounds stand for:
    spans shorter than what entering a head counts."""
    s = Setup(tq, kind, [(300, 2), (0, 1), (77, 0), (1200, 9), (64, 3)], 8, 2, 128, 64, seed=9)
    s.check(s.run(max_ctx=200000))
    s.check(s.run(max_ctx=200000, max_nodes=64))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (256, 1), (64, 20), (96, 40), (256, 20)])
def test_workgroup_for_each_head(tq, kind, D, n):
    """So many heads and row blocks that none is cut."""
    seqs = [(i * 5 % 200, n - i % min(n, 3)) for i in range(130)]
    s = Setup(tq, kind, seqs, 16, 16, D, 16, seed=n + D)
    s.check(s.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("seqs", [[(2000, 1)] * 3, [(1500, 6), (700, 8)], [(3000, 30)]])
def test_fp16_keeps_its_precision(tq, kind, D, seqs):
    """Against rounding the exact outputs to fp16: the values' rounding to fp16
    is as large as that and independent of it, all else is exact to about
    2^-20, so the error's norm is about sqrt(2) of the rounding's; over 1.5 it
    is not.  Some channels of the keys are loud, so that scores are large."""
    loud = 1.0 + 4.0 * (torch.arange(D) % 20 == 3)
    s = Setup(tq, kind, seqs, 16, 4, D, 32, "fp16", seed=D,
              k=lambda b, L: seeded(7 * b + D, (L, 4, D)) * loud)
    out = s.run().cpu().double()
    err = alone = row = 0
    for b, (c, n) in enumerate(seqs):
        o, _, _ = ref.attention(s.q[row:row + n].cpu(), s.k[b], s.v[b], s.see(b), D ** -0.5)
        err += float((out[row:row + n] - o).square().sum())
        alone += float((o.half().double() - o).square().sum())
        row += n
    assert err <= 1.5 ** 2 * alone, (err / alone) ** 0.5
