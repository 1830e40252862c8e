"""The serving-step operators together: a step captured in a HIP graph, its state
carried on inside it, gives the bits of the eager steps replay after replay, with
other work in between; side streams give the bits of the default one; the
workspace's counters stay zero; threads share a stream; the example serves."""
import os
import sys
import threading

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

HQ, HK, D, P, V, HID = 8, 2, 64, 16, 9001, 512
B, ROWS, PAGES, WIDTH, KEEP = 5, 12, 300, 60, 3


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    tq.lib()
    return tq


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """A step of five requests, its state in fixed buffers."""

    def __init__(self, tq, seed=0):
        import synth
        self.tq = tq
        g = torch.Generator().manual_seed(seed)
        self.lens, self.owned = int32([0] * B), int32([0] * B)
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(PAGES, generator=g).int().cuda()
        self.count = int32([PAGES])
        n = tq.cache_bytes(tq.Q8_0, PAGES, P, HK, D)
        self.kc, self.vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.codes = torch.zeros((PAGES, HK, D // 32, 2, 32), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((PAGES, HK, D // 32), dtype=torch.float16, device="cuda")
        w = synth.make_inputs(synth.Workload("t", synth.Q8_0, HID, V, 1, "absnormal"))
        self.head = (synth.Q8_0, tq.repack_tiles(synth.Q8_0, torch.from_numpy(w.flat).cuda(), HID, V),
                     HID, V)
        self.norm = (1 + 0.1 * torch.randn(HID, generator=g)).cuda()
        self.new = int32([0] * B)
        self.qkv = torch.zeros((ROWS, HQ + 2 * HK, D), dtype=torch.bfloat16, device="cuda")
        self.x = torch.zeros((ROWS, HID), device="cuda")
        self.u = torch.zeros(ROWS, device="cuda")
        self.temp = torch.tensor([0.0, 0.7, 1.0, 1.3] * 3, device="cuda")
        self.top_k, self.top_p = int32([0, 40, 5] * 4), torch.full((ROWS,), 0.9, device="cuda")

    def set(self, seed):
        g = torch.Generator().manual_seed(seed)
        new = torch.randint(0, 4, (B,), generator=g).int()
        new[-1] = min(ROWS - int(new[:-1].sum()), 3)
        self.new.copy_(new)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g))
        self.x.copy_(torch.randn(self.x.shape, generator=g))
        self.u.copy_(torch.rand(ROWS, generator=g))

    def __call__(self):
        tq = self.tq
        starts, pos, slots, lens, owned, count = tq.plan_step(
            self.lens, self.new, self.owned, self.table, self.free, self.count, P, ROWS)
        q, k, v = self.qkv.split((HQ, HK, HK), 1)
        tq.cache_write(tq.Q8_0, k, v, self.kc, self.vc, slots, P)
        tq.cache_bounds(tq.Q8_0, self.kc, self.table, self.lens, lens, HK, D, P, self.codes,
                        self.scales, max_new=ROWS)
        tables, ctx = tq.select_pages(q, self.codes, self.scales, self.table, self.lens, starts, P,
                                      KEEP, max_nodes=ROWS)
        o = tq.tree_attention(tq.Q8_0, q, self.kc, self.vc, tables, ctx, starts, HK, P,
                              max_nodes=ROWS, out=torch.zeros_like(q))
        x, act = tq.residual_norm(o.flatten(1), self.x, self.norm, gate=self.norm, quantize=True)
        logits = tq.matmul(*self.head, *act)
        settings = dict(temperature=self.temp, top_k=self.top_k, top_p=self.top_p)
        tokens = tq.sample(logits, self.u, **settings)
        probs = tq.sample_probs(logits, **settings)
        done = (lens > 700).int()
        owned, count = tq.release_pages(done, owned, self.table, self.free, count)
        self.lens.copy_(lens * (1 - done))
        self.owned.copy_(owned)
        self.count.copy_(count)
        return starts, pos, slots, tables, ctx, o, x, *act, tokens, probs, lens, owned, count


def state(s):
    return [t.clone() for t in (s.lens, s.owned, s.count, s.table, s.free, s.codes, s.scales, s.kc)]


def fill(s, steps):
    """Long requests, so that pages are left out."""
    s.lens.copy_(int32([690, 200, 655, 17, 0]))
    s.owned.copy_((s.lens + P - 1) // P)
    at = PAGES
    table, free = s.table.cpu(), s.free.tolist()
    for b, n in enumerate(s.owned.tolist()):
        for j in range(n):
            at -= 1
            table[b, j] = free[at]
    s.table.copy_(table)
    s.count.fill_(at)
    every = torch.arange(PAGES * P, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn((2, PAGES * P, HK, D), generator=g).bfloat16().cuda()
    s.tq.cache_write(s.tq.Q8_0, k, v, s.kc, s.vc, every, P)
    s.tq.cache_bounds(s.tq.Q8_0, s.kc, s.table, int32([0] * B), s.lens, HK, D, P, s.codes, s.scales)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_replayed_steps_are_the_eager_ones(tq):
    eager, graphed = Step(tq), Step(tq)
    for s in (eager, graphed):
        fill(s, 1)
        s.set(100)
        s()                                      # once eagerly, on both
    graph = torch.cuda.CUDAGraph()
    before = state(graphed)
    with torch.cuda.graph(graph):
        out = graphed()
    assert same(state(graphed), before)          # a capture runs nothing
    for step in range(8):
        for s in (eager, graphed):
            s.set(step)
        want = eager()
        torch.cuda.synchronize()
        graph.replay()
        if step % 2:                             # other work on the same stream
            eager.tq.sample_probs(torch.randn((3, 40000), device="cuda"))
        torch.cuda.synchronize()
        assert same(out, want), step
        assert same(state(graphed), state(eager)), step


def test_side_streams(tq):
    want = None
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        s = Step(tq)
        fill(s, 1)
        s.set(4)
        torch.cuda.synchronize()
        if stream is None:
            out = s()
        else:
            with torch.cuda.stream(stream):
                out = s()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + state(s)
        want = want or got
        assert same(got, want)


def test_threads_share_a_stream(tq):
    """Calls of several launches from many threads on one stream."""
    g = torch.Generator().manual_seed(2)
    x = [torch.randn((4, 30000 + i), generator=g).cuda() for i in range(4)]
    u = torch.rand(4, generator=g).cuda()
    p = torch.full((4,), 0.9, device="cuda")
    want = [tq.sample(a, u, top_p=p) for a in x]
    stream, failed = torch.cuda.Stream(), []
    torch.cuda.synchronize()

    def run(i):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    if not torch.equal(tq.sample(x[i], u, top_p=p), want[i]):
                        failed.append(i)
        except BaseException as e:               # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_workspace_counters_stay_zero(tq):
    from block_quantized_matmul_repack_amd import ops
    s = Step(tq)
    fill(s, 1)
    s.set(0)
    s()
    torch.cuda.synchronize()
    used = [w for w in ops._workspaces.values() if w.numel() > 1 << 20]
    assert used and all(not w[:1 << 20].any() for w in used)


def test_sampled_distributions_verify_drafts(tq):
    """sample_probs is what verify_draft takes: drafts that the target is sure of
    are accepted, and the next token is sample's for the same number."""
    g = torch.Generator().manual_seed(1)
    logits = 3 * torch.randn((4, 5000), generator=g).cuda()
    k = int32([30] * 4)
    probs = tq.sample_probs(logits, top_k=k)
    u = torch.rand(1, generator=g).cuda()
    for row in range(4):
        count, tokens, _ = tq.verify_draft(probs[row:row + 1], int32([0]), int32([0, 1]),
                                           torch.zeros(1, device="cuda"), u)
        assert count.item() == 0
        assert tokens[0, 0] == tq.sample(logits[row:row + 1], u, top_k=k)[0]
    greedy = tq.sample_probs(logits, temperature=torch.zeros(4, device="cuda"))
    likely = logits.argmax(-1).int()
    count, tokens, _ = tq.verify_draft(greedy, torch.cat((int32([7]), likely[:3])), int32([0, 4]),
                                       torch.full((4,), 0.99, device="cuda"), u, max_nodes=4)
    assert count.item() == 3 and tokens[0].tolist() == likely.tolist()


def test_example_serves(tq):
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    from examples import serve
    texts, steps, s = serve.serve(6, 9, quiet=True)
    assert [len(t) for t in texts] == [9] * 6
    assert all(0 <= t < serve.VOCAB for text in texts for t in text)
    # all pages are back
    assert s.count.item() == serve.PAGES and (s.table == -1).all() and (s.owned == 0).all()
    assert sorted(s.free.tolist()) == list(range(serve.PAGES))
    again, _, _ = serve.serve(6, 9, quiet=True)
    assert again == texts
    assert os.path.exists(os.path.join(ROOT, "examples", "serve.py"))
