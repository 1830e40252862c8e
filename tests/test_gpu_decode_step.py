"""The decode-step operators together: a step captured in a HIP graph gives
the bits of the eager step on every replay, with new inputs and other work
in between; side streams give the bits of the default one; the workspace's
counters are zero after every call; the example's step runs."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

H, HK, D, P, V, B = 8, 2, 128, 32, 4099, 3
CTX = (700, 3000, 33)
N = 5                                       # nodes of each sequence: a chain of 4 drafted ones


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    tq.lib()
    return tq


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    T = B * N
    soft = lambda: torch.softmax(2 * torch.randn((T, V), generator=g), -1)   # noqa: E731
    x = {"qkv": torch.randn((T, (H + 2 * HK) * D), generator=g).bfloat16(),
         "target": soft(), "draft": soft(), "u": torch.rand(T, generator=g),
         "r": torch.rand(B, generator=g),
         "tokens": torch.randint(0, V, (T,), generator=g, dtype=torch.int32)}
    return {k: v.cuda() for k, v in x.items()}


class Step:
    """Fixed buffers, one call of each operator."""

    def __init__(self, tq):
        self.tq = tq
        per = [-(-(c + N) // P) for c in CTX]
        n = tq.cache_bytes(tq.Q8_0, sum(per), P, HK, D)
        self.kc, self.vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        table = torch.full((B, max(per)), -1, dtype=torch.int32)
        at, slots, pos = 0, [], []
        for b in range(B):
            table[b, :per[b]] = torch.arange(at, at + per[b])
            at += per[b]
            for i in range(N):
                p = CTX[b] + i
                slots.append(int(table[b, p // P]) * P + p % P)
                pos.append(p)
        self.table = table.cuda()
        g = torch.Generator().manual_seed(1)
        every = torch.arange(sum(per) * P, dtype=torch.int32).cuda()
        fill = torch.randn((2, every.numel(), HK, D), generator=g).bfloat16().cuda()
        tq.cache_write(tq.Q8_0, fill[0], fill[1], self.kc, self.vc, every, P)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()            # noqa: E731
        self.slots, self.pos, self.ctx = i32(slots), i32(pos), i32(CTX)
        self.starts = i32([N * b for b in range(B + 1)])
        self.freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).cuda()
        self.w = torch.ones(D).bfloat16().cuda()
        self.x = inputs(0)

    def __call__(self):
        tq, x = self.tq, self.x
        q = x["qkv"][:, :H * D].unflatten(1, (H, D))
        k = x["qkv"][:, H * D:(H + HK) * D].unflatten(1, (HK, D))
        v = x["qkv"][:, (H + HK) * D:].unflatten(1, (HK, D))
        q, k = tq.qk_norm_rope(q, k, self.pos, self.freq, self.w, self.w)
        tq.cache_write(tq.Q8_0, k, v, self.kc, self.vc, self.slots, P)
        o = tq.tree_attention(tq.Q8_0, q, self.kc, self.vc, self.table, self.ctx, self.starts, HK,
                              P, max_nodes=N, max_ctx=max(CTX))
        kr, vr = tq.cache_read(tq.Q8_0, self.kc, self.vc, self.slots, HK, D, P)
        return (o, kr, vr) + tq.verify_draft(x["target"], x["tokens"], self.starts, x["u"],
                                             x["r"], draft=x["draft"], max_nodes=N)


def counters_zero():
    from block_quantized_matmul_repack_amd import ops
    torch.cuda.synchronize()
    return all(bool((ws[:1 << 20] == 0).all()) for ws in ops._workspaces.values())


def test_graph_replays_match_eager(tq):
    step = Step(tq)
    eager = []
    for seed in range(4):
        for k, v in inputs(seed).items():
            step.x[k].copy_(v)
        eager.append([t.clone() for t in step()])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()                              # the stream's workspace exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step()
    for turn, seed in enumerate((2, 0, 3, 1, 1, 2)):
        for k, v in inputs(seed).items():
            step.x[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager[seed]):
            assert torch.equal(a, b), (turn, seed)
        if turn % 2:                        # the program's own work between replays
            torch.randn(1 << 20, device="cuda").sum().item()
            assert counters_zero()
    assert counters_zero()


def captured(step, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step()
    return graph, out


def test_outgrown_workspace_stays_the_graphs(tq, monkeypatch):
    """After a capture a longer call needs a larger workspace on the same
    stream; replays still have theirs, and write nothing else."""
    from block_quantized_matmul_repack_amd import ops
    step = Step(tq)
    want = [t.clone() for t in step()]
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_outgrown", [])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    (old,) = ops._workspaces.values()
    size = old.numel()
    del old
    graph, out = captured(step, stream)
    q = torch.randn((B * N, H, D)).bfloat16().cuda()
    with torch.cuda.stream(stream):
        tq.tree_attention(tq.Q8_0, q, step.kc, step.vc, step.table, step.ctx, step.starts, HK, P,
                          max_nodes=64, max_ctx=1 << 20)
        assert max(w.numel() for w in ops._workspaces.values()) > size
        others = [torch.full((size // 4,), 77, dtype=torch.uint8, device="cuda") for _ in range(9)]
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(bool((t == 77).all()) for t in others)


def test_capture_before_there_is_a_workspace(tq, monkeypatch):
    """The graph then fills its own; eager calls on its stream have another."""
    from block_quantized_matmul_repack_amd import ops
    step = Step(tq)
    want = [t.clone() for t in step()]
    monkeypatch.setattr(ops, "_workspaces", {})
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, out = captured(step, stream)
    assert not ops._workspaces
    for _ in range(3):
        with torch.cuda.stream(stream):
            got = step()
            stream.synchronize()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert counters_zero()


def test_side_stream_matches_default(tq):
    step = Step(tq)
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert counters_zero()


def test_workspace_shared_with_the_products(tq):
    """Attention, verification and a split product one after another on one
    stream use one workspace; each still finds its counters zero."""
    import synth
    step = Step(tq)
    want = [t.clone() for t in step()]
    inp = synth.make_inputs(synth.Workload("t", synth.Q8_0, 4096, 300, 1, "absnormal"))
    tiles = tq.repack_tiles(synth.Q8_0, torch.from_numpy(inp.flat).cuda(), 4096, 300)
    x = torch.from_numpy(inp.x).cuda()
    y = tq.matmul_x(synth.Q8_0, tiles, 4096, 300, x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
        assert torch.equal(tq.matmul_x(synth.Q8_0, tiles, 4096, 300, x), y)
    assert counters_zero()


def test_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import speculative_decode
    finally:
        sys.path.pop(0)
    tokens, steps = speculative_decode.generate(new_tokens=24, prompt=40, quiet=True)
    assert len(tokens) >= 24 and 1 <= steps <= 24
    plain, _ = speculative_decode.generate(new_tokens=24, prompt=40, drafted=0, quiet=True)
    assert tokens[:8] == plain[:8]          # greedy: speculation changes no token
