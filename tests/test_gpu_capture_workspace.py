"""A graph captured on a stream that no eager call ran on, which is what
torch.cuda.graph gives by default: its calls share one workspace, cleared once
a replay, and only where it has to be."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_gpu_decode_step import B, D, H, HK, N, P, V, Step, inputs, tq  # noqa: F401

pytestmark = pytest.mark.gpu

COUNTERS = 1 << 20                          # TQ_NOALLOC_SCRATCH_BYTES


class Fills(TorchDispatchMode):
    """Bytes of tensors that are filled with zeros."""

    def __init__(self):
        super().__init__()
        self.bytes = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func.overloadpacket in (torch.ops.aten.zeros, torch.ops.aten.zero_,
                                   torch.ops.aten.fill_):
            self.bytes += out.numel() * out.element_size()
        return out


class Layers(Step):
    """Three layers of the step, with a long bound and a split product each."""

    def __init__(self, tq):
        import synth
        super().__init__(tq)
        inp = synth.make_inputs(synth.Workload("t", synth.Q8_0, 4096, 300, 1, "absnormal"))
        self.w = tq.repack_tiles(synth.Q8_0, torch.from_numpy(inp.flat).cuda(), 4096, 300)
        self.a = torch.from_numpy(inp.x).cuda()
        self.norm = torch.ones(D).bfloat16().cuda()

    def __call__(self):
        tq, x = self.tq, self.x
        q = x["qkv"][:, :H * D].unflatten(1, (H, D))
        outs = []
        for most in (4000, 40000, 400000):
            outs.append(tq.tree_attention(tq.Q8_0, q, self.kc, self.vc, self.table, self.ctx,
                                          self.starts, HK, P, max_nodes=64, max_ctx=most))
            outs.append(tq.matmul_x(tq.Q8_0, self.w, 4096, 300, self.a))
        return tuple(outs) + tq.verify_draft(x["target"], x["tokens"], self.starts, x["u"],
                                             x["r"], draft=x["draft"], max_nodes=N)


def record(step, **kw):
    graph, fills = torch.cuda.CUDAGraph(), Fills()
    with torch.cuda.graph(graph, **kw):
        with fills:
            out = step()
    return graph, out, fills.bytes


@pytest.fixture
def fresh(monkeypatch):
    from block_quantized_matmul_repack_amd import ops
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_outgrown", [])
    monkeypatch.setattr(ops, "_captured", {}, raising=False)
    return ops


def replays(step, graph, out, want):
    for turn, seed in enumerate((2, 0, 1, 1, 2)):
        for k, v in inputs(seed).items():
            step.x[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[seed]):
            assert torch.equal(a, b), (turn, seed)
        if turn % 2:                        # the program's own work between replays
            torch.randn(1 << 22, device="cuda").sum().item()
            step()
            torch.cuda.synchronize()


def eager(step):
    want = []
    for seed in range(3):
        for k, v in inputs(seed).items():
            step.x[k].copy_(v)
        want.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    return want


def test_one_workspace_for_a_capture(tq, fresh):
    step = Layers(tq)
    want = eager(step)
    graph, out, filled = record(step)
    # the three bounds need more each: at most a counter region for each
    assert filled <= 3 * COUNTERS, filled
    replays(step, graph, out, want)
    # a second capture on the same stream has its own; both stay right, in any order
    again, out2, filled = record(step)
    assert COUNTERS <= filled <= 3 * COUNTERS, filled
    for _ in range(2):
        replays(step, again, out2, want)
        replays(step, graph, out, want)
    del graph, out
    torch.cuda.empty_cache()
    others = [torch.full((1 << 22,), 77, dtype=torch.uint8, device="cuda") for _ in range(20)]
    replays(step, again, out2, want)
    assert all(bool((t == 77).all()) for t in others)


def test_the_second_layer_fills_nothing(tq, fresh):
    step = Step(tq)
    want = eager(step)
    _, _, one = record(step)
    graph, out, three = record(lambda: (step(), step(), step())[2])
    assert 0 < three == one <= COUNTERS
    replays(step, graph, out, want)


def test_graphs_of_one_pool(tq, fresh):
    """Two graphs that share their memory, replayed in the order of their
    capture."""
    step = Step(tq)
    want = eager(step)
    pool = torch.cuda.graph_pool_handle()
    first, out1, _ = record(step, pool=pool)
    kept = [torch.empty_like(t) for t in out1]
    second, out2, _ = record(step, pool=pool)
    for seed in (1, 2, 0):
        for k, v in inputs(seed).items():
            step.x[k].copy_(v)
        first.replay()
        for a, b in zip(kept, out1):
            a.copy_(b)
        second.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want[seed]))
        assert all(torch.equal(a, b) for a, b in zip(out2, want[seed]))


def test_capture_that_was_left(tq, fresh):
    """A capture that an exception ended: the next one starts anew."""
    step = Step(tq)
    want = eager(step)
    with pytest.raises(RuntimeError, match="on the way"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
            raise RuntimeError("on the way")
    del graph
    graph, out, filled = record(step)
    assert 0 < filled <= COUNTERS
    replays(step, graph, out, want)
