"""The binding without a GPU: tensors of the CPU that say they are on GPU 0 and
a library of stand-ins, to see in which order the calls reach it and which
arguments it refuses."""
import threading
import time

import pytest
import torch

import block_quantized_matmul_repack_amd as tq
from block_quantized_matmul_repack_amd import ops


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def gpu(t):
    return t.as_subclass(OnGpu)


class Library:
    """Entry points that note who is inside with which workspace."""

    def __init__(self, real):
        self.real, self.inside, self.shared, self.calls = real, {}, [], 0
        self.lock = threading.Lock()

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            at, need = args[-3], args[-2]
            if not need:
                return 0
            with self.lock:
                self.calls += 1
                if self.inside.get(at):
                    self.shared.append((name, self.inside[at]))
                self.inside[at] = name
            time.sleep(0.005)                    # between the call's two launches
            with self.lock:
                self.inside[at] = None
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    real = ops.lib()
    fake = Library(real)
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_outgrown", [])
    monkeypatch.setattr(ops, "_stream", lambda t: 7)
    monkeypatch.setattr(ops, "_stream_of", lambda dev: 7)
    return fake


def attention():
    D, P, H = 64, 16, 8
    n = tq.cache_bytes(tq.Q8_0, 4, P, H, D)
    i32 = lambda x: gpu(torch.tensor(x, dtype=torch.int32))              # noqa: E731
    cache = [gpu(torch.zeros(n, dtype=torch.uint8)) for _ in "kv"]
    q = gpu(torch.zeros((1, H, D), dtype=torch.bfloat16))
    table, ctx, starts = i32([[0, 1, 2, 3]]), i32([60]), i32([0, 1])
    return lambda: tq.tree_attention(tq.Q8_0, q, *cache, table, ctx, starts, H, P, max_ctx=8192)


def verification():
    p, f = gpu(torch.ones((2, 5000))), lambda n: gpu(torch.zeros(n))
    i32 = lambda x: gpu(torch.tensor(x, dtype=torch.int32))              # noqa: E731
    args = p, i32([0, 1]), i32([0, 2]), f(2), f(1)
    return lambda: tq.verify_draft(*args)


def product():
    K, N, M = 4096, 256, 40
    tiles = gpu(torch.zeros(tq.tiled_bytes(tq.Q8_0, K, N), dtype=torch.uint8))
    x = gpu(torch.zeros((M, K)))
    return lambda: tq.matmul_x(tq.Q8_0, tiles, K, N, x)


def test_calls_on_one_stream_take_turns(library):
    """A call is several launches over its stream's workspace: another
    thread's must not come between them."""
    work = [attention(), verification(), product(), attention()]
    failed = []

    def run(f):
        try:
            for _ in range(5):
                f()
        except BaseException as e:               # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert library.calls == 20
    assert not library.shared
    assert len(ops._workspaces) == 1


def test_outputs_of_another_rank_are_refused(library):
    """The binding's own error, not Python's from taking strides apart."""
    q, k = (gpu(torch.zeros((3, h, 64), dtype=torch.bfloat16)) for h in (8, 2))
    pos, freq = gpu(torch.zeros(3, dtype=torch.int32)), gpu(torch.ones(32))
    for bad in (gpu(torch.zeros((3, 8 * 64), dtype=torch.bfloat16)),
                gpu(torch.zeros((1, 3, 8, 64), dtype=torch.bfloat16)),
                gpu(torch.zeros((), dtype=torch.bfloat16))):
        with pytest.raises(tq.TiledqError, match="q_out"):
            tq.qk_norm_rope(q, k, pos, freq, q_out=bad)
        with pytest.raises(tq.TiledqError, match="k_out"):
            tq.qk_norm_rope(q, k, pos, freq, k_out=bad)
    q_out, k_out = tq.qk_norm_rope(q, k, pos, freq)
    assert q_out.shape == q.shape and k_out.shape == k.shape


def test_capture_number_needs_a_place():
    assert ops.lib().tq_capture_id(None, None) == 1          # TQ_E_NULL


def test_calls_of_a_capture_share_a_workspace(monkeypatch):
    """A larger need gets a larger one, another capture or stream its own, and
    only the counters are cleared."""
    monkeypatch.setattr(ops, "_captured", {})
    cpu = torch.device("cpu")
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **k).fill_(9))
    first = ops._captured_workspace(cpu, 1, 11, 1 << 21)
    assert ops._captured_workspace(cpu, 1, 11, 1 << 16) is first
    assert not first[:1 << 20].any() and bool((first[1 << 20:] == 9).all())
    larger = ops._captured_workspace(cpu, 1, 11, (1 << 21) + 1)
    assert larger is not first and ops._captured_workspace(cpu, 1, 11, 1 << 21) is larger
    assert ops._captured_workspace(cpu, 2, 11, 1 << 16) is not larger
    assert ops._captured_workspace(cpu, 1, 12, 1 << 16) is not larger
