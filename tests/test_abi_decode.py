"""Host-side refusals of the decode-step operators: bad arguments come back
as status codes before any HIP call (no GPU, the addresses are never read),
and the binding's own checks raise."""
import ctypes

import pytest
import torch

A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
A4 = ctypes.c_void_p(0x10004)
NUL = None
OK, NULL, TYPE, SHAPE, ALIGN = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    from block_quantized_matmul_repack_amd import _lib
    return _lib.lib()


class Call:
    """An entry point with good arguments by name; call with some replaced."""

    def __init__(self, fn, **good):
        self.fn, self.good = fn, good

    def __call__(self, **kw):
        assert set(kw) <= set(self.good), set(kw) - set(self.good)
        return self.fn(*{**self.good, **kw}.values())


def norm_rope(L):
    return Call(L.tq_qk_norm_rope, dtype=1, q=A, q_ts=512, q_hs=64, q_heads=8, k=A, k_ts=512,
                k_hs=64, k_heads=2, tokens=3, D=64, rot=64, interleaved=0, w_dtype=1, qw=A, kw=A,
                eps=1e-6, pos=A, freq=A, qo=A, qo_ts=512, qo_hs=64, ko=A, ko_ts=128, ko_hs=64,
                stream=NUL)


def test_norm_rope(L):
    c = norm_rope(L)
    assert c(dtype=3) == TYPE and c(w_dtype=-1) == TYPE
    for bad in (dict(D=63), dict(D=0), dict(D=514), dict(rot=65), dict(rot=66), dict(rot=-2),
                dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(q_heads=-1),
                dict(q_heads=1025), dict(q_heads=0, k_heads=0), dict(q_ts=-1), dict(k_hs=-64),
                dict(qo_hs=63), dict(qo_ts=511), dict(ko_ts=100), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert c(**bad) == SHAPE, bad
    assert c(tokens=0, q=NUL, k=NUL, pos=NUL) == OK
    for bad in ("q", "k", "qo", "ko", "pos", "freq"):
        assert c(**{bad: NUL}) == NULL, bad
        assert c(**{bad: ODD}) == ALIGN, bad
    assert c(qw=ODD) == ALIGN and c(dtype=0, q=ctypes.c_void_p(0x10002)) == ALIGN


def test_cache_bytes(L):
    # codes and one fp16 scale per 32 elements, nothing else
    assert L.tq_cache_bytes(1, 3, 16, 2, 96) == 3 * 16 * 2 * 3 * 34
    assert L.tq_cache_bytes(0, 5, 64, 8, 128) == 5 * 64 * 8 * 4 * 18
    for bad in ((2, 3, 16, 2, 96), (1, 0, 16, 2, 96), (1, 3, 8, 2, 96), (1, 3, 48, 2, 96),
                (1, 3, 2048, 2, 96), (1, 3, 16, 0, 96), (1, 3, 16, 1025, 96), (1, 3, 16, 2, 80),
                (1, 1 << 26, 64, 2, 96), (1, -1, 16, 2, 96)):
        assert L.tq_cache_bytes(*bad) == 0, bad


def cache_write(L):
    return Call(L.tq_cache_write, type=1, dtype=1, k=A, k_ts=256, k_hs=64, v=A, v_ts=256, v_hs=64,
                tokens=5, heads=4, D=64, slots=A, kc=A, vc=A, pages=10, page=16, stream=NUL)


def cache_read(L):
    return Call(L.tq_cache_read, type=1, dtype=1, kc=A, vc=A, pages=10, page=16, heads=4, D=64,
                slots=A, tokens=5, k=A, v=A, stream=NUL)


def test_cache_calls(L):
    for c in (cache_write(L), cache_read(L)):
        assert c(type=2) == TYPE and c(dtype=3) == TYPE
        for bad in (dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(heads=0), dict(D=80),
                    dict(page=24), dict(page=8), dict(pages=0), dict(pages=1 << 27),
                    dict(tokens=1 << 20, heads=1024, D=128)):
            assert c(**bad) == SHAPE, bad
        assert c(tokens=0, k=NUL, slots=NUL) == OK
        for name in ("k", "v", "slots", "kc", "vc"):
            assert c(**{name: NUL}) == NULL, name
            assert c(**{name: ODD}) == ALIGN, name
        assert c(kc=A4) == ALIGN and c(vc=A4) == ALIGN
    assert cache_write(L)(k_ts=-1) == SHAPE and cache_write(L)(v_hs=-1) == SHAPE


def attention(L):
    return Call(L.tq_tree_attention, type=1, dtype=1, q=A, q_ts=512, q_hs=64, tokens=6, heads=8,
                kv_heads=2, D=64, kc=A, vc=A, pages=10, page=16, table=A, table_stride=4,
                table_pages=4, batch=2, ctx=A, starts=A, mask=A, mask_stride=1, mask_words=1,
                max_nodes=3, max_ctx=50, scale=0.125, out=A, o_ts=512, o_hs=64, ws=A,
                ws_bytes=1 << 30, stream=NUL)


def test_attention(L):
    c = attention(L)
    assert c(type=3) == TYPE and c(dtype=0) == TYPE and c(dtype=7) == TYPE
    for bad in (dict(heads=7), dict(heads=0), dict(kv_heads=0), dict(heads=2048), dict(D=112),
                dict(tokens=-1), dict(batch=-1), dict(batch=65536), dict(pages=0), dict(page=17),
                dict(table_pages=0), dict(table_pages=1 << 27), dict(table_stride=3),
                dict(max_nodes=0), dict(max_ctx=-1), dict(max_ctx=(1 << 30) + 1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q_ts=-1), dict(o_hs=32), dict(o_ts=500),
                dict(mask_words=0), dict(mask_words=2)):
        assert c(**bad) == SHAPE, bad
    assert c(tokens=0, q=NUL) == OK and c(batch=0, table=NUL) == OK
    for name in ("q", "out", "kc", "vc", "table", "ctx", "starts"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    assert c(mask=ctypes.c_void_p(0x10002)) == ALIGN and c(kc=A4) == ALIGN
    # a long cache is cut over workgroups: the workspace has to hold their sums
    need = L.tq_tree_attention_workspace_bytes(2, 8, 2, 64, 3, 100000)
    assert need > (1 << 20)
    long = dict(max_ctx=100000)
    assert c(ws=NUL, ws_bytes=0, **long) == NULL
    assert c(ws_bytes=need - 1, **long) == SHAPE
    assert c(ws=A4, **long) == ALIGN
    for bad in ((0, 8, 2, 64, 3, 100), (2, 7, 2, 64, 3, 100), (2, 8, 2, 60, 3, 100),
                (2, 8, 2, 64, 0, 100), (2, 8, 2, 64, 3, -1), (2, 8, 0, 64, 3, 100)):
        assert L.tq_tree_attention_workspace_bytes(*bad) == 0, bad


def verify(L):
    return Call(L.tq_verify_draft, dtype=0, target=A, target_stride=100, draft=A,
                draft_stride=100, nodes=6, vocab=100, tokens=A, parents=A, starts=A, batch=2, u=A,
                r=A, width=3, accepted=A, out_tokens=A, out_nodes=A, ws=A, ws_bytes=1 << 30,
                stream=NUL)


def test_verify(L):
    c = verify(L)
    assert c(dtype=4) == TYPE
    for bad in (dict(nodes=-1), dict(batch=-1), dict(batch=65536), dict(vocab=0),
                dict(vocab=(1 << 27) + 1), dict(width=0), dict(width=1025),
                dict(target_stride=99), dict(draft_stride=99)):
        assert c(**bad) == SHAPE, bad
    assert c(batch=0, starts=NUL) == OK
    for name in ("target", "tokens", "u", "starts", "r", "accepted", "out_tokens", "out_nodes",
                 "ws"):
        assert c(**{name: NUL}) == NULL, name
    for name in ("target", "draft", "parents", "tokens", "u", "starts", "r", "accepted",
                 "out_tokens", "out_nodes", "ws"):
        assert c(**{name: ODD}) == ALIGN, name
    need = L.tq_verify_draft_workspace_bytes(2, 100)
    assert c(ws_bytes=need - 1) == SHAPE
    assert L.tq_verify_draft_workspace_bytes(0, 100) == 0
    assert L.tq_verify_draft_workspace_bytes(2, 0) == 0


def test_binding_refuses(L):
    import block_quantized_matmul_repack_amd as tq
    x = torch.zeros((2, 4, 64))
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32)
    c = torch.zeros(tq.cache_bytes(tq.Q8_0, 2, 16, 4, 64), dtype=torch.uint8)
    calls = [
        lambda: tq.qk_norm_rope(x, x, i, f),                          # not on the GPU
        lambda: tq.qk_norm_rope(x[0], x, i, f),
        lambda: tq.qk_norm_rope(x.double(), x, i, f),
        lambda: tq.cache_write(tq.Q8_0, x, x, c, c, i, 16),
        lambda: tq.cache_write(tq.Q8_0, x, x[:, :2], c, c, i, 16),
        lambda: tq.cache_read(tq.Q8_0, c, c, i, 4, 64, 16),
        lambda: tq.cache_read(tq.Q8_0, c, c, i, 4, 64, 16, dtype=torch.int8),
        lambda: tq.tree_attention(tq.Q8_0, x.half(), c, c, i[None], i, i, 4, 16),
        lambda: tq.tree_attention(tq.Q8_0, x, c, c, i[None], i, i, 4, 16),
        lambda: tq.verify_draft(x[0], i, i, f, f),
        lambda: tq.verify_draft(x, i, i, f, f),
    ]
    for call in calls:
        with pytest.raises(tq.TiledqError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    dev = "cuda"
    x = torch.zeros((2, 4, 64), device=dev)
    i = torch.zeros(2, dtype=torch.int32, device=dev)
    f = torch.zeros(32, device=dev)
    c = torch.zeros(tq.cache_bytes(tq.Q8_0, 2, 16, 4, 64), dtype=torch.uint8, device=dev)
    h = x.half()
    t = i[None].contiguous()
    p = torch.zeros((2, 9), device=dev)
    calls = [
        lambda: tq.qk_norm_rope(x, x[:1], i, f),                      # token counts differ
        lambda: tq.qk_norm_rope(x, h, i, f),                          # types differ
        lambda: tq.qk_norm_rope(x, x, i.long(), f),
        lambda: tq.qk_norm_rope(x, x, i[:1], f),
        lambda: tq.qk_norm_rope(x, x, i, f.double()),
        lambda: tq.qk_norm_rope(x, x, i, torch.zeros(40, device=dev)),   # rotates more than D
        lambda: tq.qk_norm_rope(x, x, i, f, f, f),                    # weights of another length
        lambda: tq.qk_norm_rope(x, x, i, f, q_out=x[:, :, ::2]),
        lambda: tq.qk_norm_rope(x, x, i, f, q_out=x[:, :1].expand(2, 4, 64)),   # rows overlap
        lambda: tq.qk_norm_rope(x, x, i.cpu(), f),
        lambda: tq.cache_write(tq.Q4_1, x, x, c, c, i, 16),
        lambda: tq.cache_write(tq.Q8_0, x, x, c, c[:-1], i, 16),
        lambda: tq.cache_write(tq.Q8_0, x, x, c[:-16], c[:-16], i, 16),  # no whole pages
        lambda: tq.cache_write(tq.Q8_0, x, x, c, c, i[:1], 16),
        lambda: tq.cache_write(tq.Q8_0, x, h, c, c, i, 16),
        lambda: tq.cache_write(tq.Q8_0, x, x, c, c, i, 24),
        lambda: tq.cache_write(tq.Q8_0, x[..., :48], x[..., :48], c, c, i, 16),
        lambda: tq.cache_read(tq.Q8_0, c, c, i.long(), 4, 64, 16),
        lambda: tq.cache_read(tq.Q8_0, c, c, i, 4, 64, 16, dtype=torch.float64),
        lambda: tq.tree_attention(tq.Q8_0, x, c, c, t, i, i, 4, 16),     # fp32 queries
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i[:1], 4, 16),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i.long(), i, 4, 16),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i, 3, 16),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i, 4, 16, scale=-1.0),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i, 4, 16, mask=t[:, :1]),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i, 4, 16, out=h[:1]),
        lambda: tq.tree_attention(tq.Q8_0, h, c, c, t, i, i, 4, 16, max_nodes=0),
        lambda: tq.verify_draft(p, i, i, f[:1], f),
        lambda: tq.verify_draft(p, i, i, f, f, draft=p[:1]),
        lambda: tq.verify_draft(p, i, i, f, f, draft=p.half()),
        lambda: tq.verify_draft(p, i, i, f, f, max_nodes=0),
        lambda: tq.verify_draft(p, i, i, f, f, max_nodes=2000),
        lambda: tq.verify_draft(p.int(), i, i, f, f),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(tq.TiledqError):
            call()
            print("not refused:", n)


def test_outgrown_workspaces_are_kept(monkeypatch):
    """A captured graph may hold the address of one; none is cleared twice."""
    from block_quantized_matmul_repack_amd import ops
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_outgrown", [])
    cpu = torch.device("cpu")
    first = ops.workspace(cpu, 1, 1 << 17)
    assert ops.workspace(cpu, 1, 1 << 16) is first and ops.workspace(cpu, 2, 1 << 17) is not first
    second = ops.workspace(cpu, 1, (1 << 17) + 1)
    assert second.numel() >= 2 * first.numel() and not second.any()
    assert ops._outgrown == [first] and ops.workspace(cpu, 1, 1 << 17) is second
