"""Host-side refusals of the serving-step operators: bad arguments come back
as status codes before any HIP call (no GPU, the addresses are never read),
and the binding's own checks raise."""
import ctypes

import pytest
import torch

from test_abi_decode import A, A4, ALIGN, Call, NUL, NULL, ODD, OK, SHAPE, TYPE, attention

I32 = 0x10000


def P(i):
    """Addresses apart from each other."""
    return ctypes.c_void_p(I32 + (i << 20))


@pytest.fixture(scope="module")
def L():
    from block_quantized_matmul_repack_amd import _lib
    return _lib.lib()


def plan(L):
    return Call(L.tq_plan_step, batch=3, lens=P(0), new=P(1), owned=P(2), table=P(3), table_stride=9,
                table_pages=8, page=16, free=P(4), capacity=50, count=P(5), tokens=20, starts=P(6),
                positions=P(7), slots=P(8), new_lens=P(9), new_owned=P(10), left=P(11), stream=NUL)


def test_plan(L):
    c = plan(L)
    for bad in (dict(batch=-1), dict(batch=65536), dict(page=8), dict(page=24), dict(page=2048),
                dict(table_pages=0), dict(table_pages=1 << 27), dict(table_pages=1 << 26, table_stride=1 << 26,
                                                                     page=1024),
                dict(table_stride=7), dict(table_stride=-1), dict(capacity=-1),
                dict(capacity=(1 << 26) + 1), dict(tokens=-1), dict(tokens=(1 << 20) + 1)):
        assert c(**bad) == SHAPE, bad
    for name in ("lens", "new", "owned", "table", "free", "count", "starts", "positions", "slots",
                 "new_lens", "new_owned", "left"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    # the state is read while the next one is written: they stay apart
    for name, other in (("new_lens", 0), ("new_owned", 2), ("left", 5), ("starts", 1), ("slots", 4)):
        assert c(**{name: P(other)}) == SHAPE, name
    assert c(new_lens=ctypes.c_void_p(I32 + 8)) == SHAPE
    # nothing lies in the table, which is read and written
    row2 = ctypes.c_void_p(P(3).value + 4 * (2 * 9 + 7))
    for name in ("lens", "new", "owned", "free", "count", "starts", "positions", "slots", "new_lens",
                 "new_owned", "left"):
        assert c(**{name: row2}) == SHAPE, name


def release(L):
    return Call(L.tq_release_pages, batch=3, done=P(0), owned=P(2), table=P(3), table_stride=9,
                table_pages=8, free=P(4), capacity=50, count=P(5), new_owned=P(10), left=P(11),
                stream=NUL)


def test_release(L):
    c = release(L)
    for bad in (dict(batch=-1), dict(batch=65536), dict(table_pages=0), dict(table_stride=7),
                dict(capacity=-1), dict(capacity=(1 << 26) + 1), dict(new_owned=P(2)),
                dict(new_owned=P(0)), dict(left=P(5))):
        assert c(**bad) == SHAPE, bad
    for name in ("done", "owned", "table", "free", "count", "new_owned", "left"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    # nothing lies in the table or the stack, which are written
    row2, last = ctypes.c_void_p(P(3).value + 4 * (2 * 9 + 7)), ctypes.c_void_p(P(4).value + 4 * 49)
    for name in ("done", "owned", "count", "new_owned", "left"):
        assert c(**{name: row2}) == SHAPE and c(**{name: last}) == SHAPE, name
    assert c(free=row2) == SHAPE


def residual(L, **kw):
    good = dict(dtype=1, y_dtype=0, y=A, y_ts=64, x=A, x_ts=64, tokens=3, N=64, w_dtype=1, post=A,
                pre=A, gate=A, gate_ts=0, gate_es=1, scale=1.0, eps=1e-6, x_out=A, xo_ts=64, z=A,
                z_ts=64, q=NUL, d=NUL, stream=NUL)
    return Call(L.tq_residual_norm, **{**good, **kw})


def test_residual_norm(L):
    c = residual(L)
    for bad in (dict(dtype=3), dict(y_dtype=-1), dict(w_dtype=7)):
        assert c(**bad) == TYPE, bad
    for bad in (dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(N=0), dict(N=32769),
                dict(y_ts=-1), dict(x_ts=-1), dict(xo_ts=63), dict(z_ts=63), dict(gate_ts=-1),
                dict(gate_es=2), dict(gate_es=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan"))):
        assert c(**bad) == SHAPE, bad
    assert c(tokens=0, y=NUL) == OK
    assert c(x_ts=0) == SHAPE and c(xo_ts=128) == SHAPE      # in place, at another stride
    for name in ("y", "x", "x_out", "z"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    for name in ("post", "pre", "gate"):
        assert c(**{name: ODD}) == ALIGN, name
    # z or q and d, one of them and whole
    c = residual(L, z=NUL, q=A, d=A)
    assert c(q=NUL) == NULL and c(d=NUL) == NULL and c(z=A) == NULL
    assert c(N=48) == SHAPE and c(q=ctypes.c_void_p(0x10002)) == ALIGN and c(d=ODD) == ALIGN


def sample(L):
    return Call(L.tq_sample, dtype=0, logits=A, stride=100, rows=3, vocab=100, temp=A, top_k=A,
                top_p=A, min_p=A, u=A, tokens=A, ws=A, ws_bytes=1 << 40, stream=NUL)


def probs(L):
    return Call(L.tq_sample_probs, dtype=0, logits=A, stride=100, rows=3, vocab=100, temp=A,
                top_k=A, top_p=A, min_p=A, probs=A, probs_stride=100, ws=A, ws_bytes=1 << 40,
                stream=NUL)


def test_sample(L):
    for c, outs in ((sample(L), ("u", "tokens")), (probs(L), ("probs",))):
        assert c(dtype=3) == TYPE
        for bad in (dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0),
                    dict(vocab=(1 << 27) + 1), dict(stride=-1),
                    dict(rows=1 << 10, vocab=1 << 24, stride=1 << 24)):
            assert c(**bad) == SHAPE, bad
        assert c(rows=0, logits=NUL) == OK
        for name in ("logits", *outs):
            assert c(**{name: NUL}) == NULL, name
            assert c(**{name: ODD}) == ALIGN, name
        for name in ("temp", "top_k", "top_p", "min_p"):
            assert c(**{name: ODD}) == ALIGN, name
        need = L.tq_sample_workspace_bytes(3, 100)
        if need:
            assert c(ws=NUL) == NULL and c(ws_bytes=need - 1) == SHAPE and c(ws=A4) == ALIGN
    assert probs(L)(probs_stride=99) == SHAPE
    assert L.tq_sample_workspace_bytes(0, 100) == 0 == L.tq_sample_workspace_bytes(3, 0)


def bounds(L):
    return Call(L.tq_cache_bounds, type=1, kc=A, pages=10, page=16, heads=2, D=64, table=A,
                table_stride=4, table_pages=4, batch=2, begin=A, end=A, max_new=50, codes=A,
                scales=A, stream=NUL)


def test_bounds(L):
    c = bounds(L)
    assert c(type=2) == TYPE
    for bad in (dict(pages=0), dict(page=17), dict(heads=0), dict(D=80), dict(batch=-1),
                dict(batch=65536), dict(table_pages=0), dict(table_stride=3), dict(max_new=-1),
                dict(max_new=(1 << 30) + 1),
                dict(heads=1024, D=256, table_pages=1 << 20, table_stride=1 << 20, max_new=1 << 25)):
        assert c(**bad) == SHAPE, bad
    assert c(batch=0, table=NUL) == OK and c(max_new=0, table=NUL) == OK
    for name in ("kc", "table", "begin", "end", "codes", "scales"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    assert c(codes=A4) == ALIGN


def select(L):
    return Call(L.tq_select_pages, dtype=1, q=P(0), q_ts=512, q_hs=64, tokens=6, heads=8, kv_heads=2,
                D=64, codes=P(1), scales=P(2), pages=10, page=16, table=P(3), table_stride=40,
                table_pages=40, batch=2, ctx=P(4), starts=P(5), max_nodes=3, max_ctx=600, first=1,
                last=1, keep=4, width=8, tables=P(6), ctx_out=P(7), ws=A, ws_bytes=1 << 40,
                stream=NUL)


def test_select(L):
    # 1 + 1 + 4 pages, and three new tokens on two at most
    assert L.tq_select_pages_width(16, 40, 1, 1, 4, 3) == 8
    assert L.tq_select_pages_width(16, 5, 1, 1, 4, 3) == 5
    assert L.tq_select_pages_width(16, 40, 0, 0, 0, 1) == 1
    for bad in ((8, 40, 1, 1, 4, 3), (16, 0, 1, 1, 4, 3), (16, 40, -1, 1, 4, 3), (16, 40, 1, -1, 4, 3),
                (16, 40, 1, 1, -1, 3), (16, 40, 1, 1, 4, 0)):
        assert L.tq_select_pages_width(*bad) == 0, bad
    c = select(L)
    assert c(dtype=0) == TYPE and c(dtype=4) == TYPE
    for bad in (dict(heads=7), dict(heads=0), dict(kv_heads=0), dict(D=80), dict(tokens=-1),
                dict(batch=-1), dict(batch=65536), dict(batch=65535, kv_heads=64, heads=64),
                dict(page=20), dict(table_pages=0), dict(table_stride=39), dict(max_nodes=0),
                dict(max_ctx=-1), dict(first=-1), dict(last=-1), dict(keep=-1), dict(width=7),
                dict(keep=5), dict(q_ts=-1), dict(ctx_out=P(4)), dict(tables=P(3)),
                dict(ctx_out=P(5)), dict(tables=P(4)), dict(tables=P(5))):
        assert c(**bad) == SHAPE, bad
    assert c(batch=0, table=NUL) == OK
    for name in ("q", "codes", "scales", "table", "ctx", "starts", "tables", "ctx_out"):
        assert c(**{name: NUL}) == NULL, name
        assert c(**{name: ODD}) == ALIGN, name
    # keys of heads that have a workgroup each stay on the chip
    assert (L.tq_select_pages_workspace_bytes(64, 8, 256) ==
            L.tq_select_pages_workspace_bytes(4096, 8, 256) <= (1 << 20) + 128 * 256 * 4)
    need = L.tq_select_pages_workspace_bytes(2, 2, 40)
    assert need > 1 << 20
    assert c(ws=NUL) == NULL and c(ws_bytes=need - 1) == SHAPE and c(ws=A4) == ALIGN


def test_attention_heads(L):
    """The entry with a table for each key head refuses as the other one."""
    good = attention(L).good
    args = {}
    for k, v in good.items():
        args[k] = v
        if k == "table_stride":
            args["head_stride"] = 4
    c = Call(L.tq_tree_attention_heads, **args)
    for bad in (dict(head_stride=-1), dict(head_stride=(1 << 40) + 1), dict(table_stride=3),
                dict(heads=7), dict(D=112), dict(scale=0.0)):
        assert c(**bad) == SHAPE, bad
    assert c(type=3) == TYPE and c(tokens=0, q=NUL) == OK
    assert c(table=NUL) == NULL and c(table=ODD) == ALIGN


def test_binding_refuses():
    import block_quantized_matmul_repack_amd as tq
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 64)
    calls = (lambda: tq.plan_step(i, i, i, i[None], i, i[:1], 16, 4),
             lambda: tq.release_pages(i, i, i[None], i, i[:1]),
             lambda: tq.residual_norm(f, f, f[0]),
             lambda: tq.sample(f, f[0]),
             lambda: tq.sample_probs(f),
             lambda: tq.cache_bounds(tq.Q8_0, i.byte(), i[None], i, i, 2, 64, 16, i, i),
             lambda: tq.select_pages(f[None].bfloat16(), i, i, i[None], i, i, 16, 2))
    for call in calls:
        with pytest.raises(tq.TiledqError):
            call()


def numbers(args):
    """Arguments as plain numbers: addresses, and 0 for none."""
    return [0 if a is None else a.value if isinstance(a, ctypes.c_void_p) else a for a in args]


@pytest.mark.parametrize("make", [attention, plan, release, residual, sample, probs, bounds, select])
def test_packed_is_the_same_call(L, make):
    """Each argument replaced by one that is refused gives the same status
    packed and unpacked; so do calls that cannot be packed."""
    c = make(L)
    packed = c.fn
    assert type(packed).__name__ == "_Packed"
    kinds = dict(zip(c.good, packed.plain.argtypes))
    seen = set()
    for name, kind in kinds.items():
        # (a good call is left out: it would be launched)
        for bad in ([float("nan"), -1.0, float("inf")] if kind is ctypes.c_float else
                    [None, ODD] if kind is ctypes.c_void_p else [-1, 1 << 62, 7]):
            kw = {**c.good, name: bad}
            if kind is ctypes.c_int and bad == 1 << 62:
                continue                         # not a number of that type
            # an output is missing besides, so nothing is ever launched
            off = next(o for o in ("new_lens", "left", "x_out", "u", "probs", "codes", "tables", "out")
                       if kinds.get(o) is ctypes.c_void_p)
            if off != name:
                kw[off] = None
            plain = packed.plain(*kw.values())
            assert plain in (OK, NULL, TYPE, SHAPE, ALIGN)
            if plain == OK:
                continue                         # nothing to do
            assert packed(*numbers(kw.values())) == plain, (name, bad)
            assert packed(*kw.values()) == plain, (name, bad)
            seen.add(plain)
    assert len(seen) > 1
    assert L.tq_packed(packed.which, None) == NULL


def test_packed_refuses_other_calls(L):
    for which in (-1, 9, 1 << 20):
        assert L.tq_packed(which, bytes(8 * 40)) == TYPE


def test_default_streams_of_other_devices(monkeypatch):
    """The null stream's handle says nothing of its device: asked for with
    another device current, the call is refused."""
    import block_quantized_matmul_repack_amd as tq
    from block_quantized_matmul_repack_amd import ops
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    assert ops._stream_of(0) == 0
    with pytest.raises(tq.TiledqError, match="current"):
        ops._stream_of(1)
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 64 + dev)
    assert ops._stream_of(1) == 65
