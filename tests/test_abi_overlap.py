"""Outputs of the serving-step operators that lie in their inputs or in each other
are refused before any HIP call (no GPU, the addresses are never read)."""
import ctypes

import pytest

from test_abi_decode import NUL, NULL, SHAPE
from test_abi_serving import P, probs, residual, sample


@pytest.fixture(scope="module")
def L():
    from block_quantized_matmul_repack_amd import _lib
    return _lib.lib()


def at(p, offset):
    return ctypes.c_void_p(p.value + offset)


# the arrays of a call with tokens 3, N 64: y fp32 (256 bytes a row), the rest bf16 (128)
APART = dict(y=P(0), x=P(1), post=P(2), pre=P(3), gate=P(4), gate_ts=64, x_out=P(5), z=P(6))


@pytest.mark.parametrize("name", ["x_out", "z"])
@pytest.mark.parametrize("other,size", [("y", 768), ("x", 384), ("post", 128), ("pre", 128),
                                        ("gate", 384)])
def test_residual_norm_outputs_in_inputs(L, name, other, size):
    c = residual(L, **APART)
    for offset in (0, 2, size // 2, size - 2, -2, -128, 2 - 384):
        if (name, other, offset) == ("x_out", "x", 0):
            continue                             # in place
        assert c(**{name: at(APART[other], offset)}) == SHAPE, (name, other, offset)


def test_residual_norm_shifted_in_place(L):
    """x' in x's place a row further, or z there."""
    c = residual(L, **APART)
    assert c(x_out=at(APART["x"], 128)) == SHAPE and c(x_out=at(APART["x"], -256)) == SHAPE
    assert c(x_out=APART["x"], z=APART["x"]) == SHAPE
    assert c(x_out=APART["x"], z=at(APART["x"], 128)) == SHAPE
    assert c(x_out=APART["x"], z=APART["x"], pre=NUL, z_ts=80) == SHAPE
    # a wider row stride: columns of one buffer, of which the second begins in the first
    assert c(x_ts=128, xo_ts=128, x_out=at(APART["x"], 126)) == SHAPE
    assert c(x_ts=128, xo_ts=128, x_out=at(APART["x"], 130)) == SHAPE
    # strides that differ: row 2 of x' (from byte 2 * 192) meets row 1 of x at 256
    assert c(x_ts=128, xo_ts=96, x_out=at(APART["x"], 128)) == SHAPE
    # one row for all tokens
    assert c(y_ts=0, x_out=at(APART["y"], 254)) == SHAPE


def test_residual_norm_outputs_in_outputs(L):
    c = residual(L, **APART)
    for offset in (0, 2, 382, -382):
        assert c(z=at(APART["x_out"], offset)) == SHAPE, offset
    # without a weight z is x', and may be the same array, not a shifted one
    assert c(z=at(APART["x_out"], 128), pre=NUL) == SHAPE
    assert c(z=APART["x_out"], z_ts=65, pre=NUL) == SHAPE
    c = residual(L, **{**APART, "z": NUL, "q": P(7), "d": P(8)})
    for bad in (dict(q=APART["x"]), dict(q=at(APART["y"], 764)), dict(d=at(APART["gate"], 382)),
                dict(q=at(APART["x_out"], 380)), dict(d=at(APART["x_out"], -10)),
                dict(d=at(P(7), 190)), dict(q=at(P(8), 8)), dict(d=APART["pre"])):
        assert c(**bad) == SHAPE, bad


# arrays of 8200 logits a row, which takes a workspace: without one a call that gets past
# the comparison of its arrays is refused as NULL
V = 8200
SETTINGS = dict(temp=P(10), top_k=P(11), top_p=P(12), min_p=P(13))


def test_sampling_outputs_in_inputs(L):
    c = sample(L)
    c.good.update(SETTINGS, vocab=V, stride=V, rows=3, logits=P(0), u=P(14), tokens=P(15), ws=NUL)
    assert c() == NULL
    for name in (*SETTINGS, "u"):
        for offset in (0, 8, -8):
            assert c(tokens=at(c.good[name], offset)) == SHAPE, (name, offset)
        assert c(tokens=at(c.good[name], 12)) == NULL == c(tokens=at(c.good[name], -12))
    for offset in (-8, 0, 4 * V, 12 * V - 4):
        assert c(tokens=at(P(0), offset)) == SHAPE, offset
    assert c(tokens=at(P(0), 12 * V)) == NULL == c(tokens=at(P(0), -12))
    # behind each row's logits, where the stride leaves room
    assert c(stride=V + 3, tokens=at(P(0), 4 * V)) == NULL
    assert c(stride=V + 2, tokens=at(P(0), 4 * V)) == SHAPE
    c = probs(L)
    c.good.update(SETTINGS, vocab=V, stride=V, rows=3, logits=P(0), probs=P(15), probs_stride=V,
                  ws=NUL)
    assert c() == NULL
    for name in SETTINGS:
        assert c(probs=c.good[name]) == SHAPE == c(probs=at(c.good[name], 4 - 12 * V))
    # in place: fp32 at the same stride, or one row
    assert c(probs=P(0)) == NULL == c(probs=P(0), rows=1, probs_stride=V + 9)
    assert c(probs=P(0), dtype=1) == SHAPE == c(probs=P(0), dtype=2)
    assert c(probs=P(0), probs_stride=V + 1) == SHAPE == c(probs=P(0), stride=0)
    assert c(probs=at(P(0), 4)) == SHAPE == c(probs=at(P(0), 4 * V)) == c(probs=at(P(0), -4))


def rows_meet(offset, stride_a, n_a, stride_b, n_b, rows):
    """Row i of a at i * stride_a, of b at offset + i * stride_b, all against all."""
    return any(offset + j * stride_b < i * stride_a + n_a and i * stride_a < offset + j * stride_b + n_b
               for i in range(rows) for j in range(rows))


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
def test_rows_between_rows(L, dtype, size):
    """Every place of a few strides against all pairs of rows."""
    c = probs(L)
    c.good.update(SETTINGS, vocab=V, rows=4, dtype=dtype, logits=P(0), ws=NUL)
    seen = set()
    for stride in (0, V, 2 * V, 3 * V + 1, 9 * V):
        for probs_stride in (V, V + 5, 2 * V, 3 * V + 1, 5 * V):
            for part in range(-8, 40):
                for near in (-4, 0, 4):
                    offset = part * 2 * V + near
                    want = rows_meet(offset, stride * size, V * size, probs_stride * 4, V * 4, 4)
                    if dtype == 0 and offset == 0 and stride == probs_stride:
                        want = False             # in place
                    got = c(stride=stride, probs_stride=probs_stride, probs=at(P(40), offset),
                            logits=P(40))
                    assert got == (SHAPE if want else NULL), (stride, probs_stride, offset)
                    seen.add(want)
    assert seen == {True, False}
