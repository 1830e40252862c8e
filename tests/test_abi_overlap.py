"""Outputs of the serving-step operators that lie in their inputs or in each other
are refused before any HIP call (no GPU, the addresses are never read)."""
import ctypes

import pytest

from test_abi_decode import NUL, SHAPE
from test_abi_serving import P, residual


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
