"""The norms around a block with gate and residual scale, in one pass.

Tolerances.  x' is one rounding of a sum whose terms carry fp32 errors: the
mean of up to 2^15 squares is summed in runs of at most 32, then over lanes and
waves in 6 + 16 steps, so it errs by less than 64 * 2^-24 relative, its root by
half of that, and a handful of products and the sum add 2^-24 each: 2^-18 of
the terms' size covers them.  z is compared with the norm of the x' that came
out, so it has the same errors of its own.  fp16 adds half a subnormal step,
2^-25."""
import pytest
import torch

import serving_ref as ref
from decode_ref import DTYPES, half_step

pytestmark = pytest.mark.gpu
EPS = 1e-6


def tq():
    import block_quantized_matmul_repack_amd as m
    return m


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(T, N, ydt, dt, wdt, post, pre, gate, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + N)

    def rand(*s):
        return torch.randn(s, generator=g)

    y, x = (3 * rand(T, N)).to(DTYPES[ydt]).cuda(), rand(T, N)
    x[:, ::7] *= 30
    x = x.to(DTYPES[dt]).cuda()
    w = [((1 + 0.3 * rand(N)).to(DTYPES[wdt]).cuda() if on else None) for on in (post, pre)]
    shape = {"none": None, "channel": (N,), "token": (T, N), "row": (T, 1), "one": (1,)}[gate]
    gt = None if shape is None else rand(*shape).to(DTYPES[wdt]).cuda()
    return y, x, *w, gt


def check(y, x, post, pre, gate, scale, xo, z, eps=EPS):
    dt = x.dtype
    sub = 2.0 ** -25 if dt is torch.float16 else 0.0
    want, mag = ref.residual(np64(y), np64(x), np64(post), np64(gate), scale, eps)
    got = np64(xo)
    assert (abs(got - want) <= half_step(dt) * abs(want) * 1.01 + 2.0 ** -18 * mag + sub).all()
    zr = got if pre is None else ref.rms(got, np64(pre), eps)
    if isinstance(z, tuple):
        q, d = z
        zq = (q.double().unflatten(-1, (-1, 32)) * d.double()[..., None]).flatten(-2).cpu().numpy()
        big = abs(zr).reshape(len(zr), -1, 32).max(-1, keepdims=True).repeat(32, -1).reshape(zr.shape)
        # half a step of the codes, the scale's rounding (fp16; 2^-25 where it is
        # subnormal, times a code), and z's own
        tol = 0.5 * big / 127 * (1 + 2.0 ** -9) + abs(zr) * (2.0 ** -11 + 2.0 ** -17) + 127 * 2.0 ** -25
        assert (abs(zq - zr) <= tol).all()
    else:
        tol = half_step(dt) * abs(zr) * 1.01 + 2.0 ** -18 * abs(zr) + sub
        assert (abs(np64(z) - zr) <= tol).all()


@pytest.mark.parametrize("N", [1, 2, 7, 8, 31, 64, 511, 512, 513, 1500, 2048, 2049, 4096, 4100,
                               8192, 8193, 16384, 20000, 32768])
@pytest.mark.parametrize("T", [1, 5])
def test_sizes(T, N):
    y, x, post, pre, gate = inputs(T, N, "fp32", "bf16", "bf16", True, True, "channel")
    check(y, x, post, pre, gate, 0.75, *tq().residual_norm(y, x, pre, post, gate, 0.75, EPS))


@pytest.mark.parametrize("ydt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("wdt", ["fp32", "bf16", "fp16"])
def test_types(ydt, dt, wdt):
    y, x, post, pre, gate = inputs(9, 1056, ydt, dt, wdt, True, True, "token")
    check(y, x, post, pre, gate, 1.0, *tq().residual_norm(y, x, pre, post, gate, eps=EPS))
    xo, z = tq().residual_norm(y, x, pre, post, gate, eps=EPS, quantize=True)
    check(y, x, post, pre, gate, 1.0, xo, z)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "row", "one"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
def test_forms(gate, post, pre):
    for dt, T, N in (("fp16", 33, 96), ("bf16", 3, 2600)):
        y, x, wp, wq, g = inputs(T, N, "fp32", dt, dt, post, pre, gate)
        check(y, x, wp, wq, g, -0.5, *tq().residual_norm(y, x, wq, wp, g, -0.5, EPS))


@pytest.mark.parametrize("T,N", [(6200, 513), (4099, 1504), (1100, 4100), (1031, 5120), (520, 8192),
                                 (513, 7993), (3001, 2048)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "row"])
def test_many_tokens(T, N, gate):
    """Workgroups that go through several tokens; the same bits as a few at a time."""
    dts = {"none": ("fp32", "bf16"), "channel": ("bf16", "fp16"), "token": ("fp16", "fp32"),
           "row": ("bf16", "bf16")}[gate]
    y, x, post, pre, g = inputs(T, N, *dts, "bf16", gate != "row", gate != "none", gate)
    xo, z = tq().residual_norm(y, x, pre, post, g, 0.7, EPS)
    check(y, x, post, pre, g, 0.7, xo, z)
    for a in range(0, T, 200):
        part = slice(a, a + 200)
        gp = g[part] if gate in ("token", "row") else g
        few = tq().residual_norm(y[part], x[part], pre, post, gp, 0.7, EPS)
        assert torch.equal(few[0], xo[part]) and torch.equal(few[1], z[part]), a
    if N % 32 == 0:
        xq, (q, d) = tq().residual_norm(y, x, pre, post, g, 0.7, EPS, quantize=True)
        assert torch.equal(xq, xo)
        check(y, x, post, pre, g, 0.7, xq, (q, d))
    own = x.clone()
    tq().residual_norm(y, own, pre, post, g, 0.7, EPS, x_out=own)
    assert torch.equal(own, xo)


@pytest.mark.parametrize("N", [32, 64, 96, 512, 544, 2048, 4096, 5120, 8224, 32768])
def test_quantized_as_the_products_do(N):
    """q and d are tq_quantize_act's of the fp32 z, bit for bit."""
    y, x, post, pre, gate = inputs(6, N, "fp32", "fp32", "bf16", True, True, "channel")
    xo, z = tq().residual_norm(y, x, pre, post, gate, 0.9, EPS)
    xq, (q, d) = tq().residual_norm(y, x, pre, post, gate, 0.9, EPS, quantize=True)
    q_want, d_want = tq().quantize_act(z)
    assert torch.equal(xq, xo) and torch.equal(q, q_want) and torch.equal(d, d_want)


def test_strides_and_places():
    """Rows of wider tensors at odd offsets, x' in x's place, outputs given; what
    lies beside them stays."""
    y, x, post, pre, gate = inputs(7, 100, "fp16", "bf16", "bf16", True, True, "token")
    want = tq().residual_norm(y, x, pre, post, gate, eps=EPS)
    big = torch.full((7, 131), 5.0, dtype=torch.bfloat16, device="cuda")
    xv, zv = big[:, 3:103], torch.full((7, 117), 6.0, dtype=torch.bfloat16, device="cuda")
    xv.copy_(x)
    yv = torch.zeros((7, 111), dtype=torch.float16, device="cuda")[:, 5:105]
    yv.copy_(y)
    gv = torch.zeros((7, 109), dtype=torch.bfloat16, device="cuda")[:, 1:101]
    gv.copy_(gate)
    xo, z = tq().residual_norm(yv, xv, pre, post, gv, eps=EPS, x_out=xv, z_out=zv[:, 9:109])
    assert xo is xv and torch.equal(xv, want[0]) and torch.equal(z, want[1])
    assert (big[:, :3] == 5).all() and (big[:, 103:] == 5).all()
    assert (zv[:, :9] == 6).all() and (zv[:, 109:] == 6).all()


def test_rows_are_apart():
    """A row of infinities or NaN, or of zeros, does not touch the others."""
    y, x, post, pre, gate = inputs(6, 640, "fp32", "bf16", "bf16", True, True, "channel")
    want = tq().residual_norm(y, x, pre, post, gate, eps=EPS)
    y[1, 5], y[3, 600], x[4, 1] = float("inf"), float("nan"), float("inf")
    y[5] = 0
    x[5] = 0
    xo, z = tq().residual_norm(y, x, pre, post, gate, eps=EPS)
    for r in (0, 2):
        assert torch.equal(xo[r], want[0][r]) and torch.equal(z[r], want[1][r])
    assert (xo[5] == 0).all() and (z[5] == 0).all()
    assert z[1].isnan().any() and z[3].isnan().any() and z[4].isnan().any()


def test_no_tokens_and_refusals():
    y, x, post, pre, _ = inputs(4, 64, "fp32", "bf16", "bf16", True, True, "none")
    xo, z = tq().residual_norm(y[:0], x[:0], pre, post)
    assert xo.shape == z.shape == (0, 64)
    for bad in (dict(y=y[:3]), dict(x=x.t()), dict(pre_weight=pre[:32]), dict(pre_weight=pre.float()),
                dict(gate=pre[None].expand(3, 64)), dict(gate=pre.float()), dict(y=y.cpu()),
                dict(x_out=x[:, :32]), dict(z_out=z), dict(scale=float("inf")), dict(eps=-1.0)):
        with pytest.raises(tq().TiledqError):
            tq().residual_norm(**{**dict(y=y, x=x, pre_weight=pre, post_weight=post), **bad})
    with pytest.raises(tq().TiledqError):
        tq().residual_norm(y[:, :40], x[:, :40], quantize=True)
