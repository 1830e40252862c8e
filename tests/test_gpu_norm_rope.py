"""tq_qk_norm_rope against its fp64 definition.

Tolerance: half a step of the output's type, plus 32 * 2^-24 of |a| + |b|,
the magnitudes a rotated output is combined from: the mean of squares (at
most 24 fp32 additions in a chain, halved by the square root), root,
quotient and two products, sine and cosine (2 steps and the fp32 rounding of
an angle in [-pi, pi]), and the two products and the sum of the rotation."""
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    tq.lib()
    return tq


def check(y, x, w, eps, pos, freq, interleaved):
    want, mag = ref.norm_rope(x.cpu(), None if w is None else w.cpu(), eps, pos.cpu(),
                              freq.cpu(), interleaved)
    tol = ref.half_step(y.dtype) * want.abs() + 32 * 2.0 ** -24 * mag + 1e-30
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25                            # half a subnormal step
    bad = (y.cpu().double() - want).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


def freqs(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1, 32, 8, 128, 128),      # one token: a wave per group of heads
    (5, 3, 1, 64, 64),
    (33, 12, 3, 96, 48),       # half rotated
    (700, 7, 1, 80, 80),       # 5 units of 16: idle lanes
    (9, 2, 2, 256, 64),
    (4, 5, 1, 34, 10),         # halves that are no whole eights: single elements
    (3, 1, 1, 512, 510),       # the same, four units a lane
    (6, 4, 2, 2, 2),
    (2, 3, 2, 128, 0),         # norm only
    (3, 0, 4, 64, 64),         # keys only
])
def test_matches_definition(tq, dt, T, Hq, Hk, D, rot):
    for interleaved in (False, True):
        for norm in (True, False):
            g = torch.Generator().manual_seed(T * 131 + D + rot)
            dtype = ref.DTYPES[dt]
            q = torch.randn((T, Hq, D), generator=g).to(dtype).cuda()
            k = (3 * torch.randn((T, Hk, D), generator=g)).to(dtype).cuda()
            wq = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if norm else None
            wk = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if norm else None
            pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32).cuda()
            f = freqs(rot // 2)
            yq, yk = tq.qk_norm_rope(q, k, pos, f, wq, wk, eps=1e-5, interleaved=interleaved)
            check(yq, q, wq, 1e-5, pos, f, interleaved)
            check(yk, k, wk, 1e-5, pos, f, interleaved)


def test_extreme_positions_and_rows(tq):
    """Positions over the whole int32 range; rows of zeros, tiny and large
    elements; fp32 weights on bf16 heads."""
    pos = torch.tensor([0, -1, 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(3)
    q = torch.randn((6, 4, 128), generator=g)
    q[0] = 0
    q[1] *= 1e-12
    q[2] *= 1e15
    q = q.bfloat16().cuda()
    k = torch.randn((6, 1, 128), generator=g).bfloat16().cuda()
    w = torch.randn(128, generator=g).cuda()
    f = freqs(64)
    yq, yk = tq.qk_norm_rope(q, k, pos, f, w, w)
    check(yq, q, w, 1e-6, pos, f, False)
    check(yk, k, w, 1e-6, pos, f, False)


def test_views_and_in_place(tq):
    """q and k as column ranges of one fused projection, rotated in place."""
    T, Hq, Hk, D = 21, 6, 2, 64
    qkv = torch.randn((T, (Hq + 2 * Hk) * D + 3), generator=torch.Generator().manual_seed(9))
    qkv = qkv.bfloat16().cuda()
    before = qkv.clone()
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.arange(100, 100 + T, dtype=torch.int32).cuda()
    f = freqs(32)
    w = torch.full((D,), 1.5).bfloat16().cuda()
    yq, yk = tq.qk_norm_rope(q, k, pos, f, w, w)
    rq, rk = tq.qk_norm_rope(q, k, pos, f, w, w, q_out=q, k_out=k)
    assert rq.data_ptr() == qkv.data_ptr()
    assert torch.equal(rq, yq) and torch.equal(rk, yk)
    assert torch.equal(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    # heads outermost: [H, T, D] storage seen as [T, H, D]
    ht = torch.empty((Hq, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    q0 = before[:, :Hq * D].unflatten(1, (Hq, D))
    k0 = before[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    assert torch.equal(tq.qk_norm_rope(q0, k0, pos, f, w, w, q_out=ht)[0], yq)
    check(yq, q0, w, 1e-6, pos, f, False)


def test_empty(tq):
    q = torch.empty((0, 4, 64), device="cuda")
    y, _ = tq.qk_norm_rope(q, q, torch.empty(0, dtype=torch.int32, device="cuda"), freqs(32))
    assert y.shape == (0, 4, 64)
