"""tq_cache_write / tq_cache_read against the block formats' definition: every
value read back is exactly the one its block stands for (in fp32 without
rounding, in 16 bits rounded once)."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu
KINDS = ("q8_0", "q4_0")


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_repack_amd as tq
    tq.lib()
    return tq


def ctype(tq, kind):
    return {"q8_0": tq.Q8_0, "q4_0": tq.Q4_0}[kind]


def new_cache(tq, kind, pages, P, H, D, fill=0xFF):
    n = tq.cache_bytes(ctype(tq, kind), pages, P, H, D)
    assert n > 0
    return [torch.full((n,), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]


def values(kind, x):
    return torch.from_numpy(ref.cache_values(kind, x.float().cpu().numpy()))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,H,P,T", [(64, 3, 16, 37), (96, 1, 32, 50), (128, 8, 64, 70),
                                     (256, 2, 1024, 5), (128, 1, 16, 1)])
def test_values(tq, kind, dt, D, H, P, T):
    g = torch.Generator().manual_seed(D + T)
    pages = 2 * (-(-T // P)) + 2
    k = torch.randn((T, H, D), generator=g).to(ref.DTYPES[dt]).cuda()
    v = (0.01 * torch.randn((T, H, D), generator=g)).to(ref.DTYPES[dt]).cuda()
    slots = torch.randperm(pages * P, generator=g)[:T].int().cuda()
    kc, vc = new_cache(tq, kind, pages, P, H, D)
    tq.cache_write(ctype(tq, kind), k, v, kc, vc, slots, P)
    rk, rv = tq.cache_read(ctype(tq, kind), kc, vc, slots, H, D, P)
    wk, wv = values(kind, k), values(kind, v)
    assert torch.equal(rk.cpu().double(), wk) and torch.equal(rv.cpu().double(), wv)
    for out in (torch.bfloat16, torch.float16):
        rk, rv = tq.cache_read(ctype(tq, kind), kc, vc, slots, H, D, P, dtype=out)
        assert torch.equal(rk.cpu(), wk.float().to(out)) and torch.equal(rv.cpu(), wv.float().to(out))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_runs_of_slots(tq, kind, D):
    """Consecutive slots from every offset inside a group of four, runs that
    end inside one, and neighbours left as they were."""
    H, P = 2, 16
    for first in range(5):
        for T in (1, 3, 4, 5, 8, 23):
            kc, vc = new_cache(tq, kind, 3, P, H, D, fill=0)
            g = torch.Generator().manual_seed(first * 100 + T)
            k = torch.randn((T, H, D), generator=g).bfloat16().cuda()
            v = torch.randn((T, H, D), generator=g).bfloat16().cuda()
            every = torch.arange(3 * P, dtype=torch.int32).cuda()
            base = torch.randn((3 * P, H, D), generator=g).cuda()
            tq.cache_write(ctype(tq, kind), base, base, kc, vc, every, P)
            slots = torch.arange(first, first + T, dtype=torch.int32).cuda()
            tq.cache_write(ctype(tq, kind), k, v, kc, vc, slots, P)
            want_k, want_v = values(kind, base), values(kind, base)
            want_k[first:first + T] = values(kind, k)
            want_v[first:first + T] = values(kind, v)
            rk, rv = tq.cache_read(ctype(tq, kind), kc, vc, every, H, D, P)
            assert torch.equal(rk.cpu().double(), want_k), (first, T)
            assert torch.equal(rv.cpu().double(), want_v), (first, T)


@pytest.mark.parametrize("kind", KINDS)
def test_hard_blocks(tq, kind):
    """Zeros, one element, both signs at the maximum, ties, infinities, NaN,
    magnitudes past the limit, scales that are fp16 subnormal or round to 0."""
    rows = []
    for b in ([0.0] * 32, [0.0] * 31 + [3.0], [1.0, -1.0] * 16, [-1.0, 1.0] * 16,
              list(np.linspace(-1, 1, 32)), [0.5 * i for i in range(32)],
              [float("nan")] + [1.0] * 31, [float("inf"), -2.0] * 16,
              [-float("inf"), float("nan")] * 16, [7e4] + [-3e4] * 31, [1e30, 1.0] * 16,
              [65472.0, 65504.0] * 16, [1e-4, -3e-5] * 16, [1e-6] * 32, [1e-20, 1e-21] * 16,
              [-0.0] * 32, [127.0, 63.5, -63.5, 0.5] * 8, [-8.0, 0.5, 1.5, -0.5] * 8):
        rows.append(b)
    x = torch.tensor(rows, dtype=torch.float32).reshape(len(rows) // 2, 1, 64).cuda()
    slots = torch.arange(x.shape[0], dtype=torch.int32).cuda()
    kc, vc = new_cache(tq, kind, 1, 16, 1, 64)
    tq.cache_write(ctype(tq, kind), x, x, kc, vc, slots, 16)
    rk, rv = tq.cache_read(ctype(tq, kind), kc, vc, slots, 1, 64, 16)
    want = values(kind, x)
    assert torch.equal(rk.cpu().double(), want) and torch.equal(rv.cpu().double(), want)
    assert bool(torch.isfinite(rk.half()).all())


@pytest.mark.parametrize("kind", KINDS)
def test_ties_agree_with_quantize_act(tq, kind):
    """Every bf16 of an octave against a maximum of 127 or 8: halves fall on
    the rounding borders."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randint(-254, 255, (64, 1, 128), generator=g) * 0.5).cuda()
    slots = torch.arange(64, dtype=torch.int32).cuda()
    kc, vc = new_cache(tq, kind, 4, 16, 1, 128)
    tq.cache_write(ctype(tq, kind), x, x, kc, vc, slots, 16)
    rk, _ = tq.cache_read(ctype(tq, kind), kc, vc, slots, 1, 128, 16)
    assert torch.equal(rk.cpu().double(), values(kind, x))
    if kind == "q8_0":
        q, d = tq.quantize_act(x.view(64, 128))
        same = (q.view(64, 4, 32).float() * d.float().unsqueeze(-1)).view(64, 1, 128)
        assert torch.equal(rk, same)


@pytest.mark.parametrize("kind", KINDS)
def test_slots_outside_are_skipped_and_read_as_zeros(tq, kind):
    H, D, P, pages = 1, 64, 16, 2
    n = pages * P
    kc, vc = new_cache(tq, kind, pages, P, H, D, fill=0)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((6, H, D), generator=g).cuda()
    slots = torch.tensor([-1, 3, n, n - 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    tq.cache_write(ctype(tq, kind), x, x, kc, vc, slots, P)
    rk, rv = tq.cache_read(ctype(tq, kind), kc, vc, slots, H, D, P)
    want = values(kind, x)
    want[[0, 2, 4, 5]] = 0
    assert torch.equal(rk.cpu().double(), want) and torch.equal(rv.cpu().double(), want)


def test_strided_sources(tq):
    """Keys and values as column ranges of a fused projection, and heads first."""
    T, H, D, P = 19, 2, 96, 32
    qkv = torch.randn((T, 4 * H * D), generator=torch.Generator().manual_seed(6)).half().cuda()
    k = qkv[:, H * D:2 * H * D].unflatten(1, (H, D))
    v = qkv[:, 2 * H * D:3 * H * D].unflatten(1, (H, D))
    slots = torch.arange(7, 7 + T, dtype=torch.int32).cuda()
    kc, vc = new_cache(tq, "q8_0", 1, P, H, D)
    tq.cache_write(tq.Q8_0, k, v.transpose(0, 1).contiguous().transpose(0, 1), kc, vc, slots, P)
    rk, rv = tq.cache_read(tq.Q8_0, kc, vc, slots, H, D, P)
    assert torch.equal(rk.cpu().double(), values("q8_0", k))
    assert torch.equal(rv.cpu().double(), values("q8_0", v))


def test_offsets_past_32_bits(tq):
    """A cache of 4.6 GB a buffer: the last page's bytes lie past 2^32."""
    H, D, P = 8, 256, 64
    page = tq.cache_bytes(tq.Q8_0, 1, P, H, D)
    pages = (1 << 32) // page + 300
    kc = torch.empty(pages * page, dtype=torch.uint8, device="cuda")
    vc = torch.empty(pages * page, dtype=torch.uint8, device="cuda")
    T = 40
    x = torch.randn((T, H, D), generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    slots = (pages * P - T + torch.arange(T)).int().cuda()
    tq.cache_write(tq.Q8_0, x, x, kc, vc, slots, P)
    rk, rv = tq.cache_read(tq.Q8_0, kc, vc, slots, H, D, P)
    want = values("q8_0", x)
    assert torch.equal(rk.cpu().double(), want) and torch.equal(rv.cpu().double(), want)
