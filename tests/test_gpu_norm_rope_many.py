"""tq_qk_norm_rope with so many tokens that a wave takes several of a token's
heads, and token counts on both sides of where that begins."""
import pytest
import torch

import decode_ref as ref
from test_gpu_norm_rope import check, freqs, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1638, 1639, 8192, 8193, 16385, 30011])
@pytest.mark.parametrize("Hq,Hk,D,rot,dt", [(32, 8, 128, 128, "bf16"), (40, 9, 128, 64, "fp16"),
                                            (5, 2, 72, 72, "bf16"), (12, 4, 36, 18, "fp32"),
                                            (1, 0, 64, 64, "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens(tq, T, Hq, Hk, D, rot, dt, interleaved):
    """Every head of sampled tokens (the first, the last, some between)
    against the definition; every output is written."""
    g = torch.Generator().manual_seed(T + D)
    dtype = ref.DTYPES[dt]
    rows = sorted({0, 1, T // 2, T - 2, T - 1} | set(torch.randint(0, T, (40,), generator=g).tolist()))
    x = torch.randn((T, Hq + Hk, D), generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    freq = freqs(rot // 2)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda()
    dev = x.cuda()
    out = torch.full_like(dev, float("nan"))
    tq.qk_norm_rope(dev[:, :Hq], dev[:, Hq:], pos.cuda(), freq, w, w, interleaved=interleaved,
                    q_out=out[:, :Hq], k_out=out[:, Hq:])
    assert not bool(out.isnan().any())
    check(out[torch.tensor(rows).cuda()], x[rows], w, 1e-6, pos[rows], freq, interleaved)
