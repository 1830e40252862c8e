"""Arrays of one buffer that the serving-step operators take: rows between each
other's, and results in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def tq():
    import block_quantized_matmul_repack_amd as m
    return m


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("T,N", [(1, 64), (5, 100), (70, 4096), (3000, 1024)])
def test_residual_norm_columns_of_one_buffer(T, N):
    """y, x, the gate and both outputs are columns of one buffer."""
    y, x, gate, w = randn(T, N, seed=1), randn(T, N, seed=2), randn(T, N, seed=3), randn(N)
    want = tq().residual_norm(y, x, w, post_weight=w, gate=gate)
    buf = torch.full((T, 5 * N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    cols = [buf[:, i * N:(i + 1) * N] for i in range(5)]
    for c, t in zip(cols, (y, x, gate)):
        c.copy_(t)
    got = tq().residual_norm(cols[0], cols[1], w, post_weight=w, gate=cols[2], x_out=cols[3],
                             z_out=cols[4])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(cols[0], y) and torch.equal(cols[1], x) and (buf[:, 5 * N:] == 7).all()
    # in place, and z over y is refused
    got = tq().residual_norm(cols[0], cols[1], w, post_weight=w, gate=cols[2], x_out=cols[1],
                             z_out=cols[4])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(tq().TiledqError):
        tq().residual_norm(cols[0], cols[1], w, x_out=cols[3], z_out=cols[0])


def test_residual_norm_rows_of_unlike_strides():
    """Outputs between the rows of an input that are farther apart than theirs."""
    T, N = 6, 32
    y, w = randn(T, N, seed=1), randn(N)
    x = torch.zeros(1000, dtype=torch.bfloat16, device="cuda").as_strided((T, N), (160, 1))
    x.copy_(randn(T, N, seed=2))
    want = tq().residual_norm(y, x.contiguous(), w)
    # rows of 32 every 40 elements from 32 on: three between two rows of x, the fourth past its next
    z = x.as_strided((3, N), (40, 1), 32)
    got = tq().residual_norm(y[:3], x[:3], w, z_out=z)
    assert torch.equal(got[0], want[0][:3]) and torch.equal(z, want[1][:3])
    with pytest.raises(tq().TiledqError):
        tq().residual_norm(y[:4], x[:4], w, z_out=x.as_strided((4, N), (40, 1), 32))


@pytest.mark.parametrize("T,N", [(1, 64), (9, 100), (33, 8192)])
def test_residual_norm_without_a_second_norm_may_write_one_array(T, N):
    y, x = randn(T, N, seed=4), randn(T, N, seed=5)
    want = tq().residual_norm(y, x, scale=0.5)
    one = torch.empty_like(x)
    got = tq().residual_norm(y, x, scale=0.5, x_out=one, z_out=one)
    assert got[0] is one and torch.equal(one, want[0]) and torch.equal(one, want[1])
    tq().residual_norm(y, x, scale=0.5, x_out=x, z_out=x)
    assert torch.equal(x, want[0])


@pytest.mark.parametrize("V", [50, 8192, 20001, 128001, 600001, 1048577])
@pytest.mark.parametrize("kw", [dict(top_p=0.9), dict(top_k=40, top_p=0.8), dict(temperature=0.0), {}])
def test_distributions_in_place_of_the_logits(V, kw):
    kw = {k: torch.full((3,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
          for k, v in kw.items()}
    x = 2.5 * randn(3, V, dtype=torch.float32)
    x[1] = x[1].round()                          # thousands of equal ones
    x[2, :] = 1.0
    want = tq().sample_probs(x, **kw)
    wide = torch.full((3, V + 7), 9.0, device="cuda")
    inside = wide[:, 3:V + 3]
    inside.copy_(x)
    assert tq().sample_probs(inside, **kw, out=inside) is inside
    assert torch.equal(inside, want) and (wide[:, :3] == 9).all() and (wide[:, V + 3:] == 9).all()
    tq().sample_probs(x, **kw, out=x)
    assert torch.equal(x, want)
    with pytest.raises(tq().TiledqError):
        tq().sample_probs(wide[:, :V], **kw, out=wide[:, 1:V + 1])
