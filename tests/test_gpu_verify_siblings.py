"""tq_verify_draft without draft probabilities where one node has many children:
each refused token's probability is gone for the next sibling, which another
lane may have noted."""
import pytest
import torch

from test_gpu_verify import check, make, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,V,branch", [(40, 20, 39), (65, 30, 64), (130, 50, 129), (400, 90, 399),
                                        (1000, 150, 333), (300, 40, 70)])
@pytest.mark.parametrize("seed", range(3))
def test_many_siblings(tq, n, V, branch, seed):
    """Tokens come again and again among them; nearly all are refused."""
    m = make(seed + n, [n, 7, n // 2], V, True, False, branch=branch)
    m["u"][:] = 0.97 + 0.03 * m["u"]
    check(tq, m)
    m["p"] = m["p"] * 1e-3                       # so that the threshold stays near u: all refused
    check(tq, m)
    m["p"] = torch.zeros_like(m["p"])
    m["p"][:, V - 1] = 1.0                       # the last token alone is possible
    assert check(tq, m) >= 0
