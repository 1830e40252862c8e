"""tq_verify_draft with draft rows that hold more than probabilities: NaN and
negative entries count as 0, and a row that nothing was drawn from (the last
accepted node's has no children) has no say whatever it holds."""
import numpy as np
import pytest
import torch

import decode_ref as ref
from test_gpu_verify import call, make, tq  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [(False, False), (True, False), (False, True), (True, True)]


def check(tq, m, width=None):
    """As test_gpu_verify.check, the definition's rule for NaN and negative
    draft probabilities applied before the walk."""
    counts = np.diff(m["starts"])
    width = int(max(counts.max(), 1)) if width is None else width
    got = [t.cpu().numpy() for t in call(tq, m, width)]
    q = m["q"].double().numpy()
    q = np.where(q > 0, q, 0.0)
    accepted = 0
    for b in range(len(counts)):
        s = slice(m["starts"][b], m["starts"][b + 1])
        k, t, nd = ref.verify(m["p"][s].double().numpy(), q[s], m["tokens"][s],
                              None if m["parents"] is None else m["parents"][s], m["u"][s],
                              m["r"][b], width)
        assert got[0][b] == k, b
        assert got[1][b].tolist() == t and got[2][b].tolist() == nd, b
        accepted += k
    return accepted


def leaves(m):
    """The rows whose nodes have no child."""
    out = []
    for a, e in zip(m["starts"][:-1], m["starts"][1:]):
        par = m["parents"][a:e] if m["parents"] is not None else np.arange(e - a) - 1
        out += [a + i for i in range(e - a) if i not in par[1:].tolist()]
    return out


@pytest.mark.parametrize("V", [65, 2049, 40001])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("fill", ["nan", "inf", "-inf", "-1", "uninitialised"])
def test_rows_without_children(tq, V, tree, fill):
    """All drafted tokens accepted, so that the next token comes from a leaf."""
    m = make(V, [5, 3, 1], V, tree, True, branch=2)
    m["q"] = m["p"].clone()                      # u * q < p: the first child is always accepted
    rows = leaves(m)
    if fill == "uninitialised":
        bits = np.random.default_rng(3).integers(0, 2 ** 32, (len(rows), V), dtype=np.uint32)
        m["q"][rows] = torch.from_numpy(bits.view(np.float32))
    else:
        m["q"][rows] = float(fill)
    assert check(tq, m) > 0
    _, tokens, _ = call(tq, m, 5)
    assert bool((tokens[:, 0] >= 0).all())


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seed", range(4))
def test_nan_and_negative_entries(tq, tree, dtype, seed):
    m = make(50 + seed, [9, 4, 12, 2], 777, tree, True, dtype=dtype)
    rng = np.random.default_rng(seed)
    kind = rng.integers(0, 5, m["q"].shape)
    m["q"][torch.from_numpy(kind == 0)] = float("nan")
    m["q"][torch.from_numpy(kind == 1)] *= -1.0
    check(tq, m)
    # the drafted tokens' own entries, too
    for n in range(len(m["tokens"])):
        m["q"][:, m["tokens"][n]] = float("nan") if n % 2 else -0.25
    check(tq, m)


@pytest.mark.parametrize("tree", [False, True])
def test_negative_draft_accepts_nothing_impossible(tq, tree):
    """u * q < 0 for a token that the target rules out."""
    m = make(60, [7, 7], 64, tree, True)
    m["p"][:, :32] = 0
    m["tokens"] = (m["tokens"] % 32).astype(np.int32)
    m["q"][:, :32] = -0.5
    m["u"][:] = 0.75
    assert check(tq, m) == 0


@pytest.mark.parametrize("tree", [False, True])
def test_whole_rows_of_nothing(tq, tree):
    """Draft rows that are NaN all over: w - 0 stays w, and a token comes out."""
    m = make(61, [7, 5], 300, tree, True)
    m["q"][:] = float("nan")
    m["u"][:] = 0.5
    check(tq, m)
    m["p"][:, 7] = 0
    m["tokens"][:] = 7                           # refused: nothing of the target there
    assert check(tq, m) == 0
