"""tq_verify_draft against a sequential fp64 walk: equal whole numbers."""
import numpy as np
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


def make(seed, counts, V, tree, draft, near=0.5, dtype=torch.float32, branch=3):
    """Sequences of `counts` nodes; drafted tokens likely under the draft."""
    rng = np.random.default_rng(seed)
    N = sum(counts)
    logits = 2.0 * rng.standard_normal((N, V))
    soft = lambda z: np.exp(z - z.max(1, keepdims=True)) / np.exp(  # noqa: E731
        z - z.max(1, keepdims=True)).sum(1, keepdims=True)
    p = torch.from_numpy(soft(logits)).to(dtype) if N else torch.zeros((0, V), dtype=dtype)
    q = torch.from_numpy(soft(logits + near * rng.standard_normal((N, V)))).to(dtype) \
        if draft else None
    parents, tokens, base = [], [], 0
    for n in counts:
        for i in range(n):
            par = (max(0, (i - 1) // branch) if tree else i - 1) if i else -1
            parents.append(par)
            row = base + max(par, 0)
            w = (q if draft else p)[row].double().numpy()
            tokens.append(int(rng.choice(V, p=w / w.sum())))
        base += n
    starts = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    return dict(p=p, q=q, parents=np.array(parents, np.int32) if tree else None,
                tokens=np.array(tokens, np.int32), starts=starts,
                u=rng.random(N).astype(np.float32), r=rng.random(len(counts)).astype(np.float32))


def dev(x):
    return None if x is None else torch.as_tensor(x).cuda()


def call(tq, m, width):
    return tq.verify_draft(dev(m["p"]), dev(m["tokens"]), dev(m["starts"]), dev(m["u"]),
                           dev(m["r"]), draft=dev(m["q"]), parents=dev(m["parents"]),
                           max_nodes=width)


def check(tq, m, width=None):
    counts = np.diff(m["starts"])
    width = int(max(counts.max(), 1)) if width is None else width
    got = [t.cpu().numpy() for t in call(tq, m, width)]
    accepted = 0
    for b, n in enumerate(counts):
        s = slice(m["starts"][b], m["starts"][b + 1])
        k, t, nd = ref.verify(m["p"][s].double().numpy(),
                              None if m["q"] is None else m["q"][s].double().numpy(),
                              m["tokens"][s], None if m["parents"] is None else m["parents"][s],
                              m["u"][s], m["r"][b], width)
        assert got[0][b] == k, b
        assert got[1][b].tolist() == t and got[2][b].tolist() == nd, b
        accepted += k
    return accepted


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [1, 2, 33, 2047, 2049, 10007])
def test_walk(tq, tree, draft, V):
    acc = check(tq, make(V, [5, 9, 1, 2, 17, 3, 3, 3], V, tree, draft))
    assert acc > 0 or V > 100


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree,draft", [(False, True), (True, False), (True, True)])
def test_16_bit_probabilities(tq, dtype, tree, draft):
    check(tq, make(7, [6, 4, 8], 777, tree, draft, dtype=dtype))


def test_large_vocabulary(tq):
    for tree, draft in ((False, True), (True, False), (True, True)):
        check(tq, make(11, [4, 5], 128001, tree, draft))


def test_empty_sequences_and_no_sequences(tq):
    m = make(3, [0, 3, 0, 1, 0], 100, False, True)
    check(tq, m)
    a, t, n = call(tq, m, 3)
    assert a[0] == 0 and t[0].tolist() == [-1] * 3 and n[0].tolist() == [-1] * 3
    e = torch.empty(0, device="cuda")
    out = tq.verify_draft(torch.empty((0, 5), device="cuda"), e.int(),
                          torch.zeros(1, dtype=torch.int32, device="cuda"), e, e)
    assert [x.shape[0] for x in out] == [0, 0, 0]


def test_wider_outputs_and_wide_nodes(tq):
    check(tq, make(5, [3, 4], 50, True, False), width=9)
    check(tq, make(6, [300, 1024], 40, True, False, branch=2), width=1024)
    check(tq, make(6, [200, 257], 40, True, True, branch=7), width=257)


def test_borders(tq):
    """u = 0, r = 0, r just below 1; draft equal to the target (all accepted);
    draft that excludes the target's support (all refused); one-hot rows."""
    for tree, draft in ((False, True), (False, False), (True, False), (True, True)):
        m = make(13, [6, 6, 6], 60, tree, draft)
        m["u"][:] = 0.0
        m["r"] = np.array([0.0, np.nextafter(np.float32(1), np.float32(0)), 0.5], np.float32)
        check(tq, m)
        m["u"][:] = np.nextafter(np.float32(1), np.float32(0))
        check(tq, m)
    m = make(14, [7], 64, False, True)
    m["q"] = m["p"].clone()
    assert check(tq, m) == 6
    for tree in (False, True):
        m = make(15, [7], 64, tree, True)
        m["p"][:, :32] = 0
        m["q"][:, 32:] = 0
        m["tokens"] = (m["tokens"] % 32).astype(np.int32)
        assert check(tq, m) == 0
    m = make(16, [4, 4], 64, False, False)
    m["p"][:] = 0
    m["p"][:, 63] = 1.0
    check(tq, m)
    m["tokens"][:] = 63
    assert check(tq, m) == 6


def test_same_token_twice_among_siblings(tq):
    for draft in (False, True):
        m = make(17, [9, 9], 12, True, draft, branch=8)
        m["tokens"][2:9] = m["tokens"][1]
        m["tokens"][11:18] = m["tokens"][10]
        check(tq, m)


def test_bad_tokens_parents_and_probabilities(tq):
    """Tokens outside the vocabulary, parents that do not come before, NaN,
    negative and all-zero rows: nothing is accepted for them, nothing breaks."""
    for draft in (False, True):
        m = make(18, [8, 8, 8], 70, True, draft)
        m["tokens"][3], m["tokens"][5] = -1, 70
        m["tokens"][9], m["tokens"][10] = 2 ** 31 - 1, -2 ** 31
        m["parents"][4], m["parents"][6] = 6, -3
        m["parents"][12] = 2 ** 31 - 1
        check(tq, m)
    m = make(19, [3, 3], 70, False, False)
    m["p"][:, ::2] = float("nan")
    m["p"][:, 1] = -1.0
    check(tq, m)
    m["p"][:] = 0
    a, t, _ = call(tq, m, 3)
    assert a.tolist() == [0, 0] and t.tolist() == [[-1] * 3] * 2


def test_row_strides(tq):
    m = make(20, [5, 5], 129, False, True)
    want = call(tq, m, 5)
    wide = torch.zeros((10, 150), device="cuda")
    wide[:, :129] = m["p"].cuda()
    got = tq.verify_draft(wide[:, :129], dev(m["tokens"]), dev(m["starts"]), dev(m["u"]),
                          dev(m["r"]), draft=None, max_nodes=5)
    m2 = dict(m, q=None)
    want = call(tq, m2, 5)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    check(tq, m2)


def test_starts_that_leave_the_rows(tq):
    """Starts past the rows or beyond the output's width are cut, not read."""
    m = make(21, [4, 4], 30, False, False)
    m["starts"] = np.array([0, 4, 1000], np.int32)
    a, t, _ = call(tq, m, 3)
    full = make(21, [4, 4], 30, False, False)
    full["starts"] = np.array([0, 3, 7], np.int32)        # first rows as [0, 3)
    want = call(tq, full, 3)
    assert a[0] == want[0][0] and t[0].tolist() == want[1][0].tolist()


def test_distribution(tq):
    """Chains: over many sequences with the same rows the first token out
    follows the target, whatever the draft (a chi-square at 63 degrees of
    freedom stays below 63 + 6 * sqrt(126))."""
    V, B = 64, 20000
    rng = np.random.default_rng(5)
    p = rng.dirichlet(np.ones(V)).astype(np.float32)
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    tok = np.stack([np.zeros(B), rng.choice(V, B, p=q.astype(np.float64) / q.astype(np.float64).sum())], 1)
    a, t, _ = tq.verify_draft(dev(np.tile(p, (2 * B, 1))), dev(tok.astype(np.int32).ravel()),
                              dev(np.arange(0, 2 * B + 1, 2, dtype=np.int32)),
                              dev(rng.random(2 * B).astype(np.float32)),
                              dev(rng.random(B).astype(np.float32)),
                              draft=dev(np.tile(q, (2 * B, 1))), max_nodes=2)
    n = np.bincount(t[:, 0].cpu().numpy(), minlength=V)
    e = p.astype(np.float64) / p.astype(np.float64).sum() * B
    assert ((n - e) ** 2 / e).sum() < 63 + 6 * np.sqrt(126)
