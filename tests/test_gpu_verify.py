"""Verification of drafted trees on the GPU against the 64-bit walk: paths, counts and
tokens are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from mixed_precision_quantized_gb300 import build, ekv
from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ekv.lib()


def _dev(*xs):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _check(p, q, tokens, parents, u, us, cnt=None):
    n, m, _ = p.shape
    dp, dq, dt, dpar, du, dus, dc = _dev(p, q, tokens, parents, u, us, cnt)
    got = ekv.verify_tree(dp, dt, dpar, du, dus, draft_probs=dq, n_nodes=dc)
    path, acc, nxt = (x.cpu().numpy() for x in got)
    for z in range(n):
        want, tok = serving.verify(p[z], None if q is None else q[z], tokens[z], parents[z], u[z],
                                   us[z], m if cnt is None else min(m, int(cnt[z])))
        assert path[z].tolist() == want + [-1] * (m - len(want)), f"sequence {z}"
        assert acc[z] == len(want) and nxt[z] == tok, f"sequence {z}: {nxt[z]} for {tok}"
    return path, acc, nxt


def _case(seed, n, m, V, draft, shape="tree", peak=6.0):
    """Softmaxed rows with a peak; tokens drafted from q, or the best of a blurred p."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n, m, V)) * 2
    x[np.arange(n)[:, None], np.arange(m), rng.integers(0, V, (n, m))] += peak * rng.random((n, m))
    soft = lambda t: (np.exp(t - t.max(-1, keepdims=True)) /  # noqa: E731
                      np.exp(t - t.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)
    p, q = soft(x), soft(x + rng.normal(size=x.shape) * 0.7)
    par = np.full((n, m), -1, np.int32)
    tok = np.zeros((n, m), np.int32)
    for z in range(n):
        for i in range(1, m):
            par[z, i] = i - 1 if shape == "chain" else rng.integers((i - 1) // 3, i)
            row = q[z, par[z, i]].astype(np.float64)
            if draft:
                tok[z, i] = rng.choice(V, p=row / row.sum())
            else:
                rank = int(np.sum(par[z, 1:i] == par[z, i]))
                tok[z, i] = np.argsort(-row)[min(rank, V - 1)]
    return (p, q if draft else None, tok, par, rng.random((n, m)).astype(np.float32),
            rng.random(n).astype(np.float32))


@pytest.mark.parametrize("draft", [False, True], ids=["target", "draft"])
@pytest.mark.parametrize("shape", ["tree", "chain"])
@pytest.mark.parametrize("n,m,V", [(1, 1, 1), (3, 2, 2), (5, 8, 31), (4, 16, 128), (2, 64, 129),
                                   (7, 5, 1000), (2, 9, 4099), (1, 6, 40000)])
def test_walks(n, m, V, shape, draft):
    _check(*_case(n * 100 + m, n, m, V, draft, shape))


@pytest.mark.parametrize("draft", [False, True], ids=["target", "draft"])
@pytest.mark.parametrize("V", [8192, 8193, 9001])
def test_rows_shared_by_a_cluster(V, draft):
    """Rows just past the size from which CTAs of a cluster share them (some have an empty
    slice and reach the exchange of sums first), more sequences than run at once, trees
    of no nodes among them; three calls in a row give the same."""
    n = 400
    p, q, tok, par, u, us = _case(V, 8, 5, V, draft)
    pick = np.random.default_rng(V).integers(0, 8, n)
    c = [None if x is None else x[pick] for x in (p, q, tok, par)]
    u = np.random.default_rng(V + 1).random((n, 5)).astype(np.float32)
    us = np.random.default_rng(V + 2).random(n).astype(np.float32)
    cnt = np.random.default_rng(V + 3).integers(0, 6, n).astype(np.int32)
    for _ in range(3):
        _check(*c, u, us, cnt=cnt)


@pytest.mark.parametrize("draft", [False, True], ids=["target", "draft"])
@pytest.mark.parametrize("seed", range(6))
def test_many_small_trees(seed, draft):
    """200 trees of up to 24 nodes over 50 tokens: every outcome occurs."""
    c = _case(seed, 200, 24, 50, draft)
    cnt = np.random.default_rng(seed).integers(-1, 27, 200).astype(np.int32)
    path, acc, nxt = _check(*c, cnt=cnt)
    assert acc.max() >= 3 and (acc[cnt > 1] == 0).any() and np.all(nxt[cnt <= 0] == -1)


def test_twins_and_siblings_that_use_up_the_mass():
    """Two children with one token; children that hold all of p between them (the
    residual is empty: p itself is drawn from); a token outside the vocabulary; bad
    parents."""
    V = 4
    p = np.zeros((1, 8, V), np.float32)
    p[:, :] = [0.5, 0.25, 0.25, 0.0]
    par = np.array([[-1, 0, 0, 0, 0, 0, 9, -7]], np.int32)
    tok = np.array([[0, 0, 0, 1, 9, 2, 1, 1]], np.int32)
    for us in (0.0, 0.49, 0.5, 0.75, 0.999):
        for uu in (0.999, 0.6, 0.1):
            _check(p, None, tok, par, np.full((1, 8), uu, np.float32), np.array([us], np.float32))
    # u = 1 accepts nothing that is not certain: every child rejected, mass 0 left
    path, acc, nxt = _check(p, None, tok, par, np.full((1, 8), 1.0, np.float32),
                            np.array([0.6], np.float32))
    assert acc[0] == 0 and nxt[0] == 1
    q = p.copy()
    _check(p, q, tok, par, np.full((1, 8), 1.0, np.float32), np.array([0.6], np.float32))


def test_certain_targets_and_zero_rows():
    """One-hot rows (a target at temperature 0): the walk follows them exactly.  A row
    of zeros gives the last token."""
    m, V = 6, 300
    p = np.zeros((2, m, V), np.float32)
    best = [7, 299, 0, 128, 127, 5]
    for i, b in enumerate(best):
        p[0, i, b] = 1.0
    par = np.array([[-1, 0, 0, 2, 3, 4]] * 2, np.int32)
    tok = np.array([[0, 6, 7, 0, 128, 1]] * 2, np.int32)
    u, us = np.full((2, m), 0.99, np.float32), np.array([0.99, 0.5], np.float32)
    path, acc, nxt = _check(p, None, tok, par, u, us)
    assert path[0, :3].tolist() == [2, 3, 4] and nxt[0] == 127 and acc[0] == 3
    assert acc[1] == 0 and nxt[1] == V - 1


def test_exact_edges_of_the_cumulative_sum():
    """Probabilities of 2^-12 over 4096 tokens: u k / 4096 falls on an edge, where the
    lowest index with cum > u sum is the next token."""
    V = 4096
    p = np.full((1, 1, V), 2.0 ** -12, np.float32)
    for k in (0, 1, 2, 100, 2047, 4095):
        _, _, nxt = _check(p, None, np.zeros((1, 1), np.int32), np.full((1, 1), -1, np.int32),
                           np.zeros((1, 1), np.float32), np.array([k / V], np.float32))
        assert nxt[0] == k


def test_negative_nan_and_small_entries():
    """Negative and NaN entries count as zero; entries of 2^-60 still count."""
    p = np.array([[[0.0, -3.0, np.nan, 2.0 ** -60, 2.0 ** -59]]], np.float32)
    args = _dev(np.zeros((1, 1), np.int32), np.full((1, 1), -1, np.int32),
                np.zeros((1, 1), np.float32))
    for us, want in ((0.0, 3), (0.3, 3), (0.34, 4), (0.99, 4)):
        _, _, nxt = ekv.verify_tree(_dev(p)[0], *args, torch.tensor([us], device="cuda"))
        assert nxt.item() == want


@pytest.mark.parametrize("V", [8, 9000])
@pytest.mark.parametrize("bad", [np.nan, -np.inf, -3.0, 1.5, np.inf])
@pytest.mark.parametrize("draft", [False, True], ids=["target", "draft"])
def test_entries_outside_0_to_1_at_drafted_tokens(draft, bad, V):
    """A drafted token's own p (and q) may be such an entry: the tests of it and of its
    siblings go by the clamped value, as the sums do."""
    m = 4
    p = np.zeros((6, m, V), np.float32)
    p[:, :, :5] = [0.5, 0.125, 0.125, 0.125, 0.125]
    q = np.roll(p, 1, -1) + 2.0 ** -10
    par = np.tile(np.array([-1, 0, 0, 0], np.int32), (6, 1))
    tok = np.tile(np.array([0, 1, 2, 0], np.int32), (6, 1))
    p[:, :, 1] = bad
    q[3:, :, 2] = bad
    clean = lambda x: np.clip(np.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0), 0, 1)  # noqa: E731
    for uu in (0.05, 0.11, 0.4, 0.95):
        u, us = np.full((6, m), uu, np.float32), np.linspace(0, 0.99, 6).astype(np.float32)
        a = [ekv.verify_tree(*_dev(x, tok, par, u, us), draft_probs=_dev(y if draft else None)[0])
             for x, y in ((p, q), (clean(p), clean(q)))]
        assert all(torch.equal(x, y) for x, y in zip(*a))
        _check(clean(p), clean(q) if draft else None, tok, par, u, us)


def test_strided_views_and_streams():
    """Rows inside a wider buffer (odd and aligned strides), another stream, and a
    captured graph replayed on new numbers."""
    for pad in (0, 1, 4):
        p, q, tok, par, u, us = _case(11, 3, 6, 500, True)
        big = torch.zeros(3, 7, 500 + pad, device="cuda")
        bigq = torch.zeros(3, 6, 501 + pad, device="cuda")
        big[:, :6, :500] = torch.from_numpy(p)
        bigq[:, :, 1:501] = torch.from_numpy(q)
        args = _dev(tok, par, u, us)
        want = ekv.verify_tree(*_dev(p), *args, draft_probs=_dev(q)[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = ekv.verify_tree(big[:, :6, :500], *args, draft_probs=bigq[:, :, 1:501], stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    dp, dq = _dev(p, q)
    with torch.cuda.graph(g):
        got = ekv.verify_tree(dp, *args, draft_probs=dq)
    c = _case(12, 3, 6, 500, True)
    for a, b in zip((dp, dq, *args), c):
        a.copy_(torch.from_numpy(b))
    g.replay()
    torch.cuda.synchronize()
    want = ekv.verify_tree(dp, *args, draft_probs=dq)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    p = torch.zeros(2, 3, 8, device="cuda")
    i = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    u, us = torch.zeros(2, 3, device="cuda"), torch.zeros(2, device="cuda")
    for bad in (lambda: ekv.verify_tree(p.half(), i, i, u, us), lambda: ekv.verify_tree(p, i.long(), i, u, us),
                lambda: ekv.verify_tree(p, i, i[:1], u, us), lambda: ekv.verify_tree(p, i, i, us, us),
                lambda: ekv.verify_tree(p, i, i, u, us, draft_probs=p[:, :, :4]),
                lambda: ekv.verify_tree(p[..., ::2], i, i, u, us),
                lambda: ekv.verify_tree(p, i, i, u, us, n_nodes=us)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    big = torch.zeros(1, 65, 8, device="cuda")
    with pytest.raises(ekv.EkvError):
        ekv.verify_tree(big, torch.zeros(1, 65, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, 65, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, 65, device="cuda"), us[:1])
