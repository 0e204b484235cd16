"""The speculative step's oracle against what it has to satisfy, on the CPU."""
import itertools

import numpy as np
import pytest

from oracle import spec_oracle as O


def _rows(rng, T, V):
    x = np.exp(2 * rng.standard_normal((T, V)))
    return x / x.sum(1, keepdims=True)


TREES = [[-1, 0], [-1, 0, 0], [-1, 0, 0, 0], [-1, 0, 1], [-1, 0, 0, 1, 2, 1]]


@pytest.mark.parametrize("parents", TREES)
def test_first_token_is_distributed_as_the_target(parents):
    """Integrated over every draw of the drafts and, by the lengths of the accepting intervals, over
    the numbers: the probability that the first token is x is p(x)."""
    rng = np.random.default_rng(len(parents))
    V, T = 3, len(parents)
    p, q = _rows(rng, T, V), _rows(rng, T, V)
    kids = [t for t in range(1, T) if parents[t] == 0]
    got = np.zeros(V)
    grid = (np.arange(64) + 0.5) / 64
    for drawn in itertools.product(range(V), repeat=len(kids)):
        w = np.prod([q[0, x] for x in drawn])
        # the recursion of the definition, exactly
        r, weight = p[0].copy(), w
        for x in drawn:
            a = min(1.0, r[x] / q[0, x])
            got[x] += weight * a
            weight *= 1 - a
            if weight == 0:
                break
            r = np.maximum(r - q[0], 0)
            r /= r.sum()
        got += weight * r
        # and verify_ref follows it: at numbers just inside and outside each interval
        tokens = np.zeros(T, dtype=int)
        tokens[kids] = drawn
        u = np.ones(T)
        r, Z = p[0].copy(), 1.0
        for k, (t, x) in enumerate(zip(kids, drawn)):
            a = r[x] / Z / q[0, x]
            for du in (-1e-9, 1e-9):
                v = u.copy()
                v[t] = max(0.0, min(a, 1.0 - 2e-9) + du)
                path, _ = O.verify_ref(p, q, tokens, parents, T, v, 0.5)
                assert (t in path) == (v[t] < a)
            u[t] = 1e18     # refused, whatever is left
            r = np.maximum(r - Z * q[0], 0)
            Z = r.sum()
            if Z == 0:
                break
        if Z > 0:
            nxt = [O.verify_ref(p, q, tokens, parents, T, u, g)[1] for g in grid]
            assert np.all(np.abs(np.bincount(nxt, minlength=V) / 64 - r / Z) <= 1 / 64 + 1e-12)
    assert np.allclose(got, p[0], atol=1e-12)


def test_point_masses():
    """Drafts without probabilities: child after child is accepted with its share of what is left."""
    rng = np.random.default_rng(4)
    p = _rows(rng, 4, 5)
    parents, tokens = [-1, 0, 0, 0], [0, 3, 1, 3]
    a1 = p[0, 3]
    a2 = p[0, 1] / (1 - p[0, 3])
    for u1, u2, want in ((a1 - 1e-9, 0.9, [0, 1]), (a1 + 1e-9, a2 - 1e-9, [0, 2]), (a1 + 1e-9, a2 + 1e-9, [0])):
        assert O.verify_ref(p, None, tokens, parents, 4, [0, u1, u2, 0.0], 0.5)[0] == want
    rest = np.array([O.verify_ref(p, None, tokens, parents, 4, [0, 0.999, 0.999, 0.0], g)[1] for g in (np.arange(999) + 0.5) / 999])
    assert not np.isin(rest, [1, 3]).any()       # refused tokens are not drawn


def test_draw_and_edges():
    p = np.array([[0.25, 0.0, 0.5, 0.25], [1.0, 0, 0, 0]])
    q = np.array([[0.5, 0.0, 0.25, 0.25], [1.0, 0, 0, 0]])
    par = [-1, 0]
    for u, x in ((0.0, 0), (0.2499, 0), (0.25, 2), (0.7499, 2), (0.75, 3), (0.9999, 3)):
        assert O.verify_ref(p, q, [0, 1], [-1, -1], 2, [0, 0], u) == ([0], x)
    # u q < p is strict: 0.5 * 0.5 = 0.25
    assert O.verify_ref(p, q, [0, 0], par, 2, [0, 0.5], 0.0) == ([0], 2)
    assert O.verify_ref(p, q, [0, 0], par, 2, [0, np.nextafter(0.5, 0)], 0.0) == ([0, 1], 0)
    # a token of no mass is never accepted, not even with u = 0
    assert O.verify_ref(p, q, [0, 1], par, 2, [0, 0.0], 0.0)[0] == [0]
    # p = q and refused all the same: the draw is from p
    assert O.verify_ref(p, p, [0, 0], par, 2, [0, 1.0], 0.3) == ([0], 2)
    assert O.verify_ref(0 * p, q, [0, 0], par, 2, [0, 0.0], 0.3) == ([0], -1)
    assert O.verify_ref(p, q, [0, 0], par, 0, [0, 0.0], 0.3) == ([], -1)
    assert O.verify_ref(p, q, [0, 9], par, 2, [0, 0.0], 0.3)[0] == [0]


def test_pages_hold_what_the_table_says():
    rng = np.random.default_rng(8)
    g = O.Pages(np.full((6, 8), -1, dtype=np.int32), np.zeros(20, dtype=np.int32), np.zeros(6, dtype=np.int32))
    g.resize([100, 64, 0, 1, 200, 0])
    assert g.bt[0, :2].tolist() == [0, 1] and g.bt[1, 0] == 2 and g.bt[3, 0] == 3 and g.bt[4, :4].tolist() == [4, 5, 6, 7]
    g.check()
    c = g.fork([0, 0, 4], [2, 5, 4])
    assert c.tolist() == [[1, 1, -1], [8, 9, -1], [36, 36, 0]]
    g.check()
    g.resize([0, 64, 100, 1, 130, 100])
    g.check()
    for _ in range(50):
        g.resize(rng.integers(0, 300, 6))
        g.check()
        s = int(rng.integers(0, 6))
        d = (s + 1 + int(rng.integers(0, 5))) % 6
        n = g.lens.copy()
        n[d] = 0
        g.resize(n)
        g.fork([s], [d])
        g.check()


def test_tree_decode_reduces_to_the_causal_one():
    """A chain's tree attention is the causal decode of the T new rows, which is pinned on its own;
    a full mask is the non-causal one; a tree of one node is a decode step of one token."""
    from oracle import mla_oracle as M
    rng = np.random.default_rng(0)
    B, T, H = 3, 5, 2
    lens = np.array([70, 5, 130])
    bt = rng.permutation(8)[:6].reshape(3, 2)
    bt = np.concatenate([bt, [[6], [6], [7]]], 1)
    pool = rng.standard_normal((8, 64, 576))
    ql, qp = rng.standard_normal((B, T, H, 512)) * 0.3, rng.standard_normal((B, T, H, 64))
    chain = O.ancestors(np.tile(np.arange(-1, T - 1), (B, 1)))
    assert np.array_equal(chain[0], np.tril(np.ones((T, T), dtype=bool)))
    for see, causal in ((chain, True), (np.ones((B, T, T), dtype=bool), False)):
        o, l = O.tree_decode_ref(ql, qp, pool, bt, lens, [T] * B, see)
        ro, rl = M.decode_ref(ql, qp, pool, bt, lens, causal)
        assert np.allclose(o, ro, atol=1e-12) and np.allclose(l, rl, atol=1e-12)


def test_tree_decode_is_its_branches_decoded_alone():
    """Each branch, as a chain over the prefix and its own rows only, gives the same last row."""
    from oracle import mla_oracle as M
    rng = np.random.default_rng(1)
    S, T, H = 80, 6, 2
    parents = np.array([[-1, 0, 0, 1, 2, 2]])
    see = O.ancestors(parents)
    pool = rng.standard_normal((2, 64, 576))
    ql, qp = rng.standard_normal((1, T, H, 512)) * 0.3, rng.standard_normal((1, T, H, 64))
    o, l = O.tree_decode_ref(ql, qp, pool, np.array([[0, 1]]), [S], [T], see)
    flat = pool.reshape(-1, 576)
    for t in range(T):
        rows = np.concatenate([flat[:S - T], flat[S - T:S][see[0, t]]])
        alone = np.zeros((2, 64, 576))
        alone.reshape(-1, 576)[:len(rows)] = rows
        ro, rl = M.decode_ref(ql[:, t:t + 1], qp[:, t:t + 1], alone, np.array([[0, 1]]), np.array([len(rows)]), False)
        assert np.allclose(o[0, t], ro[0, 0], atol=1e-12) and np.allclose(l[0, t], rl[0, 0], atol=1e-12)


def test_see_words():
    see = np.zeros((1, 34, 34), dtype=bool)
    see[0, 1, [0, 31, 32]] = True
    w = O.see_words(see).view(np.uint32)
    assert w.shape == (1, 34, 2)
    assert w[0, 1].tolist() == [0x80000001, 0xFFFFFFFD] and w[0, 0].tolist() == [0, 0xFFFFFFFC]
