"""mla_verify_tree against the float64 rule: accepted nodes and tokens are equal, not near.

The kernel decides in pairs of fp32 values, the oracle in 64 bits; their sums differ by
about 1e-13 of the mass, and a number lands that close to a border with a probability of
about 1e-11 per decision, so no seed is chosen."""
import numpy as np
import pytest

from oracle import spec_oracle as O

pytestmark = pytest.mark.gpu


def _f32(x):
    return np.asarray(x, dtype=np.float32)


def _probs(torch, g, B, T, V, dtype, noise=0.7, sharp=5.0):
    logits = torch.randn((B, T, V), generator=g, device="cuda") * sharp
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + noise * torch.randn((B, T, V), generator=g, device="cuda"), -1)
    return p.to(dtype), q.to(dtype)


def _parents(rng, B, T, tree):
    par = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))
    if tree:
        for t in range(1, T):
            par[:, t] = rng.integers(0, t, B) // rng.integers(1, 3, B)
    return par


class Run:
    def __init__(self, mla, torch, p, q, tokens, parents, ua, us, nodes=None, pad=0, stream=None):
        B, T, V = p.shape
        el = 8 if p.dtype == torch.bfloat16 else 4
        width = (V + el - 1) // el * el + pad * el
        nan = torch.full((B, T, width), float("nan"), dtype=p.dtype, device="cuda")
        self.p = nan.clone()
        self.p[..., :V] = p
        self.q = None
        if q is not None:
            self.q = nan
            self.q[..., :V] = q
        dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()  # noqa: E731
        self.args = (dev(tokens, np.int32), dev(parents, np.int32), None if nodes is None else dev(nodes, np.int32),
                     dev(ua, np.float32), dev(us, np.float32))
        self.out = [torch.full((B,), -7, dtype=torch.int32, device="cuda")] + [
            torch.full((B, T), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.B, self.T, self.V, self.width, self.mla = B, T, V, width, mla
        self.dtype = mla.MLA_DTYPE_BF16 if p.dtype == torch.bfloat16 else mla.MLA_DTYPE_F32

    def call(self, stream=None):
        return self.mla.mla_verify_tree(self.B, self.T, self.V, self.p, self.q, self.dtype, self.width, *self.args,
                                        *self.out, stream)

    def results(self, expect=None):
        import torch
        torch.cuda.synchronize()
        assert self.mla.mla_read_device_status(None)[0] == (self.mla.MLA_OK if expect is None else expect)
        return [x.cpu().numpy() for x in self.out]

    def check(self, expect=None):
        """The three outputs, compared with the oracle's; returns accept_len."""
        n_acc, idx, out = self.results(expect)
        p = self.p.double().cpu().numpy()[..., :self.V]
        q = None if self.q is None else self.q.double().cpu().numpy()[..., :self.V]
        tokens, parents, nodes, ua, us = [None if a is None else a.cpu().numpy() for a in self.args]
        for b in range(self.B):
            n = self.T if nodes is None else int(nodes[b])
            n = n if 0 <= n <= self.T else 0
            path, nxt = O.verify_ref(p[b], None if q is None else q[b], tokens[b], parents[b], n,
                                     ua[b].astype(np.float64), float(us[b]))
            want = [int(tokens[b, t]) for t in path[1:]] + ([nxt] if n else [])
            assert n_acc[b] == len(path), (b, n_acc[b], path)
            assert idx[b].tolist() == path + [-1] * (self.T - len(path)), b
            assert out[b].tolist() == want + [-1] * (self.T - len(want)), (b, out[b], want)
        return n_acc


def _random(mla, torch, B, T, V, dtype, draft, tree, seed=0, nodes=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + V + T)
    rng = np.random.default_rng([seed, B, T, V])
    p, q = _probs(torch, g, B, T, V, dtype, **kw)
    par = _parents(rng, B, T, tree)
    at = torch.from_numpy(np.maximum(par, 0)).long().cuda()
    rows = q.float()[torch.arange(B, device="cuda")[:, None], at].reshape(B * T, V)
    tokens = torch.multinomial(rows, 1, generator=g).view(B, T).cpu().numpy()
    r = Run(mla, torch, p, q if draft else None, tokens, par, rng.random((B, T)), rng.random(B), nodes, pad=seed % 2)
    assert r.call() == mla.MLA_OK
    return r


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,V", [(3, 1, 5), (40, 4, 1), (40, 9, 7), (33, 5, 8), (17, 6, 255), (16, 12, 256), (16, 33, 257),
                                   (9, 8, 1031), (5, 24, 32001), (3, 6, 129280), (2, 7, 262147)])
def test_verify_matches_the_rule(mla, cuda, B, T, V, dtype, draft, tree):
    import torch
    for seed in (0, 1):
        _random(mla, torch, B, T, V, getattr(torch, dtype), draft, tree, seed).check()


@pytest.mark.parametrize("B", [20, 37, 44, 50, 60, 75, 90, 140, 310])
def test_verify_whatever_the_cluster(mla, cuda, B):
    """Batches that leave room for eight CTAs per sequence, down to one; the last rows of a
    vocabulary that no slice divides."""
    import torch
    _random(mla, torch, B, 4, 5003, torch.float32, B % 2 == 0, False, B).check()


@pytest.mark.parametrize("draft", [False, True])
def test_verify_many_refused_siblings(mla, cuda, draft):
    """Wide trees over a flat, small vocabulary: residual after residual, tokens drawn twice."""
    import torch
    B, T, V = 64, 40, 300
    r = _random(mla, torch, B, T, V, torch.float32, draft, True, 3, sharp=0.5, noise=3.0)
    r.check()
    star = np.zeros((B, T), dtype=np.int32)
    star[:, 0] = -1
    tokens = r.args[0].cpu().numpy()
    tokens[:, T // 2:] = tokens[:, :T - T // 2]       # each token is drafted twice
    ua = np.random.default_rng(1).random((B, T)) * 0.3 + 0.7
    r2 = Run(mla, torch, r.p[..., :V], None if r.q is None else r.q[..., :V], tokens, star, ua, np.random.default_rng(2).random(B))
    assert r2.call() == mla.MLA_OK
    r2.check()


def test_verify_1024_nodes(mla, cuda):
    import torch
    for tree in (False, True):
        # a chain whose every draft is accepted, and a random tree
        T, V = 1024, 50
        p = torch.full((2, T, V), 1.0 / V, device="cuda")
        rng = np.random.default_rng(3)
        r = Run(mla, torch, p, p, rng.integers(0, V, (2, T)), _parents(rng, 2, T, tree), rng.random((2, T)) * 0.99, rng.random(2))
        assert r.call() == mla.MLA_OK
        n = r.check()
        assert tree or (n == T).all()


def test_verify_node_counts_and_bad_nodes(mla, cuda):
    import torch
    r = _random(mla, torch, 12, 6, 400, torch.float32, True, True, 5, nodes=[6, 0, 1, 2, 3, 4, 5, 6, 6, 6, 6, 1])
    r.check()
    # counts outside [0, T] count as 0, bad tokens and parents are passed over; both are reported
    r.args[2][7], r.args[2][8] = 7, -1
    r.call()
    r.check(expect=mla.MLA_ERR_DEVICE_CHECK)
    r.args[2][7] = r.args[2][8] = 6
    for arr, values in ((0, (400, -1, 2 ** 31 - 1, -2 ** 31)), (1, (-1, 2, 6, 2 ** 31 - 1, -2 ** 31))):
        for v in values:
            was = r.args[arr][0, 2].clone()
            r.args[arr][0, 2] = v
            r.call()
            r.check(expect=mla.MLA_ERR_DEVICE_CHECK)
            r.args[arr][0, 2] = was
    r.call()
    r.check()


def test_verify_borders(mla, cuda):
    """Numbers on a border, exactly: u q = p refuses, a running sum equal to u Z goes on to the next."""
    import torch
    p = torch.tensor([[[0.25, 0.0, 0.5, 0.25], [1.0, 0, 0, 0]]], device="cuda")
    q = torch.tensor([[[0.5, 0.0, 0.25, 0.25], [1.0, 0, 0, 0]]], device="cuda")
    below = float(np.nextafter(_f32(0.5), _f32(0)))
    cases = [(0, 0.5, 0.0), (0, below, 0.0), (0, below, 0.9), (1, 0.0, 0.0), (2, 0.99, 0.25), (1, 0.0, 0.25),
             (1, 0.0, 0.75), (1, 0.0, float(np.nextafter(_f32(0.75), _f32(0)))), (1, 0.0, float(np.nextafter(_f32(1), _f32(0))))]
    for dt in (torch.float32, torch.bfloat16):
        for x, ua, us in cases:
            for draft in (q, p, None):
                r = Run(mla, torch, p.to(dt), None if draft is None else draft.to(dt), [[0, x]], [[-1, 0]], [[0, ua]], [us])
                assert r.call() == mla.MLA_OK
                r.check()


def test_verify_rows_without_mass_and_odd_values(mla, cuda):
    """Rows of zeros give -1; NaN, infinite and negative probabilities are no mass; q may be anything where no child hangs."""
    import torch
    V = 700
    g = torch.Generator(device="cuda").manual_seed(2)
    p, q = _probs(torch, g, 4, 3, V, torch.float32)
    p[0] = 0
    p[1, :, ::2] = float("nan")
    p[1, :, 1::10] = float("inf")
    q[1, :, 5::10] = float("inf")
    p[2, :, 5:] *= -1
    q[:, 2] = float("nan")
    tokens = [[0, 4, 8], [0, 3, 9], [0, 2, 1], [0, 1, 2]]
    for us in (0.0, 0.5, 0.999):
        r = Run(mla, torch, p, q, tokens, [[-1, 0, 1]] * 4, np.full((4, 3), 0.2), [us] * 4)
        assert r.call() == mla.MLA_OK
        r.check()
        r = Run(mla, torch, p, None, tokens, [[-1, 0, 0]] * 4, np.full((4, 3), 0.2), [us] * 4)
        assert r.call() == mla.MLA_OK
        r.check()


def test_verify_last_tokens_of_the_vocabulary(mla, cuda):
    """All mass on single entries, at both ends of a row and around the edges of what a warp reads."""
    import torch
    for V in (1, 9, 256, 4099, 66000):
        for x in sorted({0, V - 1, min(7, V - 1), min(8, V - 1), min(255, V - 1), V // 2}):
            p = torch.zeros((1, 1, V), device="cuda")
            p[0, 0, x] = 1e-30
            for us in (0.0, 0.5, float(np.nextafter(_f32(1), _f32(0)))):
                r = Run(mla, torch, p, None, [[0]], [[-1]], [[0]], [us])
                assert r.call() == mla.MLA_OK
                assert r.results()[2][0, 0] == x


def test_verify_captured_and_replayed(mla, cuda):
    import torch
    r = _random(mla, torch, 8, 6, 5000, torch.float32, True, True, 1)
    first = r.results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert r.call() == mla.MLA_OK
    r.args[4].copy_(torch.rand(8, device="cuda"))
    r.args[3].copy_(torch.rand(8, 6, device="cuda"))
    for x in r.out:
        x.fill_(-7)
    g.replay()
    g.replay()
    r.check()
    assert len(first) == 3


def test_verify_emits_the_targets_distribution(mla, cuda):
    """Many draws of a three-node tree over ten tokens: the first token's counts are the target's, within
    five standard deviations of each count (a chance of 1e-5 that a right kernel fails, and the seed is fixed)."""
    import torch
    B, V = 40000, 10
    g = torch.Generator(device="cuda").manual_seed(9)
    p1 = torch.softmax(torch.randn(3, V, generator=g, device="cuda"), -1)
    q1 = torch.softmax(torch.randn(3, V, generator=g, device="cuda"), -1)
    tokens = torch.multinomial(q1[0].expand(B, V), 3, replacement=True, generator=g).cpu().numpy()
    rng = np.random.default_rng(0)
    r = Run(mla, torch, p1.expand(B, 3, V), q1.expand(B, 3, V), tokens, [[-1, 0, 0]] * B, rng.random((B, 3)), rng.random(B))
    assert r.call() == mla.MLA_OK
    count = np.bincount(r.results()[2][:, 0], minlength=V)
    p = p1[0].double().cpu().numpy()
    p /= p.sum()
    assert np.all(np.abs(count - B * p) <= 5 * np.sqrt(B * p * (1 - p)))


def test_verify_rows_past_32_bit_offsets(mla, cuda):
    """Two chains of 1024 nodes over 1.1 million entries (bf16, 4.5 GB): the last row of all decides."""
    import torch
    B, T, V = 2, 1024, 1100000
    p = torch.zeros((B, T, V), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    tokens = rng.integers(0, V, (B, T)).astype(np.int32)
    tokens[1, -1] = V - 1
    b, t = np.meshgrid(np.arange(B), np.arange(T - 1), indexing="ij")
    p[torch.from_numpy(b).cuda(), torch.from_numpy(t).cuda(), torch.from_numpy(tokens[:, 1:]).long().cuda()] = 1
    p[0, T - 1, 7] = 1
    p[1, T - 1, V - 3] = 1
    par = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    n, idx, out = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((B,), (B, T), (B, T)))
    assert mla.mla_verify_tree(B, T, V, p, None, mla.MLA_DTYPE_BF16, V, i32(tokens), i32(par), None,
                               torch.full((B, T), 0.5, device="cuda"), torch.full((B,), 0.5, device="cuda"), n, idx, out) == mla.MLA_OK
    torch.cuda.synchronize()
    assert n.tolist() == [T, T]
    assert torch.equal(idx.cpu(), torch.arange(T, dtype=torch.int32).expand(B, T))
    assert np.array_equal(out[:, :-1].cpu().numpy(), tokens[:, 1:]) and out[:, -1].tolist() == [7, V - 3]
