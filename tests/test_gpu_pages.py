"""Page calls against the one-page-at-a-time oracle: tables, counts and rows are equal."""
import numpy as np
import pytest

from oracle import spec_oracle as O

pytestmark = pytest.mark.gpu


def _i32(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _ok(mla, torch, expect=None):
    torch.cuda.synchronize()
    assert mla.mla_read_device_status(None)[0] == (mla.MLA_OK if expect is None else expect)


def _table(rng, lens, nb, width):
    order = rng.permutation(nb)
    bt, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for b, s in enumerate(lens):
        n = (int(s) + 63) // 64
        bt[b, :n] = order[at:at + n]
        at += n
    refs = np.zeros(nb, dtype=np.int32)
    refs[bt[bt >= 0]] = 1
    return bt, refs


class Dev:
    """Device copies of an oracle's table and counts; ``stride`` pads the table rows."""

    def __init__(self, mla, torch, g, stride=None):
        self.mla, self.torch, self.nb = mla, torch, len(g.refs)
        B, self.mp = g.bt.shape
        full = torch.full((B, stride or self.mp), 77, dtype=torch.int32, device="cuda")
        full[:, :self.mp] = _i32(torch, g.bt)
        self.full, self.stride, self.B = full, full.shape[1], B
        self.refs, self.lens = _i32(torch, g.refs), _i32(torch, g.lens)

    def resize(self, new, got=None):
        got = self.lens if got is None else got
        return self.mla.mla_pages_resize(self.refs, self.nb, self.full, self.stride, self.mp, self.lens, new, self.B, got)

    def fork(self, src, dst):
        n = len(src)
        self.copies = self.torch.full((3, max(n, 1)), -9, dtype=self.torch.int32, device="cuda")
        return self.mla.mla_pages_fork(self.refs, self.nb, self.full, self.stride, self.mp, self.lens, self.B,
                                       _i32(self.torch, src), _i32(self.torch, dst), n, self.copies)

    def same(self, g):
        assert np.array_equal(self.full[:, :self.mp].cpu().numpy(), g.bt)
        assert np.array_equal(self.refs.cpu().numpy(), g.refs)
        assert np.array_equal(self.lens.cpu().numpy(), g.lens)
        assert (self.full[:, self.mp:] == 77).all()


@pytest.mark.parametrize("B,width,nb", [(1, 1, 1), (3, 5, 9), (40, 33, 1400), (700, 9, 5000), (1500, 20, 40000)])
def test_resize_and_fork_follow_the_oracle(mla, cuda, B, width, nb):
    import torch
    rng = np.random.default_rng([B, nb])
    top = min(width * 64, 64 * nb // B)
    lens = rng.integers(0, top + 1, B).astype(np.int32)
    bt, refs = _table(rng, lens, nb, width)
    g = O.Pages(bt, refs, lens)
    d = Dev(mla, torch, g, stride=width + 3)
    for _ in range(4):
        new = rng.integers(0, top + 1, B).astype(np.int32)
        new[rng.random(B) < 0.3] = 0
        g.resize(new)
        assert d.resize(_i32(torch, new)) == mla.MLA_OK
        _ok(mla, torch)
        d.same(g)
        # the sequences of length 0 become forks of others (or of themselves)
        empty, full = np.nonzero(g.lens == 0)[0], np.nonzero(g.lens)[0]
        if not len(full):
            continue
        dst = empty[:4096 - 8]
        src = rng.choice(full, len(dst))
        own = np.setdiff1d(full, src)[:8]
        src, dst = np.concatenate([src, own]), np.concatenate([dst, own])
        free = int((g.refs == 0).sum())
        if len(src) == 0 or (g.lens[src] % 64 > 0).sum() > free:
            continue
        want = g.fork(src, dst)
        assert d.fork(src, dst) == mla.MLA_OK
        _ok(mla, torch)
        d.same(g)
        assert np.array_equal(d.copies.cpu().numpy(), want)
        g.check()


def test_resize_when_the_blocks_run_out(mla, cuda):
    import torch
    bt, refs = _table(np.random.default_rng(0), [64, 0, 128, 0], 8, 6)
    g = O.Pages(bt, refs, np.array([64, 0, 128, 0], dtype=np.int32))
    d = Dev(mla, torch, g)
    new = [100, 200, 0, 129]         # 1 + 4 + 3 pages asked for, 7 free after the release
    g.resize(new)
    assert g.lens.tolist() == [100, 200, 0, 128]
    assert d.resize(_i32(torch, new)) == mla.MLA_OK
    _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
    d.same(g)
    g.check()
    # nothing is free: nobody grows, and a release frees for the same call
    new = [300, 200, 0, 0]
    g.resize(new)
    assert d.resize(_i32(torch, new)) == mla.MLA_OK
    _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
    d.same(g)


def test_resize_bad_lengths_and_entries(mla, cuda):
    import torch
    lens = np.array([100, 100, 100], dtype=np.int32)
    bt, refs = _table(np.random.default_rng(1), lens, 9, 4)
    g = O.Pages(bt, refs, lens)
    for bad in (-1, 257, 2 ** 31 - 1):
        d = Dev(mla, torch, g)
        assert d.resize(_i32(torch, [0, bad, 200])) == mla.MLA_OK
        _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
        h = O.Pages(bt, refs, lens)
        h.resize([0, 100, 200])
        d.same(h)
    # an entry outside the pool, and a block that nobody holds: reported, the counts stay sound
    for k, free in ((9, None), (-5, None), (None, 0)):
        d = Dev(mla, torch, g)
        if k is not None:
            d.full[1, 1] = k
        else:
            d.refs[int(bt[1, 1])] = free
        assert d.resize(_i32(torch, [100, 0, 100])) == mla.MLA_OK
        _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
        assert (d.refs >= 0).all() and (d.full[1] == -1).all() and int(d.lens[1]) == 0
        assert int(d.refs[int(bt[1, 0])]) == 0
    # two sequences that hold one block: both give it back
    d = Dev(mla, torch, g)
    d.full[1, 0] = int(bt[0, 0])
    d.refs[int(bt[0, 0])] = 2
    d.refs[int(bt[1, 0])] = 0
    assert d.resize(_i32(torch, [0, 0, 100])) == mla.MLA_OK
    _ok(mla, torch)
    assert int(d.refs.sum()) == 2


def test_resize_into_other_lengths_arrays(mla, cuda):
    import torch
    lens = np.array([10, 70], dtype=np.int32)
    bt, refs = _table(np.random.default_rng(1), lens, 5, 3)
    g = O.Pages(bt, refs, lens)
    d = Dev(mla, torch, g)
    new, got = _i32(torch, [100, 30]), _i32(torch, [7, 7])
    assert d.resize(new, got) == mla.MLA_OK
    assert d.lens.tolist() == [10, 70] and got.tolist() == [100, 30]
    d.lens = got
    new = _i32(torch, [0, 0])
    assert d.resize(new, new) == mla.MLA_OK      # the new lengths' own array
    _ok(mla, torch)
    assert new.tolist() == [0, 0] and int(d.refs.abs().sum()) == 0


def test_fork_rules(mla, cuda):
    import torch
    lens = np.array([100, 64, 30, 0, 0, 0, 0], dtype=np.int32)
    bt, refs = _table(np.random.default_rng(3), lens, 6, 3)       # 4 blocks held, 2 free
    g = O.Pages(bt, refs, lens)
    bad = [([0, 2], [3, 3]), ([0, 3], [3, 4]), ([7], [3]), ([-1], [3]), ([0], [7]), ([0], [-1]), ([0], [2 ** 31 - 1])]
    for src, dst in bad:      # a dst named twice, a src that is a dst, rows that there are not
        d = Dev(mla, torch, g)
        assert d.fork(src, dst) == mla.MLA_OK
        _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
        good = [f for f in range(len(src)) if (src[f], dst[f]) == (0, 3) and dst.count(3) == 1]
        h = O.Pages(bt, refs, lens)
        want = h.fork([src[f] for f in good], [dst[f] for f in good])
        d.same(h)
        assert [int(x) for x in d.copies[0]] == [int(want[0, 0]) if f in good else -2 for f in range(len(src))]
        assert all(int(d.copies[2, f]) == 0 for f in range(len(src)) if f not in good)
    # two blocks are left: the first two copied pages get them, a fork of full pages needs none
    d = Dev(mla, torch, g)
    src, dst = [0, 1, 2, 0], [3, 4, 5, 6]
    want = g.fork(src, dst)
    assert want[0].tolist()[3] == -2 and want[2].tolist() == [36, 0, 30, 0]
    assert d.fork(src, dst) == mla.MLA_OK
    _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
    d.same(g)
    assert np.array_equal(d.copies.cpu().numpy(), want)


def test_two_holders_make_a_page_their_own(mla, cuda):
    import torch
    lens = np.array([100, 0], dtype=np.int32)
    bt, refs = _table(np.random.default_rng(3), lens, 9, 3)
    g = O.Pages(bt, refs, np.array([128, 0], dtype=np.int32))
    g.fork([0], [1])
    g.lens[:] = 90                    # both shortened into the page that they share
    d = Dev(mla, torch, g)
    want = g.fork([0, 1], [0, 1])
    assert d.fork([0, 1], [0, 1]) == mla.MLA_OK
    _ok(mla, torch)
    d.same(g)
    assert np.array_equal(d.copies.cpu().numpy(), want) and want[2].tolist() == [26, 26]
    g.check()
    want = g.fork([0, 1], [0, 1])     # their own by now
    assert d.fork([0, 1], [0, 1]) == mla.MLA_OK
    _ok(mla, torch)
    d.same(g)
    assert want[2].tolist() == [0, 0]


def _pool(torch, nb, kind, rng):
    """(bits on the host [nb, 64, width], device tensors, call(name) -> leading arguments)"""
    if kind == "fp8":
        host = rng.integers(0, 256, (nb, 64, 656)).astype(np.uint8)
        return host, torch.from_numpy(host).cuda()
    host = rng.integers(0, 1 << 16, (nb, 64, 576)).astype(np.uint16)
    return host, torch.from_numpy(host.view(np.int16)).cuda()


def _split(torch, pool):
    """The pool as latent rows 520 apart and RoPE rows 72 apart."""
    nb = pool.shape[0]
    c = torch.full((nb, 64, 520), 5, dtype=torch.int16, device="cuda")
    r = torch.full((nb, 64, 72), 5, dtype=torch.int16, device="cuda")
    c[..., :512], r[..., :64] = pool[..., :512], pool[..., 512:]
    return c, r


@pytest.mark.parametrize("kind", ["bf16", "split", "fp8"])
@pytest.mark.parametrize("B,T,lo,hi", [(1, 1, 1, 2), (5, 7, 7, 70), (9, 64, 64, 300), (3, 1024, 1024, 2000), (200, 6, 6, 200)])
def test_compact_moves_accepted_rows(mla, cuda, B, T, lo, hi, kind):
    import torch
    rng = np.random.default_rng([B, T])
    nodes = rng.integers(0, T + 1, B).astype(np.int32)
    nodes[0] = T
    lens = np.maximum(rng.integers(lo, hi, B), nodes).astype(np.int32)
    acc = np.array([rng.integers(0, n + 1) for n in nodes], dtype=np.int32)
    if B > 2:
        acc[1], acc[2] = nodes[1], 0          # all accepted, none accepted
    idx = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        idx[b, :acc[b]] = np.sort(rng.choice(nodes[b], acc[b], replace=False))
    width = (int(lens.max()) + 63) // 64
    nb = int(((lens + 63) // 64).sum()) + 2
    bt, refs = _table(rng, lens, nb, width)
    host, dev = _pool(torch, nb, kind, rng)
    g = O.Pages(bt, refs, lens, host)
    want = g.compact(nodes, acc, idx)
    new = torch.full((B + 4,), -7, dtype=torch.int32, device="cuda")
    args = (_i32(torch, bt), width, width, _i32(torch, lens), None if (nodes == T).all() else _i32(torch, nodes),
            _i32(torch, acc), _i32(torch, idx), B, T, new)
    if kind == "fp8":
        assert mla.mla_cache_compact_fp8(dev, nb, *args) == mla.MLA_OK
    elif kind == "split":
        c, r = _split(torch, dev)
        assert mla.mla_cache_compact(mla.cache_from_split(c, r), *args) == mla.MLA_OK
        assert (c[..., 512:] == 5).all() and (r[..., 64:] == 5).all()
        dev = torch.cat([c[..., :512], r[..., :64]], -1)
    else:
        assert mla.mla_cache_compact(mla.cache_from_pool(dev), *args) == mla.MLA_OK
    _ok(mla, torch)
    assert np.array_equal(new[:B].cpu().numpy(), want) and (new[B:] == -7).all()
    assert np.array_equal(dev.cpu().numpy().view(host.dtype), g.pool)


def test_compact_leaves_bad_sequences(mla, cuda):
    import torch
    rng = np.random.default_rng(6)
    lens, nodes, acc = [200, 200, 200], [10, 10, 10], [3, 3, 3]
    idx = np.tile(np.array([0, 4, 9, -1, -1, -1, -1, -1, -1, -1], dtype=np.int32), (3, 1))
    bt, refs = _table(rng, lens, 12, 4)
    host, dev0 = _pool(torch, 12, "bf16", rng)
    good = O.Pages(bt, refs, np.array(lens, dtype=np.int32), host)
    changes = [("lens", 257), ("lens", 9), ("lens", -1), ("nodes", 11), ("nodes", -1), ("nodes", 201), ("acc", 11),
               ("acc", -1), ("idx", 10), ("idx", 4), ("idx", 2), ("idx", -3), ("bt", 12), ("bt", -1)]
    for what, v in changes:
        a = dict(lens=np.array(lens), nodes=np.array(nodes), acc=np.array(acc), idx=idx.copy(), bt=bt.copy())
        if what == "idx":
            a["idx"][1, 2] = v
        elif what == "bt":
            a["bt"][1, 3] = v       # the page of rows 192 .. 199, some of the nodes'
        else:
            a[what][1] = v
        dev, new = dev0.clone(), torch.full((3,), -7, dtype=torch.int32, device="cuda")
        assert mla.mla_cache_compact(mla.cache_from_pool(dev), _i32(torch, a["bt"]), 4, 4, _i32(torch, a["lens"]),
                                     _i32(torch, a["nodes"]), _i32(torch, a["acc"]), _i32(torch, a["idx"]), 3, 10,
                                     new) == mla.MLA_OK
        _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
        g = O.Pages(bt, refs, np.array(lens, dtype=np.int32), host)
        g.compact(np.array(nodes), np.array([3, 0, 3]), idx)
        assert new.tolist() == [193, int(a["lens"][1]), 193], (what, v)
        assert np.array_equal(dev.cpu().numpy().view(np.uint16), g.pool), (what, v)
    assert good.pool is not None


@pytest.mark.parametrize("kind", ["bf16", "split", "fp8"])
def test_cache_copy(mla, cuda, kind):
    import torch
    rng = np.random.default_rng(2)
    nb = 40
    host, dev = _pool(torch, nb, kind, rng)
    order = rng.permutation(nb)[:24]
    copies = np.stack([np.repeat(order[:6], 3), order[6:], rng.integers(0, 65, 18)]).astype(np.int32)
    copies[2, :4] = 64, 1, 0, 63
    g = O.Pages(np.zeros((1, 1), np.int32), np.zeros(nb, np.int32), np.zeros(1, np.int32), host)
    g.copy(copies)

    def call(c, pool):
        if kind == "fp8":
            return mla.mla_cache_copy_fp8(pool, nb, _i32(torch, c), c.shape[1]), pool
        if kind == "split":
            a, r = _split(torch, pool)
            s = mla.mla_cache_copy(mla.cache_from_split(a, r), _i32(torch, c), c.shape[1])
            assert (a[..., 512:] == 5).all() and (r[..., 64:] == 5).all()
            return s, torch.cat([a[..., :512], r[..., :64]], -1)
        return mla.mla_cache_copy(mla.cache_from_pool(pool), _i32(torch, c), c.shape[1]), pool

    s, got = call(copies, dev.clone())
    assert s == mla.MLA_OK
    _ok(mla, torch)
    assert np.array_equal(got.cpu().numpy().view(host.dtype), g.pool)
    for row, v in ((0, nb), (0, -1), (1, nb), (1, -1), (2, 65), (2, -1)):
        bad = copies.copy()
        bad[row, 0] = v
        s, got = call(bad, dev.clone())
        assert s == mla.MLA_OK
        _ok(mla, torch, mla.MLA_ERR_DEVICE_CHECK)
        h = O.Pages(np.zeros((1, 1), np.int32), np.zeros(nb, np.int32), np.zeros(1, np.int32), host)
        h.copy(copies[:, 1:])
        assert np.array_equal(got.cpu().numpy().view(host.dtype), h.pool)


def test_large_pool_offsets_pass_32_bits(mla, cuda):
    """A pool of more than 2^32 bytes: rows at its end move and copy."""
    import torch
    nb = 60000                       # 4.4 GB
    pool = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    pool[nb - 1] = torch.arange(64, device="cuda").to(torch.bfloat16)[:, None]
    bt = _i32(torch, [[nb - 1]])
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mla.mla_cache_compact(mla.cache_from_pool(pool), bt, 1, 1, _i32(torch, [64]), _i32(torch, [10]),
                                 _i32(torch, [2]), _i32(torch, [[3, 9, 0, 0, 0, 0, 0, 0, 0, 0]]), 1, 10, new) == mla.MLA_OK
    assert mla.mla_cache_copy(mla.cache_from_pool(pool), _i32(torch, [[nb - 1], [nb - 2], [60]]), 1) == mla.MLA_OK
    _ok(mla, torch)
    assert new.tolist() == [56]
    assert pool[nb - 1, 54, 0] == 57 and pool[nb - 1, 55, 575] == 63 and pool[nb - 1, 56, 0] == 56
    assert torch.equal(pool[nb - 2, :60], pool[nb - 1, :60]) and (pool[nb - 2, 60:] == 0).all()
    assert (pool[:16] == 0).all()


def test_pages_captured_and_replayed(mla, cuda):
    import torch
    rng = np.random.default_rng(0)
    lens = np.array([100, 70, 30, 90], dtype=np.int32)
    bt, refs = _table(rng, lens, 12, 3)
    g = O.Pages(bt, refs, lens)
    d = Dev(mla, torch, g)
    keep, src, dst = _i32(torch, [100, 70, 0, 0]), _i32(torch, [0, 1]), _i32(torch, [2, 3])
    copies = torch.zeros((3, 4), dtype=torch.int32, device="cuda")[:, :2].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert d.resize(keep) == mla.MLA_OK
        assert mla.mla_pages_fork(d.refs, d.nb, d.full, d.stride, d.mp, d.lens, d.B, src, dst, 2, copies) == mla.MLA_OK
    for _ in range(3):
        graph.replay()
        _ok(mla, torch)
        g.resize([100, 70, 0, 0])
        want = g.fork([0, 1], [2, 3])
        d.same(g)
        assert np.array_equal(copies.cpu().numpy(), want)
