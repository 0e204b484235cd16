"""Tree attention against the float64 oracle (tolerances of tests/_tol.py: bf16 inputs, P and
outputs rounded to bf16, fp32 sums, as for the decode whose kernel this is)."""
import numpy as np
import pytest

from mla_latent_cache_gb300 import workloads as W
from oracle import spec_oracle as O
from tests._tol import parity

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


class Tree:
    """One batch: a workload of the decode's recipe (NaN past every sequence's end) and a mask."""

    def __init__(self, mla, torch, cuda, H, lens, T, nodes=None, see=None, seed=7, sharp=True, fp8=False, slots=0,
                 override=0, split=False, ahead=True):
        from mla_latent_cache_gb300.runtime import _u16_to_bf16, pool_to_device
        self.mla, self.torch = mla, torch
        w = self.w = W.custom_workload(H, lens, T=T, seed=seed, sharp=sharp)
        B = len(lens)
        rng = np.random.default_rng([seed, 5])
        self.nodes = np.full(B, T) if nodes is None else np.array(nodes)
        if see is None:
            par = np.tile(np.arange(-1, T - 1), (B, 1))
            for t in range(1, T):
                par[:, t] = rng.integers(0, t, B)
            see = O.ancestors(par)
        self.see = see
        self.geom = mla.make_geom(H)
        self.batch = mla.make_batch(B, T, False, w.max_pages, slots, override)
        self.pool = pool_to_device(torch, w, cuda)
        self.fp8 = fp8
        if split:
            self.ckv, self.kpe = self.pool[..., :512].contiguous(), self.pool[..., 512:].contiguous()
            self.cache = mla.cache_from_split(self.ckv, self.kpe)
        else:
            self.cache = mla.cache_from_pool(self.pool)
        if fp8:
            self.rows = torch.empty((w.num_blocks, 64, 656), dtype=torch.uint8, device=cuda)
            mla.check(mla.mla_fp8_pack_cache(self.cache, self.rows))
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(cuda)  # noqa: E731
        self.bt, self.lens = i32(w.block_table), i32(w.seq_lens)
        self.node_lens = None if nodes is None else i32(self.nodes)
        self.mask = i32(O.see_words(see))
        self.q_lat, self.q_pe = _u16_to_bf16(torch, w.q_lat, cuda), _u16_to_bf16(torch, w.q_pe, cuda)
        self.o = torch.full((B, T, H, 512), float("nan"), dtype=torch.bfloat16, device=cuda)
        self.lse = torch.full((B, T, H), float("nan"), dtype=torch.float32, device=cuda)
        # FP8: room to convert the pages ahead, or (ahead=False) as much as the plan needs
        size = mla.mla_tree_fp8_workspace_size if fp8 and ahead else mla.mla_workspace_size
        self.ws_bytes = size(self.geom, self.batch)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=cuda)

    def plan(self):
        self.mla.check(self.mla.mla_plan_tree(self.geom, self.batch, self.lens, self.node_lens, self.ws, self.ws_bytes))

    def decode(self, checked=1):
        if self.fp8:
            s = self.mla.mla_decode_tree_fp8(self.geom, self.batch, self.q_lat, self.q_pe, self.rows, self.w.num_blocks,
                                             self.bt, self.bt.shape[1], self.lens, self.node_lens, self.mask, checked,
                                             self.o, self.lse, self.ws, self.ws_bytes)
        else:
            s = self.mla.mla_decode_tree(self.geom, self.batch, self.q_lat, self.q_pe, self.cache, self.bt,
                                         self.bt.shape[1], self.lens, self.node_lens, self.mask, checked, self.o,
                                         self.lse, self.ws, self.ws_bytes)
        assert s == self.mla.MLA_OK, self.mla.mla_status_string(s)

    def run(self, expect=None, checked=1):
        self.plan()
        self.decode(checked)
        self.torch.cuda.synchronize()
        status, info = self.mla.mla_read_device_status(self.ws)
        assert status == (self.mla.MLA_OK if expect is None else expect), (self.mla.mla_status_string(status), info)
        return self

    def check(self, sequences=None):
        w = self.w
        f = W.bf16_bits_to_f64
        pool, bt = w.compact_view()
        pool = f(pool)
        if self.fp8:
            ids = self.torch.from_numpy(w.pool_ids).to(self.rows.device)
            r = self.rows[ids].cpu()
            lat = r[..., :512].contiguous().view(self.torch.float8_e4m3fn).float().view(*r.shape[:2], 4, 128)
            sc = r[..., 512:528].contiguous().view(self.torch.float32)
            pool = np.concatenate([(lat * sc[..., None]).reshape(*r.shape[:2], 512).numpy().astype(np.float64),
                                   pool[..., 512:]], -1)
        sel = range(w.B) if sequences is None else sequences
        ro, rl = O.tree_decode_ref(f(w.q_lat)[list(sel)], f(w.q_pe)[list(sel)], pool, bt[list(sel)],
                                   w.seq_lens[list(sel)], self.nodes[list(sel)], self.see[list(sel)])
        parity(_np(self.o)[list(sel)], ro, "o_lat")
        parity(self.lse.cpu().numpy()[list(sel)].astype(np.float64), rl, "lse")
        assert np.all(_np(self.o)[list(sel)][np.isneginf(rl)] == 0)
        return self


# lengths where the nodes start, end and straddle at page and 16-column borders
@pytest.mark.parametrize("H,lens,T", [
    (16, [512], 8), (128, [1], 1), (128, [3, 64, 65, 128], 3), (1, [40, 41, 200], 40), (8, [63, 64, 65, 127, 129], 33),
    (64, [100, 1000, 4096], 5), (128, [70, 300, 131, 2000], 17), (2, [64, 128, 192, 500], 64), (32, [200, 130], 130),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_matches_the_oracle(mla, cuda, H, lens, T, fp8):
    import torch
    Tree(mla, torch, cuda, H, lens, T, fp8=fp8, sharp=not fp8).run().check()


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_padded_batches(mla, cuda, H, fp8):
    """Fewer nodes than T, none, a sequence of nodes alone, an empty sequence, nodes shorter than T rows."""
    import torch
    t = Tree(mla, torch, cuda, H, [300, 64, 7, 0, 5, 1000, 77], 12, nodes=[12, 3, 7, 0, 2, 0, 11], fp8=fp8, sharp=not fp8)
    t.run().check()
    assert torch.isneginf(t.lse[3]).all() and torch.isneginf(t.lse[5]).all()
    # an empty sequence in a batch without counts
    Tree(mla, torch, cuda, H, [300, 0, 64], 12, fp8=fp8, sharp=not fp8).run().check()


@pytest.mark.parametrize("H", [8, 128])
@pytest.mark.parametrize("override,slots", [(0, 0), (0, 2), (3, 0)])
def test_any_mask_and_splits(mla, cuda, H, override, slots):
    """Masks that are no tree, rows that see nothing (no prefix either), work split over the cache."""
    import torch
    rng = np.random.default_rng(3)
    T = 20
    see = rng.random((4, T, T)) < 0.3
    see[:, 4] = False
    see[1] = False
    see[2] = True
    t = Tree(mla, torch, cuda, H, [700, 20, 150, 2500], T, see=see, slots=slots, override=override).run().check()
    assert torch.isneginf(t.lse[1]).all() and not torch.isneginf(t.lse[0]).any()
    assert (t.o[1] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [4, 128])
def test_unseen_rows_may_hold_anything(mla, cuda, H, fp8):
    """NaN and infinities in the rows of nodes that no node sees: the other nodes are unaffected."""
    import torch
    T = 70
    see = np.tril(np.random.default_rng(2).random((2, T, T)) < 0.6)
    dead = [0, 5, 17, 18, 40, 64, 69]
    see[:, :, dead] = False
    t = Tree(mla, torch, cuda, H, [200, 71], T, see=see, fp8=fp8, sharp=not fp8)
    w = t.w
    for b in range(2):
        for k, u in enumerate(dead):
            j = int(w.seq_lens[b]) - T + u
            blk = int(w.block_table[b, j // 64])
            v = (float("nan"), float("inf"), -float("inf"))[k % 3]
            if fp8:
                t.rows[blk, j % 64, :512] = 0x7F
                t.rows[blk, j % 64, 528:].view(torch.bfloat16)[:] = v
            else:
                t.pool[blk, j % 64] = v
    t.run().check()


@pytest.mark.parametrize("H,lens,T,nodes", [(128, [70, 300, 0, 131, 2000], 17, [17, 3, 0, 9, 17]),
                                              (16, [64, 1000, 65], 20, None)])
def test_fp8_pages_converted_ahead_or_by_each_group(mla, cuda, H, lens, T, nodes):
    """The same values either way (equal bits: the same products, rounded alike, in the same schedule)."""
    import torch
    a = Tree(mla, torch, cuda, H, lens, T, nodes=nodes, fp8=True, sharp=False).run().check()
    b = Tree(mla, torch, cuda, H, lens, T, nodes=nodes, fp8=True, sharp=False, ahead=False).run().check()
    assert a.ws_bytes > b.ws_bytes
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)
    # a block outside the pool reads as zeros and is reported, converted ahead too
    for t in (a, b):
        t.bt[1, 0] = t.w.num_blocks
        t.run(expect=mla.MLA_ERR_DEVICE_CHECK)
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)


def test_chain_is_the_causal_decode(mla, cuda):
    """A chain's tree is the causal decode of its rows."""
    import torch
    for H, T in ((128, 4), (16, 9)):
        lens = [500, 64, 130]
        see = O.ancestors(np.tile(np.arange(-1, T - 1), (3, 1)))
        t = Tree(mla, torch, cuda, H, lens, T, see=see, override=2).run()
        batch = mla.make_batch(3, T, True, t.w.max_pages, 0, 2)
        ws = torch.zeros(mla.mla_workspace_size(t.geom, batch), dtype=torch.uint8, device=cuda)
        o, lse = torch.empty_like(t.o), torch.empty_like(t.lse)
        mla.check(mla.mla_plan(t.geom, batch, t.lens, ws, ws.numel()))
        mla.check(mla.mla_decode(t.geom, batch, t.q_lat, t.q_pe, t.cache, t.bt, t.bt.shape[1], t.lens, 1, o, lse, ws, ws.numel()))
        torch.cuda.synchronize()
        assert mla.mla_read_device_status(ws)[0] == mla.MLA_OK
        parity(_np(t.o), _np(o))
        parity(_np(t.lse), _np(lse))


def test_v3_batch_sampled(mla, cuda):
    import torch
    rng = np.random.default_rng(11)
    lens = np.exp(rng.uniform(np.log(300), np.log(5000), 24)).astype(int)
    nodes = rng.integers(1, 17, 24)
    Tree(mla, torch, cuda, 128, lens, 16, nodes=nodes).run().check(sequences=[0, 7, 23])


def test_long_context_and_split_pools(mla, cuda):
    import torch
    Tree(mla, torch, cuda, 128, [30001], 3).run().check()
    Tree(mla, torch, cuda, 16, [1000, 130], 20, split=True).run().check()


def test_1024_nodes(mla, cuda):
    import torch
    Tree(mla, torch, cuda, 1, [1100, 1024], 1024, nodes=[1024, 900], sharp=False).run().check()


def test_device_checks(mla, cuda):
    import torch
    # stale plans: other node counts, a plan of the plain decode; counts out of range; a bad block
    t = Tree(mla, torch, cuda, 16, [300, 200], 8, nodes=[8, 5])
    t.plan()
    t.node_lens[1] = 6
    t.decode()
    assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_ERR_PLAN_STALE
    mla.check(mla.mla_plan(t.geom, t.batch, t.lens, t.ws, t.ws_bytes))
    t.decode()
    assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_ERR_PLAN_STALE
    t.plan()
    mla.check(mla.mla_decode(t.geom, t.batch, t.q_lat, t.q_pe, t.cache, t.bt, t.bt.shape[1], t.lens, 1, t.o, t.lse, t.ws, t.ws_bytes))
    assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_ERR_PLAN_STALE
    for n, counted in ((9, 8), (-1, 0), (2 ** 31 - 1, 8), (-2 ** 31, 0)):
        t.node_lens[1] = n
        t.plan()
        t.decode(checked=0)
        assert mla.mla_read_device_status(t.ws) == (mla.MLA_ERR_DEVICE_CHECK, 1)
        t.nodes[1] = counted
        t.check()
    t.node_lens[1] = 5
    t.lens[1] = 3              # fewer rows than nodes
    t.plan()
    assert mla.mla_read_device_status(t.ws) == (mla.MLA_ERR_DEVICE_CHECK, 1)
    t.lens[1] = 200
    t.bt[1, 0] = t.w.num_blocks
    t.plan()
    t.decode()
    assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_ERR_DEVICE_CHECK


def test_captured_and_replayed_with_new_lengths(mla, cuda):
    import torch
    t = Tree(mla, torch, cuda, 128, [700, 64, 1500], 9, nodes=[9, 4, 9])
    t.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.plan()
        t.decode()
    t.node_lens.copy_(torch.tensor([2, 9, 0], dtype=torch.int32))
    t.nodes = np.array([2, 9, 0])
    t.o.fill_(float("nan"))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_OK
    t.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_timeouts_are_reported_and_recoverable(mla, cuda, fp8):
    """Pipeline waits shortened to a few cycles (nothing faults): the launch reports and the next one is right."""
    import torch
    t = Tree(mla, torch, cuda, 128, [1024, 1000, 1024, 990], 3, fp8=fp8, sharp=not fp8, slots=12, ahead=False)
    t.plan()
    torch.cuda.synchronize()
    assert int(t.ws[:256].view(torch.int32)[mla.HDR["NUM_MERGE"]]) == 0
    try:
        mla.check(mla.mla_debug_set_wait_limit(16), "set wait limit")
        for _ in range(2):
            t.plan()
            t.decode(checked=0)
            torch.cuda.synchronize()
            status, info = mla.mla_read_device_status(t.ws)
            assert status == mla.MLA_ERR_TIMEOUT and info > 0
    finally:
        mla.check(mla.mla_debug_set_wait_limit(0), "reset wait limit")
    t.run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_at_the_end_of_a_large_pool(mla, cuda, fp8):
    """Blocks whose byte offsets pass 32 bits give the bits of the same pages in a small pool."""
    import torch
    t = Tree(mla, torch, cuda, 16, [300, 70], 20, fp8=fp8, sharp=not fp8).run()
    o, lse = t.o.clone(), t.lse.clone()
    nb, small = 110000, t.rows if fp8 else t.pool
    big = torch.zeros((nb, *small.shape[1:]), dtype=small.dtype, device=cuda)
    big[nb - len(small):] = small
    t.bt[t.bt >= 0] += nb - len(small)
    t.rows = big if fp8 else None
    t.cache = None if fp8 else mla.cache_from_pool(big)
    t.w.num_blocks = nb
    t.o.fill_(float("nan"))
    t.run()
    assert torch.equal(t.o, o) and torch.equal(t.lse, lse)


def test_two_streams_at_once(mla, cuda):
    """Two trees decoded on two streams with workspaces of their own."""
    import torch
    a = Tree(mla, torch, cuda, 128, [2000, 900], 6, seed=1)
    b = Tree(mla, torch, cuda, 16, [700, 64, 1500], 30, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for t, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                t.plan()
                t.decode()
    torch.cuda.synchronize()
    for t in (a, b):
        assert mla.mla_read_device_status(t.ws)[0] == mla.MLA_OK
        t.check()
