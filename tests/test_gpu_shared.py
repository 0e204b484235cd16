"""Attention over shared prefixes against the float64 oracle (tolerances of tests/_tol.py: bf16 inputs, P
and outputs rounded to bf16, fp32 sums, as for the decode whose kernel this is)."""
import numpy as np
import pytest

from oracle import serve_oracle as O
from tests._tol import parity

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


class Shared:
    """A batch of sets [(members, prefix rows)] and loose sequences; rows past a sequence's end, blocks that nobody
    holds and queries of tokens that are not there hold NaN.  own: rows of each sequence past its prefix."""

    def __init__(self, mla, torch, H, sets, own, T=1, counts=None, causal=False, fp8=False, slots=0, override=0, seed=0,
                 empty=(), lists=None, split=False):
        rng = np.random.default_rng([seed, H, T])
        B = self.B = len(own)
        self.mla, self.torch, self.H, self.T, self.fp8 = mla, torch, H, T, fp8
        ptr = np.concatenate([[0], np.cumsum([m for m, _ in sets])]).astype(np.int32)
        prefix = np.array([p for _, p in sets], dtype=np.int32)
        of = np.zeros(B, dtype=np.int64)
        for p in range(len(sets)):
            of[ptr[p]:ptr[p + 1]] = prefix[p]
        self.counts = np.full(B, T) if counts is None else np.array(counts)
        lens = of + np.array(own, dtype=np.int64)
        lens[list(empty)] = 0
        self.lens = lens
        pages = (lens + 63) // 64
        nb = self.num_blocks = int(pages.sum()) + 3
        order = rng.permutation(nb)
        bt = np.full((B, int(max(1, pages.max())) + 2), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            bt[b, :pages[b]] = order[at:at + pages[b]]
            at += int(pages[b])
        for p in range(len(sets)):
            live = [b for b in range(ptr[p], ptr[p + 1]) if lens[b] > 0]
            for b in live:
                n = min(int(prefix[p]), int(lens[b]), int(lens[live[0]])) // 64
                bt[b, :n] = bt[live[0], :n]
        self.bt = bt
        pool = torch.full((nb, 64, 576), float("nan"), dtype=torch.bfloat16)
        for b in range(B):
            for k in range(int(pages[b])):
                n = min(64, int(lens[b]) - 64 * k)
                if torch.isnan(pool[bt[b, k], 0, 0]):
                    pool[bt[b, k], :n] = torch.from_numpy(rng.normal(size=(n, 576)) * 0.1).bfloat16()
        self.host_pool = pool
        self.pool = pool.cuda()
        self.ckv, self.kpe = (self.pool[..., :512].contiguous(), self.pool[..., 512:].contiguous()) if split else (None, None)
        self.cache = mla.cache_from_split(self.ckv, self.kpe) if split else mla.cache_from_pool(self.pool)
        if fp8:
            self.rows = torch.empty((nb, 64, 656), dtype=torch.uint8, device="cuda")
            mla.check(mla.mla_fp8_pack_cache(mla.cache_from_pool(torch.nan_to_num(self.pool)), self.rows))
            r = self.rows.cpu()
            lat = r[..., :512].contiguous().view(torch.float8_e4m3fn).float().view(nb, 64, 4, 128)
            sc = r[..., 512:528].contiguous().view(torch.float32)
            self.f64 = np.concatenate([(lat * sc[..., None]).reshape(nb, 64, 512).double().numpy(),
                                       torch.nan_to_num(pool[..., 512:]).double().numpy()], -1)
            # rows past the ends: codes, scales and RoPE values that are NaN
            self.rows[torch.isnan(self.pool[..., 0])] = 0xFF
        else:
            self.f64 = torch.nan_to_num(pool).double().numpy()
        q = torch.from_numpy(rng.normal(size=(B, T, H, 576)) * 12).bfloat16()
        for b in range(B):
            q[b, int(self.counts[b]) if lens[b] else 0:] = float("nan")
        self.q = q
        self.q_lat, self.q_pe = q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.d_bt, self.d_lens, self.d_counts = i32(bt), i32(lens), None if counts is None else i32(self.counts)
        self.num_sets = len(sets)
        self.ptr, self.prefix = (i32(ptr), i32(prefix)) if lists is None else (i32(lists[0]), i32(lists[1]))
        self.causal = causal
        self.geom = mla.make_geom(H)
        self.batch = mla.make_batch(B, T, causal, int(max(1, pages.max())), slots, override)
        self.ws_bytes = mla.mla_shared_workspace_size(self.geom, self.batch)
        assert self.ws_bytes > 0
        self.ws = torch.full((self.ws_bytes,), 0x5A, dtype=torch.uint8, device="cuda")
        self.o = torch.full((B, T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, T, H), float("nan"), dtype=torch.float32, device="cuda")

    def plan(self, stream=None):
        self.mla.check(self.mla.mla_plan_shared(self.geom, self.batch, self.d_lens, self.d_counts, self.num_sets, self.ptr,
                                                self.prefix, self.ws, self.ws_bytes, stream))

    def decode(self, checked=1, stream=None):
        tail = (self.d_bt, self.bt.shape[1], self.d_lens, self.d_counts, checked, self.o, self.lse, self.ws, self.ws_bytes,
                stream)
        if self.fp8:
            s = self.mla.mla_decode_shared_fp8(self.geom, self.batch, self.q_lat, self.q_pe, self.rows, self.num_blocks, *tail)
        else:
            s = self.mla.mla_decode_shared(self.geom, self.batch, self.q_lat, self.q_pe, self.cache, *tail)
        assert s == self.mla.MLA_OK, self.mla.mla_status_string(s)

    def status(self):
        self.torch.cuda.synchronize()
        return self.mla.mla_read_device_status(self.ws)

    def run(self, expect=None, checked=1):
        self.plan()
        self.decode(checked)
        status, info = self.status()
        assert status == (self.mla.MLA_OK if expect is None else expect), (self.mla.mla_status_string(status), info)
        return self

    def check(self):
        f = self.torch.nan_to_num(self.q).double().numpy()
        ro, rl = O.ragged_decode_ref(f[..., :512], f[..., 512:], self.f64, self.bt, self.lens, self.counts, self.causal)
        parity(_np(self.o), ro, "o_lat")
        parity(_np(self.lse), rl, "lse")
        assert np.all(_np(self.o)[np.isneginf(rl)] == 0)
        return self

    def header(self):
        return self.ws[:256].view(self.torch.int32).cpu().numpy()

    def set_groups(self):
        """How many groups of the plan stand for shared pages: as many as the rule gives."""
        R = self.T * self.H
        n = int(self.header()[self.mla.HDR["NUM_GROUPS"]]) - self.B * ((R + 127) // 128)
        if self.ptr is not None:
            ptr, prefix = self.ptr.cpu().numpy(), self.prefix.cpu().numpy()
            if (np.diff(ptr) >= 0).all() and ptr[0] >= 0 and ptr[-1] <= self.B and (prefix >= 0).all():
                G = int(self.header()[self.mla.HDR["NUM_SLOTS"]])
                pages = O.shared_pages_ref(self.lens, self.counts, ptr, prefix, self.T, self.H, self.causal, G)
                assert n == sum((m * R + 127) // 128 for m, k in zip(np.diff(ptr), pages) if k)
        return n

    def covered(self):
        """Every visible (query row, page) is in exactly one segment, and a row's parts are merged or final."""
        h = self.header()
        HDR, R = self.mla.HDR, self.T * self.H
        n = int(h[HDR["NUM_SEGMENTS"]])
        off = int(h[HDR["OFF_SEGMENTS"]])
        seg = self.ws[off:off + 32 * n].view(self.torch.int32).cpu().numpy().reshape(n, 8)
        seen = np.zeros((self.B * R, self.bt.shape[1]), dtype=np.int64)
        rows = np.zeros(max(1, int(h[HDR["NUM_PARTIALS"]])), dtype=np.int64)
        for table, row0, p0, p1, rng, part, group, flag in seg:
            m = flag & 0xFFFF
            assert p0 < p1 and 0 < m <= 128
            seen[row0:row0 + m, p0:p1] += 1
            for b in range(row0 // R, (row0 + m - 1) // R + 1):       # the same blocks, whichever table row is read
                if self.lens[b] and self.counts[b]:
                    k = min(p1, (int(self.lens[b]) + 63) // 64)
                    assert np.array_equal(self.bt[table, p0:k], self.bt[b, p0:k])
            if part >= 0:
                rows[part:part + m] += 1
        assert rows.max(initial=0) <= 1
        assert int(h[HDR["NUM_PARTIALS"]]) <= int(h[HDR["CAP_PARTIALS"]]) and n <= int(h[HDR["CAP_SEGMENTS"]])
        for b in range(self.B):
            for t in range(int(self.counts[b])):
                S = int(self.lens[b])
                vis = max(0, min(S, S - int(self.counts[b]) + t + 1)) if self.causal else S
                for r in range(b * R + t * self.H, b * R + (t + 1) * self.H):
                    assert np.all(seen[r, :(vis + 63) // 64] == 1), (b, t)
        return self


@pytest.mark.parametrize("H,T", [(1, 1), (1, 3), (8, 1), (8, 3), (16, 1), (16, 3), (32, 1), (32, 5), (64, 1), (64, 3), (128, 1),
                                 (128, 2)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_sets_of_all_sizes(mla, cuda, H, T, causal, fp8):
    import torch
    rng = np.random.default_rng([H, T])
    sets = [(9, 1300), (1, 700), (5, 64), (2, 63), (12, 6000), (3, 900)]
    B = sum(m for m, _ in sets) + 3
    own = rng.integers(T, 200, B)
    own[0], own[3], own[12] = T, 64, 128
    counts = rng.integers(0 if B % 2 else 1, T + 1, B)
    counts[1] = T
    s = Shared(mla, torch, H, sets, own, T, counts, causal, fp8, seed=H + T, slots=8 if T > 1 else 0).run().covered().check()
    shares = (T * H) % 128 != 0
    assert (s.set_groups() > 0) == shares
    # the counters of the merge are as they were: again without a new plan, and with one
    o, lse = s.o.clone(), s.lse.clone()
    for again in range(3):
        s.o.fill_(float("nan"))
        s.lse.fill_(float("nan"))
        if again == 2:
            s.plan()
        s.decode()
        assert s.status()[0] == mla.MLA_OK
        assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("slots,override", [(1, 0), (2, 0), (7, 0), (40, 0), (0, 1), (0, 3), (5, 20), (0, 64)])
def test_splits(mla, cuda, slots, override):
    """From one range to as many as pages: up to more than sixteen parts per row, in two places."""
    import torch
    rng = np.random.default_rng(1)
    for H, T, sets in ((16, 3, [(11, 9000), (6, 640)]), (8, 1, [(30, 4096)])):
        B = sum(m for m, _ in sets) + 1
        own = rng.integers(T, 1400, B)
        s = Shared(mla, torch, H, sets, own, T, None, True, slots=slots, override=override, seed=2).run().covered().check()
        assert s.set_groups() > 0


def test_long_own_rows_and_long_prefixes(mla, cuda):
    import torch
    own = np.full(24, 40)
    own[5], own[20] = 9000, 3000
    s = Shared(mla, torch, 16, [(20, 20000), (4, 128)], own).run().covered().check()
    assert s.set_groups() > 0
    Shared(mla, torch, 32, [(12, 12345)], np.arange(1, 13) * 7, fp8=True).run().covered().check()


def test_empty_sequences_and_tokens(mla, cuda):
    """Empty members (the set's first among them), members without tokens, sets of nothing, nothing at all."""
    import torch
    sets = [(12, 1100), (0, 500), (10, 1500)]
    B = 24
    own = np.full(B, 30)
    counts = np.full(B, 2)
    counts[[3, 13, 23]] = 0
    counts[5] = 1
    for causal in (False, True):
        s = Shared(mla, torch, 16, sets, own, 2, counts, causal, empty=(0, 1, 7, 22), slots=16).run().covered().check()
        assert s.set_groups() > 0
    Shared(mla, torch, 16, [(10, 1100)], np.zeros(10) + 5, empty=range(1, 10)).run().covered().check()
    s = Shared(mla, torch, 16, [(10, 1100)], np.zeros(10) + 5, empty=range(10)).run().check()
    assert s.set_groups() == 0
    Shared(mla, torch, 16, [(10, 1100)], np.zeros(10) + 5, 1, np.zeros(10)).run().check()


def test_what_the_members_see_bounds_what_is_shared(mla, cuda):
    """Prefix lengths past a member's rows, or past what its first token sees, are cut to whole pages that all see."""
    import torch
    sets, own = [(16, 1024)], np.full(16, 1)
    # with 3 tokens per sequence the rows of the first ones lie inside the prefix
    s = Shared(mla, torch, 16, sets, own + 2, 3, None, True, lists=([0, 16], [1 << 30]), slots=8).run().covered().check()
    assert s.set_groups() > 0
    s = Shared(mla, torch, 16, sets, own - 1, 3, None, True, slots=8).run().covered().check()      # its last page is not whole for all
    assert s.set_groups() > 0
    # a sequence that is shorter than the others' prefix
    s = Shared(mla, torch, 16, [(16, 1024)], np.where(np.arange(16) == 3, -300, 20), 1, slots=8).run().covered().check()
    assert s.set_groups() > 0


def test_without_sets_it_is_the_decode(mla, cuda):
    import torch
    own = np.array([900, 5, 64, 3000, 1, 777])
    for H, T in ((16, 1), (128, 2), (64, 3)):
        s = Shared(mla, torch, H, [], np.maximum(own, T), T, None, True)
        s.ptr = s.prefix = None
        s.run().covered().check()
        ws = torch.zeros(mla.mla_workspace_size(s.geom, s.batch), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(s.o), torch.empty_like(s.lse)
        assert mla.mla_plan(s.geom, s.batch, s.d_lens, ws, ws.numel()) == mla.MLA_OK
        assert mla.mla_decode(s.geom, s.batch, s.q_lat, s.q_pe, s.cache, s.d_bt, s.bt.shape[1], s.d_lens, 0, o, lse, ws,
                              ws.numel()) == mla.MLA_OK
        torch.cuda.synchronize()
        parity(_np(s.o), _np(o), "o", max_rel=8e-3, mean_rel=4e-3)     # (two roundings of half a bf16 step, 2^-8 each)


def test_split_pools_and_many_sequences(mla, cuda):
    import torch
    Shared(mla, torch, 16, [(9, 700)], np.arange(1, 10), split=True).run().covered().check()
    B = 1500
    rng = np.random.default_rng(4)
    sets = [(10, int(p)) for p in rng.integers(0, 700, 140)]
    s = Shared(mla, torch, 8, sets, rng.integers(1, 40, B)).run().check()
    assert s.set_groups() > 0


def test_most_sets_and_sequences(mla, cuda):
    """8192 sequences; 2048 sets of four."""
    import torch
    B = 8192
    rng = np.random.default_rng(4)
    s = Shared(mla, torch, 8, [(4, 1024)] * (B // 4), rng.integers(1, 20, B))
    s.run()
    assert s.set_groups() == B // 4
    f = s.torch.nan_to_num(s.q).double().numpy()
    for part in (slice(0, 60), slice(5000, 5060), slice(B - 60, B)):
        ro, rl = O.ragged_decode_ref(f[part, ..., :512], f[part, ..., 512:], s.f64, s.bt[part], s.lens[part], s.counts[part], False)
        parity(_np(s.o[part]), ro, "o_lat")
        parity(_np(s.lse[part]), rl, "lse")


def test_problems_are_reported(mla, cuda):
    import torch
    own = np.full(12, 9)
    bad = mla.MLA_ERR_DEVICE_CHECK
    for lists in (([0, 13], [1024]), ([-1, 12], [1024]), ([5, 3], [1024]), ([0, 12], [-1])):
        s = Shared(mla, torch, 16, [(12, 1024)], own, lists=lists).run(expect=bad).check()
        assert s.set_groups() == 0 and s.status()[1] == 12
    # lengths beyond the table, more tokens than T, more tokens than rows
    s = Shared(mla, torch, 16, [(12, 1024)], own)
    s.d_lens[4] = 64 * s.batch.max_pages + 1
    s.run(expect=bad)
    assert s.status()[1] == 4
    s = Shared(mla, torch, 16, [(12, 1024)], own, 2, np.full(12, 2))
    s.d_counts[7] = 3
    s.run(expect=bad)
    assert s.status()[1] == 7
    # a block outside the pool (checked), and a plan made for other lengths or counts
    s = Shared(mla, torch, 16, [(12, 1024)], own)
    s.d_bt[5, 16] = s.num_blocks
    s.run(expect=bad)
    for what in ("lens", "counts"):
        s = Shared(mla, torch, 16, [(12, 1024)], own, 2, np.full(12, 2))
        s.plan()
        (s.d_lens if what == "lens" else s.d_counts)[3] -= 1
        s.decode()
        assert s.status()[0] == mla.MLA_ERR_PLAN_STALE
    # another kind of plan, one of other sizes, or none: nothing is attended
    for plan in ("dense", "slots", "causal", "none"):
        s = Shared(mla, torch, 16, [(12, 1024)], own, 2)
        s.ws = torch.zeros(4 * s.ws_bytes, dtype=torch.uint8, device="cuda")
        s.ws_bytes = s.ws.numel()
        other = mla.make_batch(s.B, 2, plan == "causal", s.batch.max_pages, 5 if plan == "slots" else 0)
        if plan == "dense":
            mla.check(mla.mla_plan(s.geom, other, s.d_lens, s.ws, s.ws_bytes))
        elif plan != "none":
            mla.check(mla.mla_plan_shared(s.geom, other, s.d_lens, None, 1, s.ptr, s.prefix, s.ws, s.ws_bytes))
        for checked in (0, 1):
            s.decode(checked)
            assert s.status()[0] == mla.MLA_ERR_PLAN_STALE, plan
        assert bool(torch.isnan(s.o.float()).all()) and bool(torch.isnan(s.lse).all())


def test_captured_and_on_another_stream(mla, cuda):
    import torch
    rng = np.random.default_rng(9)
    own = rng.integers(2, 300, 20)
    s = Shared(mla, torch, 16, [(13, 1500), (7, 333)], own, 2, rng.integers(1, 3, 20), True, slots=16).run().check()
    assert s.set_groups() > 0
    o, lse = s.o.clone(), s.lse.clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        s.plan()
        s.decode(0)
    for _ in range(3):
        s.o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.o, o) and torch.equal(s.lse, lse)
    # other lengths in the same graph
    s.lens = np.maximum(s.lens - 40, 2)
    s.d_lens.copy_(torch.from_numpy(s.lens.astype(np.int32)))
    g.replay()
    torch.cuda.synchronize()
    s.check()
    s.o.fill_(float("nan"))
    torch.cuda.synchronize()
    s.plan(side)
    s.decode(1, side)
    side.synchronize()
    s.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("slots", [40, 300])
def test_shared_rows_of_many_parts(mla, cuda, slots, fp8):
    """A few long sequences over many ranges: dozens of parts to a row, and more than are staged at once."""
    import torch
    s = Shared(mla, torch, 16, [(5, 9000)], [8000, 9000, 70, 1, 6000], slots=slots, fp8=fp8, seed=slots)
    s.run().check()
    assert s.header()[mla.HDR["NUM_PARTIALS"]] > 0
    s.run().check()
    if slots == 300:
        s = Shared(mla, torch, 16, [(2, 64)], [9000, 8000], slots=slots, fp8=fp8, seed=slots).run().check()
        assert s.header()[mla.HDR["PAGES_PER_RANGE"]] == 2       # (71 parts)
        s = Shared(mla, torch, 16, [(2, 64)], [20000, 8000], slots=640, fp8=fp8, seed=slots).run().check()
        assert s.header()[mla.HDR["PAGES_PER_RANGE"]] == 2       # (the fewest: 157 parts)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_plan_for_longer_tables(mla, cuda, fp8):
    """A plan for tables of more pages than the decode's may have pages past them: nothing is attended.  One for fewer is used."""
    import torch
    s = Shared(mla, torch, 16, [(12, 1024)], np.arange(1, 13) * 9, fp8=fp8)
    own, B = s.batch, s.B
    s.plan()
    for pages in (own.max_pages - 1, 1):
        s.batch = mla.make_batch(B, 1, False, pages)
        assert mla.mla_shared_workspace_size(s.geom, s.batch) == s.ws_bytes
        for checked in (0, 1):
            s.batch = own
            s.plan()
            s.batch = mla.make_batch(B, 1, False, pages)
            s.decode(checked)
            assert s.status()[0] == mla.MLA_ERR_PLAN_STALE
        assert bool(torch.isnan(s.o.float()).all()) and bool(torch.isnan(s.lse).all())
    s.batch = own
    s.plan()
    s.batch = mla.make_batch(B, 1, False, own.max_pages + 2)       # (as wide as the table is)
    s.decode()
    assert s.status()[0] == mla.MLA_OK
    s.check()


def _decode_rows(s, b, first):
    """Sequence b's tokens over its rows from `first` on."""
    f = s.torch.nan_to_num(s.q).double().numpy()[b:b + 1]
    k = int(s.lens[b]) - first
    blocks = s.bt[b:b + 1, first // 64:]
    return O.ragged_decode_ref(f[..., :512], f[..., 512:], s.f64, blocks, [k], s.counts[b:b + 1], s.causal)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,T", [(16, 1), (16, 3), (64, 1), (64, 3)])
def test_members_that_hold_other_blocks(mla, cuda, H, T, fp8):
    """A sequence in a set that does not hold the set's blocks is reported, checked or not, and sees none of them."""
    import torch
    sets, own = [(30, 4096)], np.concatenate([np.arange(30) * 5 + 4, [4500]])
    for odd, causal in (((3,), False), ((0, 8, 29), True)):
        s = Shared(mla, torch, H, sets, own, T, None, causal, fp8=fp8, slots=16)
        s.bt[list(odd), :64] = s.bt[30, :64]              # (the loose sequence's)
        s.d_bt.copy_(torch.from_numpy(s.bt))
        # through the table row of the first: if that one is odd, it is the others that hold other blocks
        alone = [b for b in range(30) if (s.bt[b, :64] != s.bt[0, :64]).any()]
        assert len(alone) == (1 if 0 not in odd else 27)
        ro, rl = O.ragged_decode_ref(*(torch.nan_to_num(s.q).double().numpy()[..., i:j] for i, j in ((0, 512), (512, 576))), s.f64, s.bt,
                                     s.lens, s.counts, causal)
        for b in alone:
            (ro[b],), (rl[b],) = _decode_rows(s, b, 4096)
        for checked in (0, 1):
            s.o.fill_(float("nan"))
            s.plan()
            assert s.set_groups() > 0
            s.decode(checked)
            status, info = s.status()
            assert status == mla.MLA_ERR_DEVICE_CHECK and info in alone
            parity(_np(s.o), ro, "o_lat")
            parity(_np(s.lse), rl, "lse")


@pytest.mark.parametrize("fp8", [False, True])
def test_one_other_block_among_the_shared(mla, cuda, fp8):
    """Checked, every page of a member is compared with the one that is read."""
    import torch
    for page in (0, 13, 31):
        s = Shared(mla, torch, 16, [(30, 2048)], np.arange(30) * 5 + 4, slots=16, fp8=fp8)
        s.d_bt[17, page] = int(s.bt[2, 32])
        s.run(expect=mla.MLA_ERR_DEVICE_CHECK)
        assert s.set_groups() > 0 and s.status()[1] == 17


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pages,shares", [(6, False), (20, False), (24, False), (29, False), (60, True), (200, True)])
def test_chunks_of_prompts_in_sets(mla, cuda, pages, shares, fp8):
    """Two sequences of 41 tokens x 16 heads each (656 rows): sharing saves one group of twelve, and costs 55 pages; tables of
    25 pages or fewer are laid out without it."""
    import torch
    s = Shared(mla, torch, 16, [(2, 64 * pages)], [50, 41, 3000 if pages == 20 else 60], 41, [41, 30, 41], True, fp8=fp8, slots=2)
    s.run().covered().check()
    assert (s.set_groups() > 0) == shares


def test_members_of_many_that_hold_other_blocks(mla, cuda):
    """As above where a CTA merges more records than it looks up at once, by a thousand and five hundred sequences."""
    import torch
    rng = np.random.default_rng(6)
    B = 1500
    s = Shared(mla, torch, 8, [(10, 700)] * 140, rng.integers(1, 40, B))
    odd = [b for b in range(3, 1400, 97) if b % 10]
    for b in odd:
        s.bt[b, :10] = s.bt[(b + 500) % 1400, :10]            # (another set's)
    s.d_bt.copy_(torch.from_numpy(s.bt))
    f = torch.nan_to_num(s.q).double().numpy()
    ro, rl = O.ragged_decode_ref(f[..., :512], f[..., 512:], s.f64, s.bt, s.lens, s.counts, False)
    for b in odd:
        (ro[b],), (rl[b],) = _decode_rows(s, b, 640)
    s.plan()
    assert s.set_groups() > 0
    s.decode(0)
    status, info = s.status()
    assert status == mla.MLA_ERR_DEVICE_CHECK and info in odd
    parity(_np(s.o), ro, "o_lat")
    parity(_np(s.lse), rl, "lse")
