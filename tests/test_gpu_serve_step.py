"""Serving steps as they are used: a prompt in chunks, forks of it, tokens drawn and decoded with the shared rows attended
once, step after step on one cache, against a float64 history of every sequence's rows."""
import numpy as np
import pytest

from mla_latent_cache_gb300 import workloads as W
from oracle import mla_oracle as M
from oracle import serve_oracle as S
from oracle import spec_oracle as O
from tests._tol import parity

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


class Harness:
    V = 1000

    def __init__(self, torch, cuda, B, H, T, fp8=False, interleaved=True, seed=0, max_pages=12, num_blocks=None, max_sets=4):
        from mla_latent_cache_gb300.runtime import ServeStep
        self.torch, self.T = torch, T
        self.rng = np.random.default_rng([seed, B, H, T])
        self.s = ServeStep(B, H, T, max_pages, num_blocks or max_pages * B, device=cuda, cache_format="fp8" if fp8 else "bf16",
                           interleaved=interleaved, max_sets=max_sets)
        ang = np.arange(max_pages * 64)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
        self.table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.cs = torch.from_numpy(self.table).to(cuda)
        self.w = [self.bf((H, 128, 512), 512 ** -0.5) for _ in range(2)]
        self.kvw = self.bf((512,), 0.1, 1.0)
        self.rows = [np.zeros((0, 576)) for _ in range(B)]      # rows as values
        self.bits = [np.zeros((0, 656 if fp8 else 1152), dtype=np.uint8) for _ in range(B)]   # and as bytes

    def bf(self, shape, scale, mean=0.0):
        b = W.f32_to_bf16_bits((mean + scale * self.rng.standard_normal(shape)).astype(np.float32))
        return self.torch.from_numpy(b.view(np.int16)).to(self.s.device).view(self.torch.bfloat16)

    def i32(self, v):
        return self.torch.tensor(v, dtype=self.torch.int32, device=self.s.device)

    def draw_inputs(self, t, counts):
        s = self.s
        self.t, self.n = t, np.clip(counts, 0, None) * (np.array(counts) <= t)
        self.q, self.kv, self.counts = self.bf((s.B, t, s.H, 192), 2.0), self.bf((s.B, t, 576), 1.0), self.i32(counts)
        for b, n in enumerate(self.n):               # tokens that are not there: never read
            self.q[b, n:] = float("nan")
            self.kv[b, n:] = float("nan")

    def attend(self, stream=None):
        self.o = self.s.attend(self.q, self.kv, self.counts, self.cs, *self.w, kv_weight=self.kvw, stream=stream)

    def step(self, t, counts):
        self.draw_inputs(t, counts)
        self.attend()
        self.check()

    def fork(self, src, dst):
        self.s.fork(self.i32(src), self.i32(dst))
        for a, b in zip(src, dst):
            self.rows[b], self.bits[b] = self.rows[a].copy(), self.bits[a].copy()

    def cached(self, b, n):
        s = self.s
        blk = s.block_table[b].cpu().numpy()
        at = np.array([blk[j // 64] * 64 + j % 64 for j in range(n)], dtype=np.int64)
        assert (at >= 0).all()
        flat = s.pool.view(self.torch.uint8).view(s.num_blocks * 64, -1)
        return flat[self.torch.from_numpy(at).to(flat.device)].cpu().numpy() if n else np.zeros((0, flat.shape[1]), np.uint8)

    def values(self, raw):
        """The values that cached bytes stand for in the attention."""
        torch = self.torch
        if not len(raw):
            return np.zeros((0, 576))
        t = torch.from_numpy(raw)
        if self.s.cache_format == "bf16":
            return t.view(torch.bfloat16).double().numpy()
        lat = t[:, :512].contiguous().view(torch.float8_e4m3fn).float().view(-1, 4, 128)
        lat = (lat * t[:, 512:528].contiguous().view(torch.float32)[..., None]).view(-1, 512)
        return np.concatenate([lat.double().numpy(), t[:, 528:].contiguous().view(torch.bfloat16).double().numpy()], 1)

    def check(self, reported=False):
        """The step just run: attention, cache, pages."""
        s = self.s
        self.torch.cuda.synchronize()
        if reported:
            with pytest.raises(Exception):
                s.check()
        else:
            s.check()
        N = s.B * self.t
        o, lse = _np(self.o), s.lse.view(-1)[:N * s.H].view(s.B, self.t, s.H).cpu().numpy().astype(np.float64)
        q, kv = _np(self.q), _np(self.kv)
        lens, bt, live = s.seq_lens.cpu().numpy(), s.block_table.cpu().numpy(), s.live.cpu().numpy()
        assert np.array_equal(live, self.n)
        self.sets()
        for b in range(s.B):
            base, n = len(self.rows[b]), int(self.n[b])
            assert lens[b] == base + n and (bt[b] >= 0).sum() == (lens[b] + 63) // 64
            raw = self.cached(b, lens[b])
            assert np.array_equal(raw[:base], self.bits[b])
            val = self.values(raw[base:])
            qn, qp, want = O.rope_append_ref(q[b, :n], kv[b, :n], None, _np(self.kvw), 1e-6, self.table.astype(np.float64),
                                             base + np.arange(n), s.interleaved)
            fp8 = s.cache_format == "fp8"
            if n:
                step = 2.0 ** -4 + 2.0 ** -7 if fp8 else 2.0 ** -8
                scale = np.maximum(np.abs(want), np.abs(want).max() * 2.0 ** -8) if fp8 else np.abs(want)
                mag = np.abs(kv[b, :n]).max() * 2.0 ** -18
                assert np.all(np.abs(val - want)[:, :512] <= step * scale[:, :512] + mag)
                assert np.all(np.abs(val - want)[:, 512:] <= 2.0 ** -8 * np.abs(want[:, 512:]) + mag)
                # attention in the decompressed form, keys and values from each cached row, per head
                hist = np.concatenate([self.rows[b], val])
                k, v = (np.matmul(hist[:, :512], _np(w).swapaxes(1, 2)) for w in self.w)      # [H, rows, 128]
                see = np.arange(base + n)[None] <= base + np.arange(n)[:, None]
                x = (np.matmul(qn.swapaxes(0, 1), k.swapaxes(1, 2)).swapaxes(0, 1) + np.matmul(qp, hist[:, 512:].T)) * M.SCALE
                x = np.where(see[:, None], x, -np.inf)
                m = x.max(-1, keepdims=True)
                e = np.exp(x - m)
                parity(o[b, :n], np.matmul((e / e.sum(-1, keepdims=True)).swapaxes(0, 1), v).swapaxes(0, 1), f"o {b}", mean_rel=8e-3)
                parity(lse[b, :n], (m + np.log(e.sum(-1, keepdims=True)))[..., 0], f"lse {b}")
            assert (o[b, n:] == 0).all() and np.isneginf(lse[b, n:]).all()
            self.rows[b], self.bits[b] = np.concatenate([self.rows[b], val]), raw
        count = np.bincount(bt[bt >= 0], minlength=s.num_blocks)
        assert np.array_equal(count, s.refs.cpu().numpy())

    def sample(self, dtype=None, **settings):
        """A token for each sequence, as the rule gives it."""
        torch, s = self.torch, self.s
        x = torch.from_numpy(self.rng.standard_normal((s.B, self.V)) * 3).to(dtype or torch.bfloat16).to(s.device)
        u = self.rng.random(s.B).astype(np.float32)
        dev = {k: torch.from_numpy(np.full(s.B, v, dtype=np.int32 if k == "top_k" else np.float32)).to(s.device)
               for k, v in settings.items()}
        got = s.sample(x, self.V, u=torch.from_numpy(u).to(s.device), **dev).tolist()
        f = lambda k, off: float(np.float32(settings.get(k, off)))  # noqa: E731
        for b in range(s.B):
            want = S.sample_ref(_np(x[b]), f("temperature", 1.0), settings.get("top_k", 0), f("top_p", 1.0), f("min_p", 0.0), float(u[b]))
            assert got[b] == want[0]
        s.check()

    def sets(self):
        """Groups of the last plan that stand for shared pages: as many as the rule gives."""
        from mla_latent_cache_gb300 import binding as L
        s = self.s
        h, R = s.workspace[:256].view(self.torch.int32).cpu().numpy(), self.t * s.H
        n = int(h[L.HDR["NUM_GROUPS"]]) - s.B * ((R + 127) // 128)
        ptr = s.set_ptr.cpu().numpy()
        pages = S.shared_pages_ref(s.seq_lens.cpu().numpy(), s.live.cpu().numpy(), ptr, s.prefix_lens.cpu().numpy(), self.t, s.H,
                                   True, int(h[L.HDR["NUM_SLOTS"]]))
        assert n == sum((m * R + 127) // 128 for m, k in zip(np.diff(ptr), pages) if k)
        return n


@pytest.mark.parametrize("H,fp8,interleaved", [(16, False, True), (16, True, True), (64, False, False), (128, False, True)])
def test_samples_of_one_prompt(mla, cuda, H, fp8, interleaved):
    """A prompt of 450 rows in chunks, seven forks of it, and tokens drawn for each: too few pages for sharing to pay."""
    import torch
    h = Harness(torch, cuda, 8, H, 200, fp8, interleaved)
    for n in (200, 187, 63):
        h.step(200, [n] + [0] * 7)
    h.fork([0] * 7, list(range(1, 8)))
    h.s.set_sharing([0, 8], [450])
    for t in (1, 1, 3, 1):
        h.step(t, [t] * 8)
        assert h.sets() == 0
        h.sample(temperature=0.8, top_k=50, top_p=0.9)
    # (the sharing is only told, never needed)
    h.s.set_sharing([0], [])
    h.step(1, [1] * 8)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_samples_of_one_prompt(mla, cuda, fp8):
    """72 samples of a prompt of 700 rows: its ten full pages are attended once for all of them."""
    import torch
    h = Harness(torch, cuda, 72, 16, 350, fp8, seed=21, max_pages=12, num_blocks=300)
    for _ in range(2):
        h.step(350, [350] + [0] * 71)
    h.fork([0] * 71, list(range(1, 72)))
    h.s.set_sharing([0, 72], [700])
    for t, counts in ((1, [1] * 72), (1, [1, 0, 1] * 24), (2, [2, 1, 0, 1, 2, 2] * 12), (1, [1] * 72)):
        h.step(t, counts)
        assert h.sets() > 0
        h.sample(temperature=0.8, top_k=50, top_p=0.9)


def test_two_prompts_release_and_refill(mla, cuda):
    """Two system prompts, each with requests behind it, of which some end and others take their place."""
    import torch
    h = Harness(torch, cuda, 7, 16, 320, seed=5)
    s = h.s
    h.step(320, [320, 0, 0, 257, 0, 0, 0])
    h.fork([0, 0, 3, 3, 3], [1, 2, 4, 5, 6])
    s.set_sharing(h.i32([0, 3, 7]), h.i32([320, 256]))
    h.step(40, [40, 3, 17, 0, 1, 40, 22])
    for i in range(3):
        h.step(1, [1, 1, 1, 1, 1, 0, 1])
        h.sample(torch.float32, temperature=1.0, min_p=0.02)
    s.release(torch.tensor([False, True, False, False, False, True, False], device=cuda))
    for b in (1, 5):
        h.rows[b], h.bits[b] = h.rows[b][:0], h.bits[b][:0]
    s.set_sharing([0, 1, 3, 5, 7], [0, 0, 256, 0])
    h.step(1, [1, 0, 1, 1, 1, 0, 1])
    h.fork([0], [1])                          # a longer one in its place: part of its rows are its own page's
    h.fork([6], [5])
    s.set_sharing([0, 3, 7], [320, 256])
    for t in (1, 9, 1):
        h.step(t, [t] * 7)


def test_steps_captured_in_a_graph(mla, cuda):
    """One captured step with its draws, replayed with new inputs, counts, sets and random numbers."""
    import torch
    h = Harness(torch, cuda, 5, 16, 300, seed=9)
    s = h.s
    h.step(300, [300, 0, 0, 0, 200])
    h.fork([0, 0, 0], [1, 2, 3])
    h.draw_inputs(2, [2] * 5)
    q, kv, counts = h.q, h.kv, h.counts
    ptr, rows = h.i32([0, 4, 5]), h.i32([300, 200])
    x, u = torch.zeros((5, h.V), device=cuda), torch.zeros(5, device=cuda)
    k = h.i32([1, 0, 40, 5, 999])
    s.set_sharing(ptr, rows)
    h.attend()
    h.check()
    s.sample(x, h.V, u=u, top_k=k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.set_sharing(ptr, rows)
        h.attend()
        tokens = s.sample(x, h.V, u=u, top_k=k)
    o = h.o
    for i in range(6):
        h.draw_inputs(2, [2, 1, 2, i % 3, 2 - i % 2])
        q.copy_(h.q), kv.copy_(h.kv), counts.copy_(h.counts)
        if i == 3:
            ptr.copy_(h.i32([0, 2, 4]))
            rows.copy_(h.i32([300, 256]))
        x.copy_(torch.from_numpy(h.rng.standard_normal((5, h.V))))
        u.copy_(torch.from_numpy(h.rng.random(5)))
        g.replay()
        h.o = o
        h.check()
        for b in range(5):
            want = S.sample_ref(_np(x[b]), 1.0, int(k[b]), 1.0, 0.0, float(u[b]))
            assert int(tokens[b]) == want[0]


def test_counts_that_are_none_and_pages_that_are_none(mla, cuda):
    """Sequences past the free blocks, past their table, and with counts below 0 or past t sit out and go on later."""
    import torch
    h = Harness(torch, cuda, 4, 16, 128, seed=13, max_pages=4, num_blocks=7)
    h.step(128, [100, 128, 0, 60])                    # 2 + 2 + 1 of 7 blocks
    h.draw_inputs(128, [50, -1, 129, 0])
    h.n[:] = [50, 0, 0, 0]
    h.attend()
    h.check(reported=True)                            # counts that are none are reported
    h.draw_inputs(60, [60, 60, 60, 60])               # one block is free: sequence 0's (210 rows)
    h.n[:] = [60, 0, 0, 0]
    h.attend()
    h.check(reported=True)
    h.draw_inputs(60, [60, 0, 0, 4])                  # past its table; the last one has room in its block
    h.n[:] = [0, 0, 0, 4]
    h.attend()
    h.check(reported=True)
    h.s.release(torch.tensor([True, False, False, False], device=cuda))
    h.rows[0], h.bits[0] = h.rows[0][:0], h.bits[0][:0]
    h.step(1, [1, 1, 1, 1])


def test_another_stream_than_the_current_one(mla, cuda):
    import torch
    h = Harness(torch, cuda, 3, 16, 150, seed=17)
    side = torch.cuda.Stream()
    h.draw_inputs(150, [150, 1, 0])
    side.wait_stream(torch.cuda.current_stream())
    h.attend(stream=side)
    side.synchronize()
    h.check()
    h.s.fork(h.i32([0, 0]), h.i32([1, 2]), stream=side)
    for b in (1, 2):
        h.rows[b], h.bits[b] = h.rows[0].copy(), h.bits[0].copy()
    h.s.set_sharing([0, 3], [150], stream=side)
    h.draw_inputs(1, [1, 1, 1])
    side.wait_stream(torch.cuda.current_stream())
    h.attend(stream=side)
    side.synchronize()
    h.check()


def test_one_sequence_one_token(mla, cuda):
    import torch
    h = Harness(torch, cuda, 1, 8, 1, seed=19, max_pages=2, max_sets=0)
    for _ in range(66):
        h.step(1, [1])
    h.sample(temperature=0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_sets_that_lose_members_without_being_told(mla, cuda, fp8):
    """Members of sets are released and filled with other rows, or become forks of other sequences, and nobody tells the
    step: what it gives is each sequence's own, eagerly and replayed."""
    import torch
    h = Harness(torch, cuda, 66, 16, 350, fp8, seed=23, max_pages=14, num_blocks=330)
    s = h.s
    h.step(350, [350, 340] + [0] * 63 + [300])
    h.step(350, [350, 350] + [0] * 63 + [330])
    h.fork([0] * 40 + [1] * 23, list(range(2, 42)) + list(range(42, 65)))
    h.fork([0], [1])                                   # 0 to 41 are samples of one prompt, 42 to 64 of another
    s.set_sharing([0, 42, 65], [700, 640])
    h.step(1, [1] * 66)
    both = h.sets()
    assert both > 0
    # a member of the second set ends, and a longer request comes in its place
    which = torch.zeros(66, dtype=torch.bool, device=cuda)
    which[50] = True
    s.release(which)
    h.rows[50], h.bits[50] = h.rows[50][:0], h.bits[50][:0]
    h.step(350, [0] * 50 + [350] + [0] * 15)
    h.step(350, [0] * 50 + [350] + [0] * 15)
    h.step(1, [1] * 66)
    assert 0 < h.sets() < both
    # a member of the first becomes a fork of the other prompt's
    h.fork([65], [3])
    h.step(2, [2] * 66)
    assert h.sets() == 0
    # told anew, and a release that is replayed
    s.set_sharing([0, 3, 4, 42], [0, 0, 700])
    h.step(1, [1] * 66)
    assert h.sets() > 0
    which.zero_()
    s.release(which)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.release(which)
    which[20] = True
    g.replay()
    h.rows[20], h.bits[20] = h.rows[20][:0], h.bits[20][:0]
    h.step(130, [0] * 20 + [130] + [0] * 45)
    h.step(1, [1] * 66)
    assert h.sets() == 0


def test_an_empty_member_that_begins_anew_is_reported(mla, cuda):
    import torch
    h = Harness(torch, cuda, 40, 16, 350, seed=27, max_pages=14, num_blocks=200)
    s = h.s
    for _ in range(2):
        h.step(350, [350] + [0] * 39)
    h.fork([0] * 38, list(range(1, 39)))
    s.set_sharing([0, 40], [700])                        # (the last one is empty)
    h.step(1, [1] * 39 + [0])
    assert h.sets() > 0
    h.step(350, [0] * 39 + [350])                        # its first rows: nothing is shared beside them
    for t in (350, 1):
        h.draw_inputs(t, [1] * 39 + [t])
        h.attend()
    torch.cuda.synchronize()
    with pytest.raises(mla.MlaError, match=r"\(39\)"):
        s.check()
    # told anew, all is as it should be
    s.set_sharing([0, 39], [700])
    h.draw_inputs(1, [1] * 40)
    h.attend()
    torch.cuda.synchronize()
    s.check()
    assert h.sets() > 0


def test_draws_do_not_overwrite_one_another(mla, cuda):
    """Two settings on the same logits, a captured draw among them: each keeps its own tokens."""
    import torch
    h = Harness(torch, cuda, 9, 16, 1, seed=29, max_pages=1)
    s = h.s
    x = torch.from_numpy(h.rng.standard_normal((9, h.V))).float().to(cuda)
    low, high = torch.zeros(9, device=cuda), torch.full((9,), 1 - 2.0 ** -24, device=cuda)
    first, last = x.argmax(1).tolist(), x.argmin(1).tolist()
    a = s.sample(x, h.V, u=low)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = s.sample(x, h.V, u=high)
    b = s.sample(x, h.V, u=high)
    g.replay()
    d = s.sample(x, h.V, u=low)
    assert (a.tolist(), b.tolist(), c.tolist(), d.tolist()) == (first, last, last, first) and s.tokens is d
    low.fill_(1 - 2.0 ** -24)
    high.zero_()
    g.replay()
    assert (a.tolist(), b.tolist(), c.tolist(), d.tolist()) == (first, last, first, first)
