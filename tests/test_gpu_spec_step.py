"""Speculative steps as they are used: pages, append, tree attention, verification, compaction,
forks, step after step on one cache, against a float64 history of every sequence's rows."""
import numpy as np
import pytest

from mla_latent_cache_gb300 import workloads as W
from oracle import mla_oracle as M
from oracle import spec_oracle as O
from tests._tol import parity

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


class Harness:
    def __init__(self, torch, cuda, B, H, T, V, fp8=False, interleaved=True, seed=0, num_blocks=None):
        from mla_latent_cache_gb300.runtime import SpecStep
        self.torch, self.V = torch, V
        self.rng = np.random.default_rng(seed)
        self.s = SpecStep(B, H, T, max_pages=8, num_blocks=num_blocks or 8 * B, device=cuda,
                          cache_format="fp8" if fp8 else "bf16", interleaved=interleaved)
        ang = np.arange(600)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
        self.table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.cs = torch.from_numpy(self.table).to(cuda)
        self.w = [self.bf((H, 128, 512), 512 ** -0.5) for _ in range(2)]
        self.kvw = self.bf((512,), 0.1, 1.0)
        self.rows = [np.zeros((0, 576)) for _ in range(B)]      # committed rows, as values
        self.bits = [np.zeros((0, 656 if fp8 else 1152), dtype=np.uint8) for _ in range(B)]   # and as bytes
        self.q = torch.empty((B, T, H, 192), dtype=torch.bfloat16, device=cuda)
        self.kv = torch.empty((B, T, 576), dtype=torch.bfloat16, device=cuda)
        self.p = torch.empty((B, T, V), device=cuda)
        self.d = torch.empty((B, T, V), device=cuda)
        self.tokens = torch.empty((B, T), dtype=torch.int32, device=cuda)
        self.ua, self.us = torch.empty((B, T), device=cuda), torch.empty((B,), device=cuda)

    def bf(self, shape, scale, mean=0.0):
        b = W.f32_to_bf16_bits((mean + scale * self.rng.standard_normal(shape)).astype(np.float32))
        return self.torch.from_numpy(b.view(np.int16)).to(self.s.device).view(self.torch.bfloat16)

    def draw_inputs(self, tree):
        s, rng, torch = self.s, self.rng, self.torch
        par = np.tile(np.arange(-1, s.T - 1), (s.B, 1))
        if tree:
            for t in range(1, s.T):
                par[:, t] = rng.integers(0, t, s.B)
        self.par, self.n = par, rng.integers(1, s.T + 1, s.B)
        s.set_tree(par, self.n)
        self.q.copy_(self.bf(self.q.shape, 2.0))
        self.kv.copy_(self.bf(self.kv.shape, 1.0))
        x = rng.standard_normal((s.B, s.T, self.V)) * 2
        p, d = np.exp(x), np.exp(x + rng.standard_normal(x.shape))
        self.p.copy_(torch.from_numpy(p / p.sum(-1, keepdims=True)))
        self.d.copy_(torch.from_numpy(d / d.sum(-1, keepdims=True)))
        self.tokens.copy_(torch.from_numpy(rng.integers(0, self.V, (s.B, s.T)).astype(np.int32)))
        self.ua.copy_(torch.from_numpy(rng.random((s.B, s.T)) * 0.5))
        self.us.copy_(torch.from_numpy(rng.random(s.B)))

    def device_step(self):
        s = self.s
        s.attend(self.q, self.kv, self.cs, *self.w, kv_weight=self.kvw)
        s.accept(self.p, self.d, self.tokens, self.ua, self.us, self.V)
        s.commit()

    def cached(self, b, rows):
        """Bytes of the listed logical rows of sequence b."""
        s = self.s
        blk = s.block_table[b].cpu().numpy()
        flat = s.pool.view(self.torch.uint8).view(s.num_blocks * 64, -1)
        at = np.array([blk[j // 64] * 64 + j % 64 for j in rows], dtype=np.int64)
        assert (at >= 0).all()
        return flat[self.torch.from_numpy(at).to(flat.device)].cpu().numpy() if len(at) else np.zeros((0, flat.shape[1]), np.uint8)

    def values(self, raw):
        """The bf16 values that cached bytes stand for in the attention."""
        torch = self.torch
        if not len(raw):
            return np.zeros((0, 576))
        t = torch.from_numpy(raw)
        if self.s.cache_format == "bf16":
            return t.view(torch.bfloat16).double().numpy()
        lat = t[:, :512].contiguous().view(torch.float8_e4m3fn).float().view(-1, 4, 128)
        lat = (lat * t[:, 512:528].contiguous().view(torch.float32)[..., None]).view(-1, 512).bfloat16()
        return np.concatenate([lat.double().numpy(), t[:, 528:].contiguous().view(torch.bfloat16).double().numpy()], 1)

    def check(self):
        """The step just run: attention, decisions, cache, pages."""
        s, torch = self.s, self.torch
        torch.cuda.synchronize()
        s.check()
        f = lambda t: _np(t)  # noqa: E731
        depth = O.ancestors(self.par).sum(-1) - 1
        see = O.ancestors(self.par)
        o, lse = _np(s.o), s.lse.cpu().numpy().astype(np.float64)
        acc_len, acc_idx, out = s.accept_len.cpu().numpy(), s.accept_idx.cpu().numpy(), s.out_tokens.cpu().numpy()
        lens, bt = s.seq_lens.cpu().numpy(), s.block_table.cpu().numpy()
        p, d, tok = self.p.double().cpu().numpy(), self.d.double().cpu().numpy(), self.tokens.cpu().numpy()
        for b in range(s.B):
            base, n = len(self.rows[b]), int(self.n[b])
            qn, qp, rows = O.rope_append_ref(f(self.q[b]), f(self.kv[b]), None, f(self.kvw), 1e-6, self.table.astype(np.float64),
                                             base + depth[b], s.interleaved)
            path, nxt = O.verify_ref(p[b], d[b], tok[b], self.par[b], n, self.ua[b].double().cpu().numpy(), float(self.us[b]))
            assert acc_len[b] == len(path) and acc_idx[b, :len(path)].tolist() == path
            assert out[b, :len(path)].tolist() == [int(tok[b, t]) for t in path[1:]] + [nxt]
            # attention in the decompressed form: keys and values from each row, per head.  The nodes'
            # rows are the definition's; FP8 rows as the cache holds them (accepted ones) are within its steps
            hist = np.concatenate([self.rows[b], rows[:n]])
            k = np.einsum("jc,hnc->hjn", hist[:, :512], f(self.w[0]))
            v = np.einsum("jc,hvc->hjv", hist[:, :512], f(self.w[1]))
            vis = O.tree_visible(base + n, n, see[b])[:n]
            x = (np.einsum("thn,hjn->thj", qn[:n], k) + np.einsum("thr,jr->thj", qp[:n], hist[:, 512:])) * M.SCALE
            x = np.where(vis[:, None], x, -np.inf)
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            if s.cache_format == "bf16":
                parity(o[b, :n], np.einsum("thj,hjv->thv", e / e.sum(-1, keepdims=True), v), f"o {b}", mean_rel=8e-3)
                parity(lse[b, :n], (m + np.log(e.sum(-1, keepdims=True)))[..., 0], f"lse {b}")
            assert (o[b, n:] == 0).all() and np.isneginf(lse[b, n:]).all()
            # the cache: history unchanged, accepted rows in place, and the right number of pages
            assert lens[b] == base + len(path)
            assert (bt[b] >= 0).sum() == (lens[b] + 63) // 64
            raw = self.cached(b, range(lens[b]))
            assert np.array_equal(raw[:base], self.bits[b])
            val = self.values(raw[base:])
            want = rows[path]
            step = 2.0 ** -8 if s.cache_format == "bf16" else 2.0 ** -4 + 2.0 ** -7
            scale = np.abs(want) if s.cache_format == "bf16" else np.maximum(np.abs(want), np.abs(want).max() * 2.0 ** -8)
            mag = np.abs(f(self.kv[b]))[path].max() * 2.0 ** -18
            assert np.all(np.abs(val - want)[:, :512] <= step * scale[:, :512] + mag)
            assert np.all(np.abs(val - want)[:, 512:] <= 2.0 ** -8 * np.abs(want[:, 512:]) + mag)
            self.rows[b], self.bits[b] = np.concatenate([self.rows[b], val]), raw
        held = bt[bt >= 0]
        count = np.bincount(held, minlength=s.num_blocks)
        assert np.array_equal(count, s.refs.cpu().numpy())


@pytest.mark.parametrize("B,H,T,fp8,interleaved", [(3, 16, 7, False, True), (2, 128, 5, False, False), (4, 8, 40, False, True),
                                                   (3, 32, 9, True, True)])
def test_speculative_steps_from_an_empty_cache(mla, cuda, B, H, T, fp8, interleaved):
    import torch
    h = Harness(torch, cuda, B, H, T, 200, fp8, interleaved, seed=B)
    for step in range(9):
        h.draw_inputs(tree=step % 3 != 0)
        h.device_step()
        h.check()
    assert max(len(r) for r in h.rows) > 9


def test_forks_between_steps(mla, cuda):
    """Sequences of more than a page forked, shortened into a shared page, and decoded on."""
    import torch
    h = Harness(torch, cuda, 4, 16, 60, 52, seed=3)
    for _ in range(3):
        h.draw_inputs(tree=False)
        h.ua.zero_()                 # nearly every draft is accepted
        h.device_step()
        h.check()
    s = h.s
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    s.fork(i32([0, 0]), i32([2, 3]))
    for d in (2, 3):
        h.rows[d], h.bits[d] = h.rows[0].copy(), h.bits[0].copy()
    assert int(s.refs.max()) == 3
    for step in range(3):
        h.draw_inputs(tree=True)
        h.device_step()
        # (check: shared pages count every holder)
        h.check()
    # sequence 3 goes back into a page that it shares, makes it its own, and goes on
    keep = s.seq_lens.clone()
    keep[3] = 37
    mla.check(mla.mla_pages_resize(s.refs, s.num_blocks, s.block_table, 8, 8, s.seq_lens, keep, 4, s.seq_lens))
    copies = torch.empty((3, 1), dtype=torch.int32, device=cuda)
    mla.check(mla.mla_pages_fork(s.refs, s.num_blocks, s.block_table, 8, 8, s.seq_lens, 4, i32([3]), i32([3]), 1, copies))
    mla.check(mla.mla_cache_copy(s.cache, copies, 1))
    assert copies[2, 0] == 37
    h.rows[3], h.bits[3] = h.rows[3][:37], h.bits[3][:37]
    for step in range(2):
        h.draw_inputs(tree=True)
        h.device_step()
        h.check()


def test_step_captured_in_a_graph(mla, cuda):
    """One captured step, replayed with new inputs, trees and node counts."""
    import torch
    h = Harness(torch, cuda, 3, 16, 6, 100, seed=7)
    h.draw_inputs(tree=True)
    h.device_step()
    h.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.device_step()
    for _ in range(5):
        h.draw_inputs(tree=True)
        g.replay()
        h.check()


def test_sequences_without_pages_sit_the_step_out(mla, cuda):
    """Two of three sequences get the pages of a step: the third answers nothing, keeps its rows
    and its pages, and goes on when blocks are free again."""
    import torch
    h = Harness(torch, cuda, 3, 16, 40, 64, seed=11, num_blocks=5)
    h.draw_inputs(tree=False)
    h.n[:] = 40
    s = h.s
    s.set_tree(h.par, h.n)
    h.ua.zero_()
    h.device_step()
    h.check()
    before = [len(r) for r in h.rows]
    # every sequence holds one block of five; two of them get a second one
    h.draw_inputs(tree=True)
    h.n[:] = [40, 40, 40]
    assert all(0 < n and n + 40 > 64 for n in before)
    s.set_tree(h.par, h.n)
    h.device_step()
    torch.cuda.synchronize()
    with pytest.raises(mla.MlaError):
        s.check()
    assert s.accept_len[2] == 0 and (s.out_tokens[2] == -1).all()
    assert (s.o[2] == 0).all() and torch.isneginf(s.lse[2]).all()
    assert s.seq_lens[2] == before[2] and (s.block_table[2] >= 0).sum() == 1
    assert np.array_equal(h.cached(2, range(before[2])), h.bits[2])
    lens = s.seq_lens.cpu().numpy()
    for b in (0, 1):
        assert lens[b] == before[b] + int(s.accept_len[b]) and s.accept_len[b] > 0
        assert np.array_equal(h.cached(b, range(before[b])), h.bits[b])
    # sequence 0 is given back; the other two go on
    keep = s.seq_lens.clone()
    keep[0] = 0
    mla.check(mla.mla_pages_resize(s.refs, s.num_blocks, s.block_table, 8, 8, s.seq_lens, keep, 3, s.seq_lens))
    for b in range(3):
        h.bits[b] = h.cached(b, range(int(s.seq_lens[b])))
        h.rows[b] = h.values(h.bits[b])
    h.draw_inputs(tree=True)
    h.n[:] = [3, 9, 40]
    s.set_tree(h.par, h.n)
    h.device_step()
    h.check()


def test_one_token_steps_from_strided_views(mla, cuda):
    """T = 1 (plain decoding): inputs that are views of wider arrays, sequences that take no part."""
    import torch
    h = Harness(torch, cuda, 4, 16, 1, 64, seed=13)
    s = h.s
    for step in range(3):
        h.draw_inputs(tree=False)
        h.n[step] = 0
        s.set_tree(np.full((4, 1), -1), h.n)
        wide = torch.full((4, 5, 16, 192), float("nan"), dtype=torch.bfloat16, device=cuda)
        wide[:, :1] = h.q
        wide_kv = torch.full((4, 3, 576), float("nan"), dtype=torch.bfloat16, device=cuda)
        wide_kv[:, :1] = h.kv
        wide_p = torch.full((4, 2, 80), float("nan"), device=cuda)
        wide_p[:, :1, :64] = h.p
        s.attend(wide[:, :1], wide_kv[:, :1], h.cs, *h.w, kv_weight=h.kvw)
        s.accept(wide_p[:, :1], None, h.tokens, h.ua, h.us, 64)
        s.commit()
        assert s.accept_len.cpu().tolist() == h.n.tolist()
        torch.cuda.synchronize()
        s.check()
        qn, qp, rows = O.rope_append_ref(_np(h.q)[:, 0], _np(h.kv)[:, 0], None, _np(h.kvw), 1e-6,
                                         h.table.astype(np.float64), [len(r) for r in h.rows], s.interleaved)
        p = h.p.double().cpu().numpy()
        for b in range(4):
            raw = h.cached(b, range(int(s.seq_lens[b])))
            assert np.array_equal(raw[:len(h.bits[b])], h.bits[b]) and len(raw) == len(h.bits[b]) + h.n[b]
            if h.n[b]:
                _, nxt = O.verify_ref(p[b], None, np.zeros(1, int), np.array([-1]), 1, np.zeros(1), float(h.us[b]))
                assert int(s.out_tokens[b, 0]) == nxt
                mag = np.abs(_np(h.kv)[b]).max() * 2.0 ** -18
                assert np.all(np.abs(h.values(raw[-1:]) - rows[b]) <= 2.0 ** -8 * np.abs(rows[b]) + mag)
            h.bits[b], h.rows[b] = raw, h.values(raw)
