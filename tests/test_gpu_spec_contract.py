"""What the calls of a speculative step promise beyond their results at aligned, well-formed inputs."""
import numpy as np
import pytest

from oracle import mla_oracle as M
from oracle import spec_oracle as O
from tests._tol import parity
from tests.test_gpu_spec_step import Harness
from tests.test_gpu_tree import Tree
from tests.test_gpu_verify import _random

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_queries_need_16_byte_alignment_only(mla, cuda, fp8):
    """Queries, positions' queries, masks and lengths at 16 bytes past a 32-byte border, several segments
    to each CTA pair: the bits of the aligned call."""
    import torch
    t = Tree(mla, torch, cuda, 128, [300, 200, 70], 5, nodes=[5, 4, 5], fp8=fp8, sharp=not fp8, slots=2).run().check()
    o, lse = t.o.clone(), t.lse.clone()

    def moved(x):
        pad = 16 // x.element_size()
        y = torch.empty(x.numel() + 2 * pad, dtype=x.dtype, device=cuda)
        y = y[pad:pad + x.numel()] if y.data_ptr() % 32 == 0 else y[:x.numel()]
        assert y.data_ptr() % 32 == 16
        return y.view(x.shape).copy_(x)

    for name in ("q_lat", "q_pe", "mask", "lens", "node_lens", "bt"):
        setattr(t, name, moved(getattr(t, name)))
    t.o.fill_(float("nan"))
    t.run()
    assert torch.equal(t.o, o) and torch.equal(t.lse, lse)
    assert np.isfinite(t.o.float().cpu().numpy()).all()


def _committed(torch, cuda, lens, B, num_blocks=32, **kw):
    """A SpecStep whose sequences hold rows of random bytes, and those rows' bytes."""
    from mla_latent_cache_gb300 import binding as L
    from mla_latent_cache_gb300.runtime import SpecStep
    s = SpecStep(B, 16, 4, max_pages=4, num_blocks=num_blocks, device=cuda, **kw)
    s.pool.view(torch.uint8).random_(0, 100)
    L.check(L.mla_pages_resize(s.refs, num_blocks, s.block_table, 4, 4, s.seq_lens,
                               torch.tensor(lens, dtype=torch.int32, device=cuda), B, s.seq_lens))
    torch.cuda.synchronize()
    return s


def _held(s):
    """Length, table row and rows' bytes of each sequence."""
    lens, bt = s.seq_lens.tolist(), s.block_table.cpu().numpy()
    pool = s.pool.view(s.torch.uint8).cpu().numpy()
    return {b: (n, bt[b].tolist(), b"".join(pool[bt[b, j // 64], j % 64].tobytes() for j in range(n))) for b, n in enumerate(lens)}


def _counts(s):
    bt = s.block_table.cpu().numpy()
    assert np.array_equal(np.bincount(bt[bt >= 0], minlength=s.num_blocks), s.refs.cpu().numpy())


@pytest.mark.parametrize("src,dst", [([0], [-1]), ([0], [4]), ([0], [2 ** 31 - 1]), ([0], [-2 ** 31]), ([-1], [1]), ([4], [1]),
                                     ([0, 2], [1, 1]), ([1, 0], [1, 1])])
def test_refused_forks_change_nothing(mla, cuda, src, dst):
    import torch
    s = _committed(torch, cuda, [70, 130, 5, 64], 4)
    before = _held(s)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    s.fork(i32(src), i32(dst))
    with pytest.raises(mla.MlaError):
        s.check()
    assert _held(s) == before
    s.fork(i32([*src, 0]), i32([*dst, 3]))          # a good one beside them
    with pytest.raises(mla.MlaError):
        s.check()
    after = _held(s)
    assert all(after[b] == before[b] for b in (0, 1, 2)) and after[3][0] == 70 and after[3][2] == before[0][2]
    _counts(s)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_sequence_forked_from_itself(mla, cuda, fmt):
    import torch
    s = _committed(torch, cuda, [70, 130, 5, 0], 4, cache_format=fmt)
    before = _held(s)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    s.fork(i32([0, 1, 3]), i32([0, 1, 3]))          # nobody else holds their pages
    s.check()
    assert _held(s) == before
    # sequence 3 takes sequence 1's pages over, last one included, and then a last page of its own
    s.block_table[3] = s.block_table[1]
    s.refs[s.block_table[1, :3].long()] += 1
    s.seq_lens[3] = 130
    s.fork(i32([3]), i32([3]))
    s.check()
    after = _held(s)
    assert all(after[b] == before[b] for b in (0, 1, 2)) and after[3][2] == before[1][2]
    assert after[3][1][:2] == before[1][1][:2] and after[3][1][2] != before[1][1][2]
    _counts(s)


def test_forks_captured_and_replayed(mla, cuda):
    """A captured fork takes the numbers that its arrays hold when it is replayed, refused ones among them."""
    import torch
    s = _committed(torch, cuda, [70, 130, 5, 64], 4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    src, dst = i32([-1, -1]), i32([-1, -1])
    s.fork(src, dst)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.fork(src, dst)
    for a, b in (([0, 0], [1, 9]), ([1, 2], [3, 3]), ([2, 2], [0, 2]), ([0, 0], [1, 3])):
        before = _held(s)
        src.copy_(i32(a))
        dst.copy_(i32(b))
        g.replay()
        torch.cuda.synchronize()
        after = _held(s)
        for k in range(4):
            f = [x for x, y in zip(a, b) if y == k and b.count(k) == 1 and x not in b]
            assert (after[k][0], after[k][2]) == (before[f[0]][0], before[f[0]][2]) if f else after[k] == before[k]
        _counts(s)
    assert mla.mla_read_device_status(None)[0] == mla.MLA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_steps_on_a_stream_of_their_own(mla, cuda, fp8, handle):
    """Steps and forks given a stream while torch's current one is busy: nothing of them waits for it, and
    nothing that they keep is taken by what runs there."""
    import torch
    h = Harness(torch, cuda, 4, 16, 30, 52, fp8=fp8, seed=4)
    s, side = h.s, torch.cuda.Stream()
    st = side.cuda_stream if handle else side
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    src, dst = i32([0, 2, 1]), i32([3, 2, -1])
    for step in range(6):
        h.draw_inputs(tree=step % 2 == 1)
        par, n = h.par, h.n
        s.set_tree(np.tile(np.arange(-1, 29), (4, 1)), np.full(4, 1))   # not this step's
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)                # ~50 ms
        busy = [torch.full((4, 30), -1, dtype=torch.int32, device=cuda) for _ in range(40)]
        s.set_tree(par, n, stream=st)
        s.attend(h.q, h.kv, h.cs, *h.w, kv_weight=h.kvw, stream=st)
        s.accept(h.p, h.d, h.tokens, h.ua, h.us, h.V, stream=st)
        s.commit(stream=st)
        side.synchronize()
        assert step < 2 or not torch.cuda.current_stream().query()    # (first uses load kernels, which may wait)
        h.check()
        del busy
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        s.fork(src, dst, stream=st)
        busy = [torch.full((4,), 1 << 20, dtype=torch.int32, device=cuda) for _ in range(40)]
        side.synchronize()
        assert step < 2 or not torch.cuda.current_stream().query()
        with pytest.raises(mla.MlaError):             # (the fork to -1)
            s.check(stream=st)
        h.rows[3], h.bits[3] = h.rows[0].copy(), h.bits[0].copy()
        del busy
    _counts(s)
    assert max(len(r) for r in h.rows) > 6


@pytest.mark.parametrize("B,H,T", [(3, 32, 9), (3, 16, 7), (2, 128, 20)])
def test_attention_of_fp8_steps(mla, cuda, B, H, T):
    """A step over FP8 rows attends to the rows that the cache holds, pages converted ahead (T H > 128) or by group."""
    import torch
    h = Harness(torch, cuda, B, H, T, 64, fp8=True, seed=T)
    s = h.s
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    for step in range(5):
        h.draw_inputs(tree=step % 2 == 0)
        base = s.seq_lens.tolist()
        s.attend(h.q, h.kv, h.cs, *h.w, kv_weight=h.kvw)
        torch.cuda.synchronize()
        see = O.ancestors(h.par)
        o, lse = f(s.o), s.lse.cpu().numpy().astype(np.float64)
        for b in range(B):
            n = int(h.n[b])
            qn, qp, _ = O.rope_append_ref(f(h.q[b]), f(h.kv[b]), None, f(h.kvw), 1e-6, h.table.astype(np.float64),
                                          base[b] + see[b].sum(-1) - 1, s.interleaved)
            hist = h.values(h.cached(b, range(base[b] + n)))
            assert np.array_equal(hist[:base[b]], h.rows[b])
            k = np.einsum("jc,hnc->hjn", hist[:, :512], f(h.w[0]))
            v = np.einsum("jc,hvc->hjv", hist[:, :512], f(h.w[1]))
            x = (np.einsum("thn,hjn->thj", qn[:n], k) + np.einsum("thr,jr->thj", qp[:n], hist[:, 512:])) * M.SCALE
            x = np.where(O.tree_visible(base[b] + n, n, see[b])[:n, None], x, -np.inf)
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            total = e.sum(-1, keepdims=True)
            # (the bf16 step's tolerances: from the cached rows on, the arithmetic is the same)
            parity(o[b, :n], np.einsum("thj,hjv->thv", e / total, v), f"o {b}", mean_rel=8e-3)
            parity(lse[b, :n], (m + np.log(total))[..., 0], f"lse {b}")
        s.accept(h.p, h.d, h.tokens, h.ua, h.us, h.V)
        s.commit()
        h.check()


def test_fp8_steps_without_room_for_converted_pages(mla, cuda):
    """The same bits, step after step."""
    import torch
    from mla_latent_cache_gb300.runtime import SpecStep
    a, b = (Harness(torch, cuda, 2, 32, 9, 64, fp8=True, seed=5) for _ in range(2))
    b.s = SpecStep(2, 32, 9, max_pages=8, num_blocks=16, device=cuda, cache_format="fp8", convert_ahead=False)
    assert b.s.ws_bytes < a.s.ws_bytes
    for step in range(6):
        for h in (a, b):
            h.draw_inputs(tree=step % 2 == 0)
            h.device_step()
            h.check()
        assert torch.equal(a.s.o, b.s.o) and torch.equal(a.s.lse, b.s.lse) and torch.equal(a.s.pool, b.s.pool)


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("power", [-60, 30])
def test_verify_rows_far_from_a_sum_of_one(mla, cuda, power, draft):
    """Rows whose values sum to 2^-60 and to 2^30 decide by the rule as it stands (a first test's mass is 1)."""
    import torch
    r = _random(mla, torch, 24, 9, 3001, torch.float32, draft, True, 2, sharp=1.0, noise=2.0)
    r.p *= 2.0 ** power
    if draft:
        r.q *= 2.0 ** power
    assert r.call() == mla.MLA_OK
    r.check()


def test_verify_replays_give_what_the_eager_call_gave(mla, cuda):
    import torch
    r = _random(mla, torch, 8, 6, 5000, torch.float32, True, True, 1)
    r.check()
    first = [x.copy() for x in r.results()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert r.call() == mla.MLA_OK
    for x in r.out:
        x.fill_(-7)
    g.replay()
    assert all(np.array_equal(x, y) for x, y in zip(r.results(), first))
    r.args[3].copy_(torch.rand(8, 6, device="cuda"))
    r.args[4].copy_(torch.rand(8, device="cuda"))
    g.replay()
    r.check()
