"""What a serving step promises on the host (no GPU needed): the library's calls are stood in for by plain
versions on CPU tensors."""
import numpy as np
import pytest

from oracle import serve_oracle as S
from oracle import spec_oracle as O

torch = pytest.importorskip("torch")


class Library:
    def __init__(self, monkeypatch):
        from mla_latent_cache_gb300 import runtime
        self.calls, self.answers, self.args = [], {}, {}
        for name in ("mla_pages_resize", "mla_pages_fork", "mla_cache_copy", "mla_rope_append", "mla_absorb_q", "mla_batch_map",
                     "mla_plan_shared", "mla_decode_shared", "mla_unabsorb_o", "mla_sample"):
            monkeypatch.setattr(runtime.L, name, self._call(name, getattr(self, name, None)))

    def _call(self, name, plain):
        def call(*args):
            self.calls.append(name)
            self.args[name] = args
            answer = self.answers.get(name, 0)
            if isinstance(answer, BaseException):
                raise answer
            if answer == 0 and plain is not None:
                plain(*args)
            return answer
        return call

    def mla_pages_resize(self, refs, nb, bt, stride, max_pages, cur, new, B, got, stream):
        pages = O.Pages(bt.numpy(), refs.numpy(), cur.numpy())
        pages.resize(new.numpy())
        for t, v in ((refs, pages.refs), (bt, pages.bt), (got, pages.lens)):
            t.copy_(torch.from_numpy(v))

    def mla_batch_map(self, B, T, N, cached, counts, held, bt, stride, max_pages, nb, depth, live, lens, cu, seq, pos, slots, stream):
        m = S.batch_map_ref(T, N, cached.numpy(), counts.numpy(), held.numpy(), bt.numpy(), max_pages, nb)
        for t, k in ((live, "live"), (lens, "seq_lens")):
            t.copy_(torch.from_numpy(m[k]))
        pos[:N].copy_(torch.from_numpy(m["positions"]))
        slots[:N].copy_(torch.from_numpy(m["slots"]))


@pytest.fixture
def lib(mla, monkeypatch):
    return Library(monkeypatch)


@pytest.fixture
def step(lib):
    from mla_latent_cache_gb300.runtime import ServeStep
    return lambda B=3, T=4, H=16, max_pages=4, num_blocks=16, **kw: ServeStep(B, H, T, max_pages, num_blocks, device="cpu", **kw)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _inputs(s, t, **kw):
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    return {**dict(q=z(s.B, t, s.H, 192), kv=z(s.B, t, 576), counts=_i32([t] * s.B), cos_sin=z(64, 64, dtype=torch.float32),
                   w_uk=z(s.H, 128, 512), w_uv=z(s.H, 128, 512), kv_weight=z(512)), **kw}


def _pages(s):
    return {b: (int(s.seq_lens[b]), s.block_table[b].tolist()) for b in range(s.B)}, s.refs.tolist()


def test_tokens_become_rows(step, lib):
    s = step()
    for t, counts, lens in ((4, [4, 2, 0], [4, 2, 0]), (1, [1, 1, 1], [5, 3, 1]), (3, [3, 0, 2], [8, 3, 3])):
        o = s.attend(**_inputs(s, t, counts=_i32(counts)))
        assert o.shape == (3, t, 16, 128) and s.seq_lens.tolist() == lens and s.live.tolist() == counts
        assert lib.args["mla_plan_shared"][1].T == t and lib.args["mla_rope_append"][1] == 3 * t
    assert lib.calls[-8:] == ["mla_pages_resize", "mla_batch_map", "mla_rope_append", "mla_absorb_q", "mla_plan_shared",
                              "mla_decode_shared", "mla_unabsorb_o", "mla_pages_resize"]
    O.Pages(s.block_table.numpy(), s.refs.numpy(), s.seq_lens.numpy()).check()


def test_what_does_not_fit_sits_out_and_holds_nothing(step, lib):
    s = step(B=3, T=64, max_pages=2, num_blocks=3)
    s.attend(**_inputs(s, 64, counts=_i32([60, 60, 0])))
    s.attend(**_inputs(s, 64, counts=_i32([10, 64, 5])))       # one block is free: the first sequence's
    assert s.live.tolist() == [10, 0, 0] and s.seq_lens.tolist() == [70, 60, 0]
    s.attend(**_inputs(s, 64, counts=_i32([59, -3, 65])))      # past its table; counts that are none
    assert s.live.tolist() == [0, 0, 0] and s.seq_lens.tolist() == [70, 60, 0]
    O.Pages(s.block_table.numpy(), s.refs.numpy(), s.seq_lens.numpy()).check()
    s.release(torch.tensor([True, False, True]))
    assert s.seq_lens.tolist() == [0, 60, 0] and s.refs.tolist().count(0) == 2


@pytest.mark.parametrize("name", ["mla_batch_map", "mla_rope_append", "mla_absorb_q", "mla_plan_shared", "mla_decode_shared",
                                  "mla_unabsorb_o"])
@pytest.mark.parametrize("answer", [-6, KeyboardInterrupt()])
def test_a_call_that_fails_leaves_the_step_where_it_was(step, lib, name, answer):
    s = step()
    s.attend(**_inputs(s, 4))
    before = _pages(s)
    lib.answers[name] = answer
    with pytest.raises(BaseException):
        s.attend(**_inputs(s, 4, counts=_i32([4, 4, 4])))
    assert _pages(s) == before
    del lib.answers[name]
    s.attend(**_inputs(s, 4))
    assert s.seq_lens.tolist() == [8, 8, 8]


def test_arguments_that_do_not_fit(step, lib):
    s = step(max_sets=2)
    z = torch.zeros
    for bad in (dict(q=z(3, 5, 16, 192, dtype=torch.bfloat16)), dict(q=z(3, 0, 16, 192, dtype=torch.bfloat16)),
                dict(q=z(3, 4, 16, 192)), dict(q=z(2, 4, 16, 192, dtype=torch.bfloat16)), dict(kv=z(3, 3, 576, dtype=torch.bfloat16)),
                dict(q=z(3, 4, 16, 192, dtype=torch.bfloat16, device="meta")), dict(counts=z(3)), dict(counts=_i32([1, 2])),
                dict(eps=-1.0), dict(cos_sin=z(0, 64)), dict(w_uk=z(16, 128, 511, dtype=torch.bfloat16)),
                dict(kv=z(3, 4, 580, dtype=torch.bfloat16)[..., :576])):
        with pytest.raises(ValueError):
            s.attend(**{**_inputs(s, 4), **bad})
    for ptr, rows in (([0, 1], []), ([0], [5]), ([0, 1, 2, 3], [1, 1, 1]), ([0, 4], [1]), ([2, 1], [1]), ([-1, 1], [1]), ([0, 3], [-1]),
                      (_i32([0, 3]).long(), _i32([64]))):
        with pytest.raises(ValueError):
            s.set_sharing(ptr, rows)
    x = z(3, 104)
    good = dict(logits=x, V=100, u=z(3))
    for bad in (dict(V=0), dict(V=105), dict(u=None), dict(u=z(2)), dict(logits=z(104)), dict(logits=z(3, 101)),
                dict(logits=x.double()), dict(top_k=z(3)), dict(temperature=z(3, 1)), dict(probs=z(2, 104)),
                dict(logits=z(104, 3).t()), dict(probs=z(3, 99))):
        with pytest.raises(ValueError):
            s.sample(**{**good, **bad})
    with pytest.raises(ValueError):
        s.release(z(3))
    assert lib.calls == []
    with pytest.raises(ValueError):
        step(max_sets=-1)


def test_sharing_and_sampling_arguments(step, lib):
    s = step(B=3, max_sets=4)
    s.set_sharing([0, 2], [130])
    assert s.set_ptr.tolist() == [0, 2, 2, 2, 2] and s.prefix_lens.tolist() == [130, 0, 0, 0]
    s.set_sharing(_i32([0, 1, 3]), _i32([64, 70]))
    assert s.set_ptr.tolist() == [0, 1, 3, 3, 3] and s.prefix_lens.tolist() == [64, 70, 0, 0]
    s.set_sharing([0], [])
    assert s.set_ptr.tolist() == [0] * 5 and s.prefix_lens.tolist() == [0] * 4
    x = torch.zeros(7, 112, dtype=torch.bfloat16)
    assert s.sample(x, 100, u=torch.zeros(7)).shape == (7,)
    assert lib.args["mla_sample"][:5] == (7, 100, x, 1, 112)
    p = torch.zeros(3, 104)
    assert s.sample(torch.zeros(3, 104), 101, probs=p) is None
    args = lib.args["mla_sample"]
    assert args[3] == 0 and args[9:14] == (None, None, p, 0, 104)
    assert s.sample(torch.zeros(3, 104), 101, u=torch.zeros(3)) is s.tokens


def test_a_vocabulary_past_the_samplings_sums(step, lib):
    s = step(B=1)
    x = torch.zeros(1, 1 << 20)
    with pytest.raises(ValueError):
        s.sample(x, 1 << 20, u=torch.zeros(1))
    assert lib.calls == []
    s.sample(x, (1 << 20) - 1, u=torch.zeros(1))
    assert lib.args["mla_sample"][1] == (1 << 20) - 1


def test_a_set_that_loses_a_member_shares_nothing(step, lib):
    """Released and forked sequences hold other blocks from then on: their sets' prefixes are forgotten, the others' stand."""
    s = step(B=7, T=8, max_sets=6, num_blocks=30)
    s.attend(**_inputs(s, 8))
    release = lambda *b: s.release(torch.tensor([i in b for i in range(7)]))  # noqa: E731
    fork = lambda src, dst: s.fork(_i32(src), _i32(dst))  # noqa: E731
    told = [100, 200, 300, 400]
    for what, args, left in ((release, (), told), (release, (0,), told), (release, (1,), [0, 200, 300, 400]),
                             (release, (2, 5), [0, 200, 300, 0]), (release, range(7), [0, 200, 0, 0]),
                             (fork, ([0], [4]), [100, 200, 0, 400]), (fork, ([4, 4], [5, 6]), [100, 200, 300, 0]),
                             (fork, ([4], [0]), told),
                             # a last page of its own, and forks that are refused: the rows stay
                             (fork, ([4], [4]), told), (fork, ([0, 6], [4, 4]), told), (fork, ([-1], [4]), told), (fork, ([0], [7]), told)):
        s.set_sharing([1, 3, 3, 5, 6], told)          # 1 and 2; none; 3 and 4; 5
        what(*args)
        assert s.prefix_lens.tolist() == left + [0, 0], (what, args)
        assert s.set_ptr.tolist() == [1, 3, 3, 5, 6, 6, 6]
    none = step(max_sets=0)
    none.release(torch.tensor([True, False, True]))


def test_bounds_that_leave_the_batch_keep_no_set(step, lib):
    """Bounds on the device are not looked at on the host; the plan reports them, and release does not go by them."""
    s = step(B=3, max_sets=3)
    s.set_sharing(_i32([-5, 2, 1 << 30]), _i32([64, 64]))
    s.release(torch.tensor([False, True, False]))
    assert s.prefix_lens.tolist() == [0, 64, 0]
    s.release(torch.tensor([False, False, True]))
    assert s.prefix_lens.tolist() == [0, 0, 0]


def test_tokens_of_an_earlier_draw_stay(step, lib):
    s = step(B=3)
    x = torch.zeros(3, 104)
    draws = []
    for i in range(3):
        draws.append(s.sample(x, 101, u=torch.zeros(3)))
        assert lib.args["mla_sample"][10] is draws[-1] is s.tokens
        draws[-1].fill_(i)
    assert [d.tolist() for d in draws] == [[0] * 3, [1] * 3, [2] * 3]
    assert s.sample(x, 101, probs=torch.zeros(3, 104)) is None and s.tokens is draws[2]
    lib.answers["mla_sample"] = -6
    with pytest.raises(Exception):
        s.sample(x, 101, u=torch.zeros(3))
    assert s.tokens is draws[2]
