"""What a speculative step promises on the host (no GPU needed): the library's calls are stood in for by
plain versions on CPU tensors."""
import numpy as np
import pytest

from oracle import spec_oracle as O

torch = pytest.importorskip("torch")


class Library:
    """Plain versions of the page calls, in the binding's place; every call is kept in `calls`."""

    def __init__(self, binding, monkeypatch):
        from mla_latent_cache_gb300 import runtime
        self.calls, self.answers, self.reported = [], {}, False
        for name in ("mla_pages_resize", "mla_pages_fork", "mla_cache_copy", "mla_rope_append", "mla_absorb_q",
                     "mla_plan_tree", "mla_decode_tree", "mla_unabsorb_o", "mla_verify_tree", "mla_cache_compact"):
            monkeypatch.setattr(runtime.L, name, self._call(name, getattr(self, name, None)))

    def _call(self, name, plain):
        def call(*args):
            self.calls.append(name)
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
        self.reported |= not np.array_equal(pages.lens, new.numpy())
        for t, v in ((refs, pages.refs), (bt, pages.bt), (got, pages.lens)):
            t.copy_(torch.from_numpy(v))

    def mla_pages_fork(self, refs, nb, bt, stride, max_pages, lens, B, src, dst, F, copies, stream):
        s, d = src.tolist(), dst.tolist()
        inside = lambda b: 0 <= b < B  # noqa: E731
        good = [f for f in range(F) if inside(s[f]) and inside(d[f]) and d.count(d[f]) == 1 and (s[f] == d[f] or s[f] not in d)]
        self.reported |= len(good) < F
        pages = O.Pages(bt.numpy(), refs.numpy(), lens.numpy())
        copies[0], copies[1], copies[2] = -2, -1, 0
        copies[:, good] = torch.from_numpy(pages.fork([s[f] for f in good], [d[f] for f in good]))
        for t, v in ((refs, pages.refs), (bt, pages.bt), (lens, pages.lens)):
            t.copy_(torch.from_numpy(v))


@pytest.fixture
def lib(mla, monkeypatch):
    return Library(mla, monkeypatch)


@pytest.fixture
def step(lib):
    from mla_latent_cache_gb300.runtime import SpecStep

    def make(lens=(), B=2, T=4, H=16, max_pages=4, num_blocks=16):
        s = SpecStep(B, H, T, max_pages=max_pages, num_blocks=num_blocks, device="cpu")
        if len(lens):
            lib.mla_pages_resize(s.refs, num_blocks, s.block_table, max_pages, max_pages, s.seq_lens,
                                 torch.tensor(lens, dtype=torch.int32), B, s.seq_lens, None)
        lib.calls.clear()
        return s
    return make


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _pages(s):
    return {b: (int(s.seq_lens[b]), s.block_table[b].tolist()) for b in range(s.B)}


@pytest.mark.parametrize("src,dst", [
    ([0], [-1]), ([0], [4]), ([0], [2 ** 31 - 1]), ([0], [-2 ** 31]),       # no such sequence
    ([-1], [1]), ([4], [1]), ([-2 ** 31], [1]),
    ([0, 2], [1, 1]),                                                       # a sequence forked from two
    ([1, 0], [2, 1]),                                                       # a source that is written over
    ([1, 0], [1, 1]),
])
def test_refused_forks_change_nothing(step, lib, src, dst):
    s = step(lens=[70, 130, 5, 64], B=4)
    before, refs = _pages(s), s.refs.tolist()
    s.fork(_i32(src), _i32(dst))
    touched = {1} if (src, dst) == ([1, 0], [2, 1]) else set()     # (the fork of 0 to 1 itself stands)
    assert lib.reported
    for b in range(4):
        if b not in touched:
            assert _pages(s)[b] == before[b]
    if touched:
        assert _pages(s)[1][0] == 70 and _pages(s)[1][1][0] == before[0][1][0]
    else:
        assert s.refs.tolist() == refs


def test_good_forks_among_refused_ones(step, lib):
    s = step(lens=[70, 130, 5, 64], B=4)
    before = _pages(s)
    s.fork(_i32([0, 0, 3, -1]), _i32([2, -1, 4, 1]))
    after = _pages(s)
    assert after[0] == before[0] and after[1] == before[1] and after[3] == before[3]
    assert after[2][0] == 70 and after[2][1][0] == before[0][1][0] and after[2][1][1] != before[0][1][1]
    O.Pages(s.block_table.numpy(), s.refs.numpy(), s.seq_lens.numpy()).check()


def test_a_sequence_forked_from_itself_keeps_its_rows(step, lib):
    s = step(lens=[70, 130], B=2)
    before = _pages(s)
    s.fork(_i32([0]), _i32([0]))                    # its last page is its own already
    assert _pages(s) == before and not lib.reported
    s.block_table[1] = s.block_table[0]             # both sequences hold the same two pages
    s.refs.copy_(torch.zeros(16, dtype=torch.int32))
    s.refs[s.block_table[0, :2].long()] = 2
    s.seq_lens[1] = 70
    s.fork(_i32([1]), _i32([1]))
    after = _pages(s)
    assert after[0] == before[0] and after[1][0] == 70
    assert after[1][1][0] == before[0][1][0] and after[1][1][1] not in before[0][1]
    O.Pages(s.block_table.numpy(), s.refs.numpy(), s.seq_lens.numpy()).check()


def _inputs(s, V=60):
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    B, T, H = s.B, s.T, s.H
    return (dict(q=z(B, T, H, 192), kv=z(B, T, 576), cos_sin=z(64, 64, dtype=torch.float32), w_uk=z(H, 128, 512),
                 w_uv=z(H, 128, 512), kv_weight=z(512)),
            dict(target_probs=torch.zeros(B, T, 64), draft_probs=None, tokens=torch.zeros(B, T, dtype=torch.int32),
                 u_accept=torch.zeros(B, T), u_sample=torch.zeros(B), V=V))


def test_what_a_call_would_refuse_is_refused_before_anything_runs(step, lib):
    s = step(lens=[70, 5])
    attend, accept = _inputs(s)
    before = _pages(s)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(cos_sin=torch.zeros(0, 64)),
                dict(q=torch.zeros(2, 4, 16, 192, dtype=torch.bfloat16, device="meta"))):
        with pytest.raises(ValueError):
            s.attend(**{**attend, **bad})
    assert lib.calls == [] and _pages(s) == before
    s.attend(**attend)
    lib.calls.clear()
    for bad in (dict(V=0), dict(V=-3), dict(V=65), dict(target_probs=torch.zeros(1, 1, 64).expand(2, 4, 64)),
                dict(draft_probs=torch.zeros(2, 4, 64, device="meta"))):
        with pytest.raises(ValueError):
            s.accept(**{**accept, **bad})
    assert lib.calls == []
    s.accept(**accept)                        # the step goes on as if nothing had been asked
    s.commit()


def test_sizes_that_no_call_takes(lib):
    from mla_latent_cache_gb300.runtime import SpecStep
    ok = dict(B=2, H=16, T=4, max_pages=4, num_blocks=8, device="cpu")
    SpecStep(**ok)
    for bad in (dict(T=0), dict(T=1025), dict(B=8193), dict(B=-1), dict(num_blocks=0), dict(num_blocks=1 << 25),
                dict(max_pages=0), dict(max_pages=1 << 25)):
        with pytest.raises(ValueError):
            SpecStep(**{**ok, **bad})


@pytest.mark.parametrize("name,answer", [("mla_rope_append", -1), ("mla_absorb_q", -6), ("mla_plan_tree", -2),
                                         ("mla_decode_tree", -6), ("mla_unabsorb_o", MemoryError()),
                                         ("mla_rope_append", KeyboardInterrupt())])
def test_a_failed_attend_gives_its_pages_back(step, lib, mla, name, answer):
    s = step(lens=[62, 130], T=8)
    s.set_tree(np.tile(np.arange(-1, 7), (2, 1)), np.array([8, 3]))
    attend, accept = _inputs(s)
    before, refs = _pages(s), s.refs.tolist()
    lib.answers[name] = answer
    with pytest.raises(mla.MlaError if isinstance(answer, int) else type(answer)):
        s.attend(**attend)
    assert _pages(s) == before and s.refs.tolist() == refs
    with pytest.raises(RuntimeError):
        s.accept(**accept)                    # nothing is attended
    lib.answers.clear()
    s.attend(**attend)
    assert s.held_lens.tolist() == [70, 133] and int((s.block_table[0] >= 0).sum()) == 2
    O.Pages(s.block_table.numpy(), s.refs.numpy(), s.held_lens.numpy()).check()


def test_failed_accept_and_commit_can_be_repeated(step, lib, mla):
    s = step(lens=[62, 130])
    attend, accept = _inputs(s)
    s.attend(**attend)
    lib.answers["mla_verify_tree"] = -6
    with pytest.raises(mla.MlaError):
        s.accept(**accept)
    with pytest.raises(RuntimeError):
        s.commit()
    lib.answers["mla_verify_tree"] = 0
    s.accept(**accept)
    lib.answers["mla_cache_compact"] = -6
    with pytest.raises(mla.MlaError):
        s.commit()
    lib.answers.update(mla_cache_compact=0, mla_pages_resize=-6)
    with pytest.raises(mla.MlaError):
        s.commit()
    lib.answers.clear()
    lib.calls.clear()
    s.commit()
    assert lib.calls == ["mla_pages_resize"]  # the rows were moved already
    s.attend(**attend)


def test_trees_are_set_between_steps(step, lib):
    """The verification goes by the trees that were attended."""
    s = step(lens=[70, 5])
    attend, accept = _inputs(s)
    chain, star = np.tile(np.arange(-1, 3), (2, 1)), np.array([[-1, 0, 0, 0]] * 2)
    s.set_tree(chain, np.array([4, 4]))
    for part in (lambda: s.attend(**attend), lambda: s.accept(**accept)):
        part()
        with pytest.raises(RuntimeError):
            s.set_tree(star, np.array([4, 4]))
        assert s.parents.tolist() == chain.tolist()
    s.commit()
    s.set_tree(star, np.array([4, 4]))
    assert s.parents.tolist() == star.tolist()


def test_current_stream_with_and_without_torchs_own_names(mla):
    from types import SimpleNamespace as N
    cuda = N(current_stream=lambda: N(cuda_stream=7))
    own = {"_cuda_getDevice": lambda: 3, "_cuda_getCurrentRawStream": lambda device: 10 + device}
    assert mla._stream_getter(N(_C=N(**own), cuda=cuda))() == 13
    for missing in own:
        assert mla._stream_getter(N(_C=N(**{k: v for k, v in own.items() if k != missing}), cuda=cuda))() == 7


def test_more_forks_than_a_call_takes(step, lib):
    """Refused before anything is given back."""
    s = step(lens=[70, 130], B=2)
    before = _pages(s)
    with pytest.raises(ValueError):
        s.fork(torch.zeros(4097, dtype=torch.int32), torch.ones(4097, dtype=torch.int32))
    assert lib.calls == [] and _pages(s) == before
    s.fork(torch.zeros(0, dtype=torch.int32), torch.zeros(0, dtype=torch.int32))
    assert _pages(s) == before


def test_the_workspace_for_converted_pages_can_be_declined(lib, mla):
    from mla_latent_cache_gb300.runtime import SpecStep
    size = lambda **kw: SpecStep(3, 32, 9, max_pages=5, num_blocks=8, device="cpu", cache_format="fp8", num_slots=4, **kw).ws_bytes  # noqa: E731
    plan = mla.mla_workspace_size(mla.make_geom(32), mla.make_batch(3, 9, False, 5, 4))
    assert size(convert_ahead=False) == plan
    assert plan + 15 * 64 * 1152 <= size() <= plan + 15 * 64 * 1152 + 512
