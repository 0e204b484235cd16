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
