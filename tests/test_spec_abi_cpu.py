"""Host-side validation of the speculative step's entry points (no GPU needed): every refusal
comes before any CUDA call."""
import numpy as np
import pytest

from oracle import spec_oracle as O


def _cache(mla, **kw):
    c = dict(ckv=0x1000, kpe=0x1400, ckv_row_stride=576, ckv_block_stride=64 * 576, kpe_row_stride=576,
             kpe_block_stride=64 * 576, num_blocks=8)
    c.update(kw)
    return mla.mla_cache(*c.values())


def _caller(fn, names, ok):
    """fn(**ok) with some arguments replaced, by name."""
    def call(**kw):
        unknown = set(kw) - set(names)
        assert not unknown, unknown
        return fn(*[kw.get(n, ok[n]) for n in names], 0)
    return call


def test_rope_append_refusals(mla):
    names = ["geom", "N", "q", "qt", "qh", "kv", "kvt", "wq", "wk", "eps", "cs", "max_pos", "pos", "il", "cache",
             "slots", "q_nope", "q_pe"]
    ok = dict(geom=mla.make_geom(16), N=4, q=0x10000, qt=16 * 192, qh=192, kv=0x20000, kvt=576, wq=None, wk=0x30000,
              eps=1e-6, cs=0x40000, max_pos=4096, pos=0x50000, il=1, cache=_cache(mla), slots=0x60000, q_nope=0x70000,
              q_pe=0x80000)
    call = _caller(mla.mla_rope_append, names, ok)
    assert call(N=0) == mla.MLA_OK
    assert call(N=-1) == mla.MLA_ERR_ARG
    assert call(geom=mla.make_geom(24)) == mla.MLA_ERR_SHAPE
    assert call(max_pos=0) == mla.MLA_ERR_ARG
    assert call(eps=-1.0) == mla.MLA_ERR_ARG
    assert call(eps=float("nan")) == mla.MLA_ERR_ARG
    for name in ("q", "kv", "cs", "pos", "slots", "q_nope", "q_pe"):
        assert call(**{name: None}) == mla.MLA_ERR_ARG, name
    for name in ("q", "kv", "wq", "wk", "cs", "pos", "slots", "q_nope", "q_pe"):
        assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
    for name in ("qt", "qh", "kvt"):
        assert call(**{name: 580}) == mla.MLA_ERR_ALIGN, name
        assert call(**{name: -8}) == mla.MLA_ERR_ARG, name
    assert call(cache=_cache(mla, num_blocks=0)) == mla.MLA_ERR_ARG
    assert call(cache=_cache(mla, ckv=0x1002)) == mla.MLA_ERR_ALIGN
    assert call(cache=_cache(mla, num_blocks=1 << 25)) == mla.MLA_ERR_SHAPE    # slots are 32-bit row numbers
    assert call(N=(1 << 31) - 1) == mla.MLA_ERR_SHAPE

    names8 = names[:14] + ["rows", "nb"] + names[15:]
    call8 = _caller(mla.mla_rope_append_fp8, names8, {**ok, "rows": 0x90000, "nb": 8})
    assert call8(N=0) == mla.MLA_OK
    assert call8(rows=None) == mla.MLA_ERR_ARG
    assert call8(nb=0) == mla.MLA_ERR_ARG
    assert call8(rows=0x90008) == mla.MLA_ERR_ALIGN
    assert call8(nb=1 << 25) == mla.MLA_ERR_SHAPE
    assert call8(q_pe=None) == mla.MLA_ERR_ARG


def test_verify_tree_refusals(mla):
    names = ["B", "T", "V", "target", "draft", "dtype", "stride", "tokens", "parents", "nodes", "ua", "us", "n", "idx",
             "out"]
    ok = dict(B=2, T=4, V=1000, target=0x10000, draft=0x20000, dtype=mla.MLA_DTYPE_F32, stride=1000, tokens=0x30000,
              parents=0x40000, nodes=None, ua=0x50000, us=0x60000, n=0x70000, idx=0x80000, out=0x90000)
    call = _caller(mla.mla_verify_tree, names, ok)
    assert call(B=0) == mla.MLA_OK
    for kw in (dict(B=-1), dict(T=0), dict(V=0), dict(stride=999), dict(dtype=2), dict(dtype=-1)):
        assert call(**kw) == mla.MLA_ERR_ARG, kw
    assert call(T=1025) == mla.MLA_ERR_SHAPE
    assert call(V=(1 << 30) + 1, stride=1 << 31) == mla.MLA_ERR_SHAPE
    for name in ("target", "tokens", "parents", "ua", "us", "n", "idx", "out"):
        assert call(**{name: None}) == mla.MLA_ERR_ARG, name
    for name in ("target", "draft", "tokens", "parents", "nodes", "ua", "us", "n", "idx", "out"):
        assert call(**{name: 0x10008}) == mla.MLA_ERR_ALIGN, name
    assert call(stride=1001) == mla.MLA_ERR_ALIGN
    assert call(stride=1004, dtype=mla.MLA_DTYPE_BF16) == mla.MLA_ERR_ALIGN     # 2008 bytes


def test_cache_compact_and_copy_refusals(mla):
    names = ["bt", "stride", "mp", "lens", "nodes", "acc", "idx", "B", "T", "new"]
    ok = dict(bt=0x10000, stride=8, mp=8, lens=0x20000, nodes=0x30000, acc=0x40000, idx=0x50000, B=2, T=4, new=0x60000)
    for first, bad in ((["cache"], [(dict(cache=_cache(mla, num_blocks=0)), mla.MLA_ERR_ARG),
                                    (dict(cache=_cache(mla, ckv=0x1004)), mla.MLA_ERR_ALIGN),
                                    (dict(cache=_cache(mla, num_blocks=1 << 25)), mla.MLA_ERR_SHAPE)]),
                       (["rows", "nb"], [(dict(rows=None), mla.MLA_ERR_ARG), (dict(nb=0), mla.MLA_ERR_ARG),
                                         (dict(rows=0x70004), mla.MLA_ERR_ALIGN), (dict(nb=1 << 25), mla.MLA_ERR_SHAPE)])):
        fp8 = first[0] == "rows"
        pool = dict(rows=0x70000, nb=8) if fp8 else dict(cache=_cache(mla))
        call = _caller(mla.mla_cache_compact_fp8 if fp8 else mla.mla_cache_compact, first + names, {**pool, **ok})
        assert call(B=0) == mla.MLA_OK
        for kw, want in bad:
            assert call(**kw) == want, kw
        for kw in (dict(B=-1), dict(T=0), dict(mp=0), dict(mp=9)):
            assert call(**kw) == mla.MLA_ERR_ARG, kw
        assert call(T=1025) == mla.MLA_ERR_SHAPE
        assert call(mp=1 << 25, stride=1 << 25) == mla.MLA_ERR_SHAPE
        for name in ("bt", "lens", "acc", "idx", "new"):
            assert call(**{name: None}) == mla.MLA_ERR_ARG, name
        for name in ("bt", "lens", "nodes", "acc", "idx", "new"):
            assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
        for name in ("lens", "nodes", "acc", "idx"):   # several CTAs' inputs: the new lengths need their own array
            assert call(new=ok[name]) == mla.MLA_ERR_ARG, name
        copy = _caller(mla.mla_cache_copy_fp8 if fp8 else mla.mla_cache_copy, first + ["copies", "n"],
                       {**pool, "copies": 0x80000, "n": 3})
        assert copy(n=0) == mla.MLA_OK
        assert copy(n=-1) == mla.MLA_ERR_ARG
        assert copy(copies=None) == mla.MLA_ERR_ARG
        assert copy(copies=0x80008) == mla.MLA_ERR_ALIGN
        for kw, want in bad:
            assert copy(**kw) == want, kw


def test_pages_resize_and_fork_refusals(mla):
    names = ["refs", "nb", "bt", "stride", "mp", "cur", "new", "B", "got"]
    ok = dict(refs=0x10000, nb=64, bt=0x20000, stride=8, mp=8, cur=0x30000, new=0x40000, B=4, got=0x30000)
    call = _caller(mla.mla_pages_resize, names, ok)
    assert call(B=0) == mla.MLA_OK
    for kw in (dict(B=-1), dict(nb=0), dict(mp=0), dict(mp=9), *({n: None} for n in ("refs", "bt", "cur", "new", "got"))):
        assert call(**kw) == mla.MLA_ERR_ARG, kw
    for name in ("refs", "bt", "cur", "new", "got"):
        assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
    assert call(B=8193) == mla.MLA_ERR_SHAPE
    assert call(mp=1 << 25, stride=1 << 25) == mla.MLA_ERR_SHAPE
    assert call(B=4096, mp=1 << 20, stride=1 << 20) == mla.MLA_ERR_SHAPE

    names = ["refs", "nb", "bt", "stride", "mp", "lens", "B", "src", "dst", "F", "copies"]
    call = _caller(mla.mla_pages_fork, names, {**ok, "lens": 0x30000, "src": 0x50000, "dst": 0x60000, "F": 2, "copies": 0x70000})
    assert call(F=0) == mla.MLA_OK
    for kw in (dict(B=-1), dict(B=0), dict(F=-1), dict(nb=0), dict(mp=9),
               *({n: None} for n in ("refs", "bt", "lens", "src", "dst", "copies"))):
        assert call(**kw) == mla.MLA_ERR_ARG, kw
    for name in ("refs", "bt", "lens", "src", "dst", "copies"):
        assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
    assert call(F=4097) == mla.MLA_ERR_SHAPE
    assert call(B=65537) == mla.MLA_ERR_SHAPE


def test_tree_decode_refusals(mla):
    g, b = mla.make_geom(16), mla.make_batch(2, 8, False, 8, num_slots=4)
    ws = mla.mla_workspace_size(g, b)
    plan = _caller(mla.mla_plan_tree, ["geom", "batch", "lens", "nodes", "ws", "bytes"],
                   dict(geom=g, batch=b, lens=0x10000, nodes=0x20000, ws=0x40000, bytes=ws))
    names = ["geom", "batch", "q_lat", "q_pe", "cache", "bt", "stride", "lens", "nodes", "mask", "checked", "o", "lse",
             "ws", "bytes"]
    ok = dict(geom=g, batch=b, q_lat=0x10000, q_pe=0x20000, cache=_cache(mla), bt=0x30000, stride=8, lens=0x40000,
              nodes=0x50000, mask=0x60000, checked=0, o=0x70000, lse=0x80000, ws=0x90000, bytes=ws)
    dec = _caller(mla.mla_decode_tree, names, ok)
    names8 = names[:4] + ["rows", "nb"] + names[5:]
    dec8 = _caller(mla.mla_decode_tree_fp8, names8, {**ok, "rows": 0xA0000, "nb": 8})
    for call in (plan, dec, dec8):
        assert call(batch=mla.make_batch(2, 8, True, 8, num_slots=4)) == mla.MLA_ERR_ARG      # causal
        assert call(batch=mla.make_batch(2, 0, False, 8, num_slots=4)) == mla.MLA_ERR_ARG
        assert call(batch=mla.make_batch(2, 1025, False, 8, num_slots=4)) == mla.MLA_ERR_SHAPE
        assert call(geom=mla.make_geom(24)) == mla.MLA_ERR_SHAPE
        assert call(bytes=ws - 1) == mla.MLA_ERR_WORKSPACE
        assert call(ws=None) == mla.MLA_ERR_ARG
        assert call(ws=0x90010) == mla.MLA_ERR_ALIGN
        assert call(lens=None) == mla.MLA_ERR_ARG
        for name in ("lens", "nodes"):
            assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
    # FP8 pages converted ahead: B * max_pages bf16 pages and their table, where T * H > 128
    assert mla.mla_tree_fp8_workspace_size(g, b) == ws
    b2 = mla.make_batch(2, 9, False, 8, num_slots=4)
    assert mla.mla_tree_fp8_workspace_size(g, b2) == mla.mla_workspace_size(g, b2) + 256 + 2 * 8 * 64 * 1152
    for bad in (mla.make_batch(2, 9, True, 8, num_slots=4), mla.make_batch(2, 1025, False, 8, num_slots=4),
                mla.make_batch(2, 0, False, 8, num_slots=4)):
        assert mla.mla_tree_fp8_workspace_size(g, bad) == 0
    assert mla.mla_tree_fp8_workspace_size(mla.make_geom(24), b) == 0
    for call in (dec, dec8):
        assert call(batch=mla.make_batch(0, 8, False, 8, num_slots=4)) == mla.MLA_OK
        for name in ("q_lat", "q_pe", "bt", "mask", "o", "lse"):
            assert call(**{name: None}) == mla.MLA_ERR_ARG, name
            assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
        assert call(o=0x70010) == mla.MLA_ERR_ALIGN
        assert call(stride=7) == mla.MLA_ERR_ARG
    assert dec(cache=_cache(mla, num_blocks=0)) == mla.MLA_ERR_ARG
    assert dec8(rows=None) == mla.MLA_ERR_ARG
    assert dec8(nb=0) == mla.MLA_ERR_ARG
    assert dec8(rows=0xA0008) == mla.MLA_ERR_ALIGN


def test_rotation_oracle_is_a_rotation():
    """Inner products of rotated pairs depend on the difference of the angles only, both pairings
    agree up to the order of the values, and position 0 turns nothing."""
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal(64), rng.standard_normal(64)
    inv = 10000.0 ** (-np.arange(0, 64, 2) / 64)

    def cs(p):
        return np.concatenate([np.cos(p * inv), np.sin(p * inv)])

    for il in (False, True):
        assert np.array_equal(O.rotate_ref(a, cs(0), il), a)
        x = O.rotate_ref(a, cs(30), il) @ O.rotate_ref(b, cs(11), il)
        y = O.rotate_ref(a, cs(19), il) @ b
        assert abs(x - y) < 1e-12
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    assert np.allclose(O.rotate_ref(a[order], cs(7), False), O.rotate_ref(a, cs(7), True)[order], atol=1e-15)
    # the textbook form, written out for one pair
    z = O.rotate_ref(a, cs(3), True)
    c, s = np.cos(3 * inv[4]), np.sin(3 * inv[4])
    assert np.isclose(z[8], a[8] * c - a[9] * s) and np.isclose(z[9], a[9] * c + a[8] * s)


def test_tree_words(mla):
    from mla_latent_cache_gb300.runtime import tree_words
    par = np.array([[-1, 0, 0, 1, 2, 4], [-1, 0, 1, 2, 3, 4]])
    words, depth = tree_words(par)
    see = O.ancestors(par)
    assert np.array_equal(words[..., 0], (see << np.arange(6)).sum(-1))
    assert np.array_equal(depth, see.sum(-1) - 1)
    with pytest.raises(ValueError):
        tree_words(np.array([[-1, 0, 2]]))
