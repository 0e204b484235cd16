"""Host-side validation of the speculative step's entry points (no GPU needed): every refusal
comes before any CUDA call."""
import numpy as np

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
