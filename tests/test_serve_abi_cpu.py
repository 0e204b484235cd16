"""Host-side validation of the serving step's entry points (no GPU needed): every refusal comes
before any CUDA call."""
from tests.test_spec_abi_cpu import _caller


def test_sample_refusals(mla):
    names = ["N", "V", "logits", "dtype", "stride", "temp", "k", "p", "mp", "u", "tokens", "probs", "pd", "ps"]
    ok = dict(N=2, V=1000, logits=0x10000, dtype=mla.MLA_DTYPE_F32, stride=1000, temp=0x20000, k=0x30000, p=0x40000,
              mp=0x50000, u=0x60000, tokens=0x70000, probs=0x80000, pd=mla.MLA_DTYPE_F32, ps=1000)
    call = _caller(mla.mla_sample, names, ok)
    assert call(N=0) == mla.MLA_OK
    for kw in (dict(N=-1), dict(V=0), dict(stride=999), dict(dtype=2), dict(dtype=-1), dict(pd=2), dict(ps=999),
               dict(logits=None), dict(u=None), dict(tokens=None, probs=None), dict(probs=0x10000)):
        assert call(**kw) == mla.MLA_ERR_ARG, kw
    assert call(V=(1 << 20) + 1, stride=1 << 21, ps=1 << 21) == mla.MLA_ERR_SHAPE
    for name in ("logits", "temp", "k", "p", "mp", "u", "tokens", "probs"):
        assert call(**{name: 0x10008}) == mla.MLA_ERR_ALIGN, name
    assert call(stride=1001) == mla.MLA_ERR_ALIGN
    assert call(ps=1001) == mla.MLA_ERR_ALIGN
    assert call(stride=1004, dtype=mla.MLA_DTYPE_BF16) == mla.MLA_ERR_ALIGN     # 2008 bytes
    assert call(ps=1004, pd=mla.MLA_DTYPE_BF16) == mla.MLA_ERR_ALIGN
    # without probabilities their type and stride are not looked at
    assert call(N=0, probs=None, pd=9, ps=0) == mla.MLA_OK


def test_batch_map_refusals(mla):
    names = ["B", "T", "N", "cached", "counts", "held", "bt", "stride", "mp", "nb", "depth", "live", "lens", "cu", "seq",
             "pos", "slots"]
    ok = dict(B=4, T=0, N=10, cached=0x10000, counts=0x20000, held=0x30000, bt=0x40000, stride=8, mp=8, nb=16, depth=None,
              live=0x50000, lens=0x60000, cu=0x70000, seq=0x80000, pos=0x90000, slots=0xA0000)
    packed = _caller(mla.mla_batch_map, names, ok)
    padded = _caller(mla.mla_batch_map, names, {**ok, "T": 3, "N": 12, "cu": None, "seq": None, "depth": 0xB0000})
    for call in (packed, padded):
        for kw in (dict(B=-1), dict(T=-1), dict(N=-1), dict(mp=0), dict(mp=9), dict(nb=0)):
            assert call(**kw) == mla.MLA_ERR_ARG, kw
        assert call(mp=1 << 25, stride=1 << 25) == mla.MLA_ERR_SHAPE
        assert call(nb=1 << 25) == mla.MLA_ERR_SHAPE
        for name in ("cached", "counts", "bt", "live", "lens", "pos", "slots"):
            assert call(**{name: None}) == mla.MLA_ERR_ARG, name
        for name in ("cached", "counts", "held", "bt", "live", "lens", "pos", "slots"):
            assert call(**{name: 0x10004}) == mla.MLA_ERR_ALIGN, name
        for name in ("live", "lens", "pos", "slots"):     # outputs are none of the inputs
            for other in ("cached", "counts", "held", "bt"):
                assert call(**{name: ok[other]}) == mla.MLA_ERR_ARG, (name, other)
    assert packed(cu=0x10004) == mla.MLA_ERR_ALIGN and packed(seq=0x10004) == mla.MLA_ERR_ALIGN
    assert padded(depth=0x10004) == mla.MLA_ERR_ALIGN and padded(pos=0xB0000) == mla.MLA_ERR_ARG
    assert packed(depth=0xB0000) == mla.MLA_ERR_ARG       # positions of a tree: padded tokens
    assert padded(cu=0x70000) == mla.MLA_ERR_ARG and padded(seq=0x80000) == mla.MLA_ERR_ARG
    assert padded(N=11) == mla.MLA_ERR_ARG
    assert packed(B=8193) == mla.MLA_ERR_SHAPE and packed(N=1 << 30) == mla.MLA_ERR_SHAPE
    assert padded(B=1 << 21, T=1 << 10, N=0) == mla.MLA_ERR_SHAPE
    assert padded(B=0, N=0) == mla.MLA_OK
    assert packed(B=0, N=0, cu=None) == mla.MLA_OK


def test_shared_workspace_size(mla):
    g = mla.make_geom(16)
    size = lambda B, T, **kw: mla.mla_shared_workspace_size(kw.pop("g", g), mla.make_batch(B, T, False, 64, **{"num_slots": 8, **kw}))  # noqa: E731
    # two rows of 512 fp32 per query row, and one per row of a range's cut
    assert size(64, 3) >= (2 * 64 * 48 + 8 * 128) * 512 * 4
    assert size(64, 3) % 256 == 0 and size(0, 1) > 0
    # rows that are multiples of 128 share nothing: two cuts per range
    assert size(64, 8) < 2 * 8 * 128 * 512 * 4 + (1 << 20)
    assert size(4, 3, num_splits_override=5) >= 2 * 4 * 48 * 5 * 512 * 4
    assert size(8192, 1) > 0 and size(8193, 1) == 0
    assert size(4, 0) == 0 and size(-1, 1) == 0 and size(4, 1, g=mla.make_geom(24)) == 0
    assert size(8192, 1000, num_splits_override=64) == 0          # partial rows are 32-bit numbers


def test_shared_refusals(mla):
    from tests.test_spec_abi_cpu import _cache
    g, b = mla.make_geom(16), mla.make_batch(4, 3, True, 8, num_slots=4)
    size = mla.mla_shared_workspace_size(g, b)
    names = ["geom", "batch", "lens", "q_lens", "sets", "ptr", "prefix", "ws", "bytes"]
    plan = _caller(mla.mla_plan_shared, names, dict(geom=g, batch=b, lens=0x10000, q_lens=0x20000, sets=2, ptr=0x30000,
                                                    prefix=0x40000, ws=0x50000, bytes=size))
    for kw in (dict(sets=-1), dict(ptr=None), dict(prefix=None), dict(ws=None), dict(lens=None),
               dict(batch=mla.make_batch(4, 0, True, 8))):
        assert plan(**kw) == mla.MLA_ERR_ARG, kw
    for kw in (dict(sets=8193), dict(geom=mla.make_geom(24)), dict(batch=mla.make_batch(8193, 1, False, 8))):
        assert plan(**kw) == mla.MLA_ERR_SHAPE, kw
    for name in ("lens", "q_lens", "ptr", "prefix", "ws"):
        assert plan(**{name: 0x10008}) == mla.MLA_ERR_ALIGN, name
    assert plan(ws=0x10010) == mla.MLA_ERR_ALIGN                  # 32 bytes, as every plan
    assert plan(bytes=size - 1) == mla.MLA_ERR_WORKSPACE
    names = ["geom", "batch", "q_lat", "q_pe", "cache", "bt", "stride", "lens", "q_lens", "checked", "o", "lse", "ws", "bytes"]
    ok = dict(geom=g, batch=b, q_lat=0x10000, q_pe=0x20000, cache=_cache(mla), bt=0x30000, stride=8, lens=0x40000,
              q_lens=None, checked=0, o=0x50000, lse=0x60000, ws=0x70000, bytes=size)
    bf16 = _caller(mla.mla_decode_shared, names, ok)
    fp8 = _caller(mla.mla_decode_shared_fp8, names[:4] + ["rows", "nb"] + names[5:], {**ok, "rows": 0x80000, "nb": 8})
    for call in (bf16, fp8):
        assert call(batch=mla.make_batch(0, 3, True, 8)) == mla.MLA_OK
        for name in ("q_lat", "q_pe", "bt", "lens", "o", "lse", "ws"):
            assert call(**{name: None}) == mla.MLA_ERR_ARG, name
        for name in ("q_lat", "q_pe", "bt", "lens", "q_lens", "o", "lse", "ws"):
            assert call(**{name: 0x10008}) == mla.MLA_ERR_ALIGN, name
        for name in ("o", "ws"):
            assert call(**{name: 0x10010}) == mla.MLA_ERR_ALIGN, name
        assert call(stride=7) == mla.MLA_ERR_ARG
        assert call(bytes=size - 1) == mla.MLA_ERR_WORKSPACE
        assert call(geom=mla.make_geom(24)) == mla.MLA_ERR_SHAPE
        assert call(batch=mla.make_batch(8193, 1, False, 8)) == mla.MLA_ERR_SHAPE
    assert bf16(cache=_cache(mla, num_blocks=0)) == mla.MLA_ERR_ARG
    assert bf16(cache=_cache(mla, ckv=0x1002)) == mla.MLA_ERR_ALIGN
    assert fp8(rows=None) == mla.MLA_ERR_ARG and fp8(nb=0) == mla.MLA_ERR_ARG
    assert fp8(rows=0x80008) == mla.MLA_ERR_ALIGN and fp8(nb=1 << 25) == mla.MLA_ERR_SHAPE


def test_sample_vocabularies_whose_sums_do_not_fit(mla):
    """2^20 equal logits have a mass of 2^44 units each, together 2^64: one more than the sums hold."""
    names = ["N", "V", "logits", "dtype", "stride", "temp", "k", "p", "mp", "u", "tokens", "probs", "pd", "ps"]
    call = _caller(mla.mla_sample, names, dict(N=0, V=1 << 20, logits=0x10000, dtype=mla.MLA_DTYPE_F32, stride=1 << 20, temp=None,
                                               k=None, p=None, mp=None, u=0x60000, tokens=0x70000, probs=None, pd=0, ps=0))
    assert call() == mla.MLA_ERR_SHAPE and call(N=2) == mla.MLA_ERR_SHAPE
    assert call(V=(1 << 20) - 1) == mla.MLA_OK


def test_shared_workspace_of_what_can_share(mla):
    """Chunks of prompts that no set can save anything of need no partial states for sharing."""
    import numpy as np
    from oracle import serve_oracle as S
    size = lambda B, T, H, pages, **kw: mla.mla_shared_workspace_size(mla.make_geom(H), mla.make_batch(B, T, True, pages, num_slots=8, **kw))  # noqa: E731
    row = 512 * 4 + 4
    cuts = 2 * 8 * 128 * row
    assert size(64, 1023, 16, 64) < cuts + (4 << 20)
    assert size(64, 1, 16, 1) >= 2 * 64 * 16 * row          # a page is enough for samples
    assert size(64, 1023, 16, 64, num_splits_override=4) < 1.01 * 4 * 64 * 1023 * 16 * row + (16 << 20)
    # what can share by the planner's rule, for any number of members, has a part for every row twice
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(300):
        H, T, pages, m = (int(v) for v in (rng.choice([1, 8, 16, 64, 128]), 2 ** rng.uniform(0, 9), 2 ** rng.uniform(0, 12),
                                           rng.integers(2, 40)))
        shares = S.shared_pages_ref([64 * pages] * m, [T] * m, [0, m], [64 * pages], T, H, False, 0) != [0]
        seen.add(shares)
        if shares:
            assert size(m, T, H, pages) >= 2 * m * T * H * row, (H, T, pages, m)
    assert seen == {False, True}
