"""mla_rope_append / mla_rope_append_fp8 against the float64 definition.

Bound of each value: one rounding to bf16 (2^-8 of the value), plus the fp32 steps before
it: at most 24 additions deep in a sum of squares (halved by the root), 4 half steps of
rsqrt, 2 products, 3 roundings of a rotation whose terms may cancel: under 32 half steps
(2^-24) of the magnitude |a| + |b| that went in, 2^-19.
"""
import numpy as np
import pytest

from mla_latent_cache_gb300 import workloads as W
from oracle import spec_oracle as O

pytestmark = pytest.mark.gpu

EPS = 1e-6
MAX_POS = 4096


def _table():
    ang = np.arange(MAX_POS)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _bits(rng, shape, scale=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * np.float32(scale))


def _dev(torch, bits, cuda):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(cuda).view(torch.bfloat16)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    def __init__(self, torch, cuda, N, H, q_norm=True, kv_norm=True, seed=0, spare=1, strided=False):
        rng = np.random.default_rng([seed, N, H])
        self.N, self.H, self.nb = N, H, (N + 63) // 64 + spare
        qb, kvb = _bits(rng, (N, H, 192)), _bits(rng, (N, 576), 1.5)
        wq = W.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(192)).astype(np.float32))
        wk = W.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(512)).astype(np.float32))
        f = W.bf16_bits_to_f64
        self.ref_in = (f(qb), f(kvb), f(wq) if q_norm else None, f(wk) if kv_norm else None)
        self.table = _table()
        self.pos = rng.integers(0, MAX_POS, N).astype(np.int32)
        self.pos[0] = 0
        self.slot = rng.permutation(self.nb * 64)[:N].astype(np.int32)
        if strided:   # a head row of 200, a token row of H heads and 8 values more; kv rows 592 apart
            qs = torch.full((N, H * 200 + 8), float("nan"), dtype=torch.bfloat16, device=cuda)
            self.q = torch.as_strided(qs, (N, H, 192), (H * 200 + 8, 200, 1))
            self.q.copy_(_dev(torch, qb, cuda))
            ks = torch.full((N, 592), float("nan"), dtype=torch.bfloat16, device=cuda)
            self.kv = ks[:, :576]
            self.kv.copy_(_dev(torch, kvb, cuda))
        else:
            self.q, self.kv = _dev(torch, qb, cuda), _dev(torch, kvb, cuda)
        self.wq = _dev(torch, wq, cuda) if q_norm else None
        self.wk = _dev(torch, wk, cuda) if kv_norm else None
        self.cs = torch.from_numpy(self.table).to(cuda)
        self.positions, self.slots = torch.from_numpy(self.pos).to(cuda), torch.from_numpy(self.slot).to(cuda)
        self.q_nope = torch.full((N, H, 128), 7.0, dtype=torch.bfloat16, device=cuda)
        self.q_pe = torch.full((N, H, 64), 7.0, dtype=torch.bfloat16, device=cuda)
        self.pool = torch.full((self.nb, 64, 576), 7.0, dtype=torch.bfloat16, device=cuda)

    def call(self, mla, interleaved, cache=None, stream=None):
        c = mla.cache_from_pool(self.pool) if cache is None else cache
        return mla.mla_rope_append(mla.make_geom(self.H), self.N, self.q, self.q.stride(0), self.q.stride(1), self.kv,
                                   self.kv.stride(0), self.wq, self.wk, EPS, self.cs, MAX_POS, self.positions,
                                   interleaved, c, self.slots, self.q_nope, self.q_pe, stream)

    def call_fp8(self, mla, interleaved, rows):
        return mla.mla_rope_append_fp8(mla.make_geom(self.H), self.N, self.q, self.q.stride(0), self.q.stride(1),
                                       self.kv, self.kv.stride(0), self.wq, self.wk, EPS, self.cs, MAX_POS,
                                       self.positions, interleaved, rows, self.nb, self.slots, self.q_nope, self.q_pe)

    def check(self, interleaved, pool=None, tokens=None):
        q, kv, wq, wk = self.ref_in
        ref = O.rope_append_ref(q, kv, wq, wk, EPS, self.table.astype(np.float64), self.pos, interleaved)
        # the magnitudes that went in: the two values of a pair, after the norm
        flat = np.zeros((MAX_POS, 64))
        flat[:, :32] = 1.0
        norm = O.rope_append_ref(q, kv, wq, wk, EPS, flat, self.pos, interleaved)
        pool = _f64(self.pool) if pool is None else pool
        rows = pool.reshape(-1, 576)[self.slot]
        tokens = slice(None) if tokens is None else tokens
        for name, got, want, mag in (("q_nope", _f64(self.q_nope), ref[0], np.abs(norm[0])),
                                     ("q_pe", _f64(self.q_pe), ref[1], _pair_mag(norm[1], interleaved)),
                                     ("latent", rows[:, :512], ref[2][:, :512], np.abs(norm[2][:, :512])),
                                     ("k_pe", rows[:, 512:], ref[2][:, 512:], _pair_mag(norm[2][:, 512:], interleaved))):
            bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * mag
            assert not bad[tokens].any(), (name, np.argwhere(bad)[:4], np.abs(got - want)[tokens].max())


def _pair_mag(x, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    m = np.abs(a) + np.abs(b)
    return np.repeat(m, 2, -1) if interleaved else np.concatenate([m, m], -1)


def _ok(mla, torch):
    torch.cuda.synchronize()
    assert mla.mla_read_device_status(None) == (mla.MLA_OK, 0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,q_norm,kv_norm", [(1, 128, False, True), (1, 1, True, True), (7, 2, True, False),
                                                (65, 8, False, False), (333, 16, True, True), (1000, 128, True, True)])
def test_append_matches_the_definition(mla, cuda, N, H, q_norm, kv_norm, interleaved):
    import torch
    c = Case(torch, cuda, N, H, q_norm, kv_norm)
    assert c.call(mla, interleaved) == mla.MLA_OK
    _ok(mla, torch)
    c.check(interleaved)
    # rows that no slot names are as they were
    rest = np.setdiff1d(np.arange(c.nb * 64), c.slot)
    assert np.all(_f64(c.pool).reshape(-1, 576)[rest] == 7.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_strided_inputs_and_split_pools(mla, cuda, interleaved):
    import torch
    c = Case(torch, cuda, 77, 16, strided=True)
    ckv = torch.full((c.nb, 64, 528), 7.0, dtype=torch.bfloat16, device=cuda)   # rows 528 apart: 16 values of padding
    kpe = torch.full((c.nb, 64, 64), 7.0, dtype=torch.bfloat16, device=cuda)
    assert c.call(mla, interleaved, cache=mla.cache_from_split(ckv, kpe)) == mla.MLA_OK
    _ok(mla, torch)
    c.check(interleaved, pool=np.concatenate([_f64(ckv)[..., :512], _f64(kpe)], -1))
    assert torch.all(ckv[..., 512:] == 7.0)


@pytest.mark.parametrize("N,H,interleaved", [(1, 16, True), (300, 32, False)])
def test_append_fp8_writes_the_packed_row(mla, cuda, N, H, interleaved):
    import torch
    c = Case(torch, cuda, N, H)
    c.pool.zero_()
    assert c.call(mla, interleaved) == mla.MLA_OK
    packed = torch.zeros((c.nb, 64, 656), dtype=torch.uint8, device=cuda)
    mla.check(mla.mla_fp8_pack_cache(mla.cache_from_pool(c.pool), packed))
    q_nope, q_pe = c.q_nope.clone(), c.q_pe.clone()
    rows = torch.full((c.nb, 64, 656), 99, dtype=torch.uint8, device=cuda)
    assert c.call_fp8(mla, interleaved, rows) == mla.MLA_OK
    _ok(mla, torch)
    s = c.slots.long()
    assert torch.equal(rows.view(-1, 656)[s], packed.view(-1, 656)[s])
    assert torch.equal(c.q_nope, q_nope) and torch.equal(c.q_pe, q_pe)
    rest = torch.ones(c.nb * 64, dtype=torch.bool, device=cuda)
    rest[s] = False
    assert torch.all(rows.view(-1, 656)[rest] == 99)


def test_append_padding_bad_slots_and_bad_positions(mla, cuda):
    import torch
    c = Case(torch, cuda, 9, 8)
    c.slots[2] = -1                      # a padding token: queries only, nothing reported
    assert c.call(mla, True) == mla.MLA_OK
    _ok(mla, torch)
    q_nope = c.q_nope.clone()
    written = c.pool.clone()
    assert np.all(_f64(written).reshape(-1, 576)[c.slot[2]] == 7.0)
    for slot in (c.nb * 64, -2, 2 ** 31 - 1, -2 ** 31):
        c.pool.fill_(7.0)
        c.q_nope.fill_(7.0)
        c.slots[2] = slot
        assert c.call(mla, True) == mla.MLA_OK
        assert mla.mla_read_device_status(None)[0] == mla.MLA_ERR_DEVICE_CHECK
        assert torch.equal(c.pool, written) and torch.equal(c.q_nope, q_nope)
    c.slots[2] = int(c.slot[2])
    for pos in (-1, MAX_POS, 2 ** 31 - 1):
        c.pool.fill_(7.0)
        c.q_nope.fill_(7.0)
        c.q_pe.fill_(7.0)
        c.positions[4] = pos
        assert c.call(mla, True) == mla.MLA_OK
        assert mla.mla_read_device_status(None)[0] == mla.MLA_ERR_DEVICE_CHECK
        assert torch.all(c.q_nope[4] == 7.0) and torch.all(c.q_pe[4] == 7.0)
        assert np.all(_f64(c.pool).reshape(-1, 576)[c.slot[4]] == 7.0)
        c.check(True, tokens=[0, 1, 2, 3, 5, 6, 7, 8])
    assert mla.mla_read_device_status(None) == (mla.MLA_OK, 0)


def test_append_zero_rows_and_nan(mla, cuda):
    """A zero row norms to zero (eps), and a NaN stays in its own head and row."""
    import torch
    c = Case(torch, cuda, 4, 8)
    c.q[1, 3] = 0
    c.kv[2, :512] = 0
    c.q[3, 5, 9] = float("nan")
    assert c.call(mla, False) == mla.MLA_OK
    _ok(mla, torch)
    assert torch.all(c.q_nope[1, 3] == 0) and torch.all(c.q_pe[1, 3] == 0)
    assert torch.all(c.pool.view(-1, 576)[int(c.slot[2]), :512] == 0)
    assert torch.isnan(c.q_nope[3, 5]).all() and torch.isnan(c.q_pe[3, 5]).all()
    q = torch.cat([c.q_nope, c.q_pe], -1)
    q[3, 5] = 0
    assert not torch.isnan(q).any() and not torch.isnan(c.pool).any()


def test_append_on_a_side_stream_and_in_a_graph(mla, cuda):
    import torch
    c = Case(torch, cuda, 50, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert c.call(mla, True, stream=side) == mla.MLA_OK
    side.synchronize()
    c.check(True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert c.call(mla, True) == mla.MLA_OK
    c.pool.fill_(7.0)
    c.q_nope.fill_(7.0)
    g.replay()
    _ok(mla, torch)
    c.check(True)


def test_append_at_the_end_of_a_large_pool(mla, cuda):
    """Rows whose byte offsets pass 32 bits, bf16 and FP8."""
    import torch
    c = Case(torch, cuda, 3, 8)
    small = c.call(mla, True)
    assert small == mla.MLA_OK
    rows = c.pool.view(-1, 576)[c.slots.long()].clone()
    fp8 = torch.zeros((c.nb, 64, 656), dtype=torch.uint8, device=cuda)
    assert c.call_fp8(mla, True, fp8) == mla.MLA_OK
    bytes_ = fp8.view(-1, 656)[c.slots.long()].clone()
    c.nb = 110000                                  # 8.1 GB of bf16 rows, 4.6 GB of FP8 rows
    c.slots.copy_(torch.tensor([c.nb * 64 - 1, 0, c.nb * 64 - 65], dtype=torch.int32))
    c.pool = torch.zeros((c.nb, 64, 576), dtype=torch.bfloat16, device=cuda)
    assert c.call(mla, True) == mla.MLA_OK
    _ok(mla, torch)
    flat = c.pool.view(-1, 576)
    assert torch.equal(torch.stack([flat[int(s)] for s in c.slots]), rows)
    assert int((flat[1:4096] != 0).sum()) == 0
    c.pool = flat = None
    big = torch.zeros((c.nb, 64, 656), dtype=torch.uint8, device=cuda)
    assert c.call_fp8(mla, True, big) == mla.MLA_OK
    _ok(mla, torch)
    assert torch.equal(torch.stack([big.view(-1, 656)[int(s)] for s in c.slots]), bytes_)
