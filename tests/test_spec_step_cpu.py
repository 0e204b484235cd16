"""What a speculative step refuses on the host (no GPU needed), and its trees."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def step(mla):
    from mla_latent_cache_gb300.runtime import SpecStep
    return lambda B=2, T=4, H=16: SpecStep(B, H, T, max_pages=4, num_blocks=8, device="cpu")


def _attend_args(s, **kw):
    B, T, H = s.B, s.T, s.H
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    a = dict(q=z(B, T, H, 192), kv=z(B, T, 576), cos_sin=z(64, 64, dtype=torch.float32), w_uk=z(H, 128, 512),
             w_uv=z(H, 128, 512), q_weight=None, kv_weight=z(512))
    a.update(kw)
    return a


def test_attend_refuses_what_it_would_misread(step):
    s = step()
    bad = dict(
        q=[torch.zeros(2, 4, 16, 192), torch.zeros(2, 4, 16, 576, dtype=torch.bfloat16),
           torch.zeros(2, 6, 16, 192, dtype=torch.bfloat16)[:, :4],            # sequences further apart than T rows
           torch.zeros(2, 4, 192, 16, dtype=torch.bfloat16).transpose(2, 3),
           torch.zeros(2, 4, 16, 196, dtype=torch.bfloat16)[..., :192]],       # heads 392 bytes apart
        kv=[torch.zeros(2, 4, 576), torch.zeros(2, 4, 512, dtype=torch.bfloat16),
            torch.zeros(2, 5, 576, dtype=torch.bfloat16)[:, :4], torch.zeros(2, 4, 577, dtype=torch.bfloat16)[..., 1:]],
        cos_sin=[torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, 32), torch.zeros(64, 128)[:, :64]],
        w_uk=[torch.zeros(16, 512, 128, dtype=torch.bfloat16)], w_uv=[torch.zeros(16, 128, 512)],
        q_weight=[torch.zeros(192)], kv_weight=[torch.zeros(576, dtype=torch.bfloat16)])
    for name, values in bad.items():
        for t in values:
            with pytest.raises(ValueError):
                s.attend(**_attend_args(s, **{name: t}))
    with pytest.raises(RuntimeError):
        s.commit()                                                              # nothing is attended


def test_accept_refuses_what_it_would_misread(step):
    s = step()
    ok = dict(target_probs=torch.zeros(2, 4, 64), draft_probs=torch.zeros(2, 4, 64),
              tokens=torch.zeros(2, 4, dtype=torch.int32), u_accept=torch.zeros(2, 4), u_sample=torch.zeros(2), V=60)
    bad = dict(
        target_probs=[torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 4, 64, dtype=torch.float64),
                      torch.zeros(2, 4, 56), torch.zeros(2, 3, 64), torch.zeros(2, 4, 66), torch.zeros(2, 5, 64)[:, :4]],
        draft_probs=[torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 68), torch.zeros(2, 4, 68)[..., :64]],
        tokens=[torch.zeros(2, 4, dtype=torch.int64)], u_accept=[torch.zeros(2, 4, dtype=torch.float64), torch.zeros(4, 2)],
        u_sample=[torch.zeros(1)], V=[65])
    for name, values in bad.items():
        for t in values:
            with pytest.raises(ValueError):
                s.accept(**{**ok, name: t})
    with pytest.raises(RuntimeError):
        s.accept(**ok)                                                          # nothing is attended


def test_rows_of_one_token_steps(step):
    s = step(B=3, T=1)
    wide = torch.zeros(3, 5, 16, 192, dtype=torch.bfloat16)
    assert s._fits("q", wide[:, :1], (torch.bfloat16,), (3, 1, 16, 192), rows=True) == 5 * 16 * 192
    one = step(B=1, T=1)
    assert one._fits("p", torch.zeros(1, 1, 50), (torch.float32,), (1, 1, None), rows=True) >= 50


def test_trees_are_checked_and_padding_is_not(step):
    s = step()
    par = np.array([[-1, 0, 1, 7], [-1, -1, -1, -1]])
    with pytest.raises(ValueError):
        s.set_tree(par, np.array([4, 1]))          # node 3 hangs on no earlier node
    with pytest.raises(ValueError):
        s.set_tree(par, np.array([3, 5]))
    with pytest.raises(ValueError):
        s.set_tree(par[:, :3], np.array([3, 1]))
    s.set_tree(par, np.array([3, 1]))              # the same past the counts does not matter
    assert s.mask[0, :3, 0].tolist() == [1, 3, 7] and s.depth[0, :3].tolist() == [0, 1, 2]


def test_forks_stay_between_steps(step):
    s = step()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        s.fork(i32([0]), torch.tensor([1]))
    s._stage = "accept"
    with pytest.raises(RuntimeError):
        s.fork(i32([0]), i32([1]))
