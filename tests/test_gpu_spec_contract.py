"""What the calls of a speculative step promise beyond their results at aligned, well-formed inputs."""
import numpy as np
import pytest

from tests.test_gpu_tree import Tree

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
