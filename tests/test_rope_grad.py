"""mla_rope and autograd: a lost graph is refused, and the inverse call is the gradient."""
import pytest
import torch

import __graft_entry__ as G
from tests import prefill_reference as P


@pytest.fixture(scope="module")
def M():
    G._load_by_path("_libmla_build", "paged_mla_decode_10_gb300/build.py").build()
    import paged_mla_decode_10_gb300
    return paged_mla_decode_10_gb300


def test_tensors_that_require_a_graph_are_refused(M):
    x, pos, plan = torch.zeros((3, 2, 64)), torch.arange(3, dtype=torch.int32), M.mla_rope_plan(64)
    leaf = x.clone().requires_grad_()
    for kw in (dict(x=leaf), dict(x=leaf * 2), dict(x=x, out=leaf)):
        with pytest.raises(ValueError, match="no graph"):
            M.mla_rope(positions=pos, plan=plan, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):    # only the device is wrong now
            M.mla_rope(positions=pos, plan=plan, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        M.mla_rope(x, pos, plan)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("scaling", [None, dict(kind="yarn", factor=40.0, original_max_position=4096)])
def test_gradient_in_a_function(M, interleaved, scaling):
    plan = M.mla_rope_plan(32, interleaved=interleaved, scaling=scaling)
    pos = torch.tensor([0, 1, 77, 100_000, 3_000_000], dtype=torch.int32, device="cuda")

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return M.mla_rope(x, pos, plan)

        @staticmethod
        def backward(ctx, g):
            return M.mla_rope(g.contiguous(), pos, plan, inverse=True)

    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((5, 3, 48), generator=gen, device="cuda").requires_grad_()
    w = torch.randn((5, 3, 48), generator=gen, device="cuda")
    (Rotate.apply(x) * w).sum().backward()
    freq, factor = P.frequencies(32, 10000.0, scaling)
    want, bound = P.rotate(w[..., 16:], pos, freq.cuda(), factor, interleaved, inverse=True)
    assert torch.equal(x.grad[..., :16], w[..., :16])
    assert ((x.grad[..., 16:].double() - want).abs() <= bound + P.half_step(want, torch.float32)).all()
