"""The norm and rotation is outside autograd: it refuses tensors that a gradient is wanted of, and serves as the two halves of
an autograd function."""
import pytest
import torch

from tests import _layer_ref as ref

NAMES = ["q", "k", "gamma_q", "gamma_k", "cos", "sin"]


@pytest.fixture(scope="module")
def sg():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    import sparse_bit_attention_smoothing_b200 as s
    return s


def tensors(device, N=5, dtype=torch.float32):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(q=r(1, N, 4, 32).to(dtype).to(device), k=r(1, N, 2, 32).to(dtype).to(device), gamma_q=r(32).to(dtype).to(device),
                gamma_k=r(32).to(dtype).to(device), cos=r(N, 16).to(device), sin=r(N, 16).to(device))


@pytest.mark.parametrize("name", NAMES)
def test_refused_while_gradients_are_recorded(sg, name):
    """(On the CPU: the refusal comes before the tensors' device is looked at.)"""
    t = tensors("cpu")
    t[name].requires_grad_()
    with pytest.raises(ValueError, match="records no gradient"):
        sg.sagesla_qk_norm_rope(**t)
    with pytest.raises(ValueError, match="records no gradient"):
        sg.sagesla_qk_norm_rope_bwd(t["q"].detach(), t["k"].detach(), **t)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors are needed"):
        sg.sagesla_qk_norm_rope(**t)


def test_backward_refused_where_a_second_derivative_is_wanted(sg):
    t = tensors("cpu")
    with pytest.raises(ValueError, match="records no gradient"):
        sg.sagesla_qk_norm_rope_bwd(torch.zeros_like(t["q"]).requires_grad_(), torch.zeros_like(t["k"]), **t)


@pytest.mark.gpu
@pytest.mark.parametrize("il", [True, False])
def test_halves_of_an_autograd_function(sg, il):
    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, gq, gk, cos, sin):
            ctx.save_for_backward(q, k, gq, gk, cos, sin)
            return sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin, interleaved=il)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq, dk):
            return *sg.sagesla_qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors, interleaved=il), None, None

    t = tensors("cuda", 40)
    leaves = [t[n].clone().requires_grad_() for n in NAMES[:4]]
    yq, yk = NormRope.apply(*leaves, t["cos"], t["sin"])
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    torch.autograd.backward([yq, yk], [gq, gk])
    for x, g, dy, y in ((leaves[0], leaves[2], gq, yq), (leaves[1], leaves[3], gk, yk)):
        want, tol = ref.norm_rope(x.detach(), g.detach(), t["cos"], t["sin"], None, 1e-6, il)
        ref.inside(y.detach(), want, tol, "y")
        (dx, tx), (dg, tg) = ref.norm_rope_bwd(dy, x.detach(), g.detach(), t["cos"], t["sin"], None, 1e-6, il)
        ref.inside(x.grad, dx, tx, "dx")
        ref.inside(g.grad, dg, (60 + 40 * x.shape[2]) * tg, "dgamma")
    with torch.no_grad():  # parameters as they are, where nothing is recorded
        a, b = sg.sagesla_qk_norm_rope(*leaves, t["cos"], t["sin"], interleaved=il)
    assert torch.equal(a, yq) and torch.equal(b, yk) and not a.requires_grad
