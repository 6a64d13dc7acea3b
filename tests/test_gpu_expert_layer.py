"""The example that runs the routed layer (examples/expert_layer.py), served in 8 bits and differentiated in 16."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


# The rows' and matrices' 8 bits round each value by at most 2^-4 of itself; the layer is two products of
# two such operands, whose errors add in their 2-norm to at most 4 * 2^-4 (the activation's slope is below 1.1).
# index_add_ adds a token's two answers in either order: a + b is b + a.
@pytest.mark.parametrize("T,H,F,E,k", [(24, 512, 640, 8, 2), (1, 128, 128, 4, 1), (300, 256, 1000, 3, 2), (70, 384, 208, 33, 2)])
def test_served(layer, T, H, F, E, k):
    for replayed, direct, exact in layer.serve(T=T, H=H, F=F, E=E, k=k):
        assert torch.equal(replayed, direct)
        assert torch.isfinite(direct).all()
        assert float((direct.double() - exact).norm()) <= 1.1 * 4 * 2.0 ** -4 * float(exact.norm())


# About ten roundings to bf16 (2^-9 of a value each) lie between the leaves and a gradient, each of
# the size of what it rounds, whose errors add in the 2-norm: 16 * 2^-9.
@pytest.mark.parametrize("T,H,F,E,k", [(150, 256, 384, 6, 2), (1, 64, 64, 2, 1), (700, 128, 200, 3, 1)])
def test_gradients_and_their_clipping(layer, T, H, F, E, k):
    for max_norm in (0.5, 1e9):
        grads, total, wide = layer.train(T=T, H=H, F=F, E=E, k=k, max_norm=max_norm)
        want = float(torch.stack([w.norm() for w in wide]).norm())
        assert abs(float(total) - want) <= 16 * 2.0 ** -9 * want
        factor = min(1.0, max_norm / (float(total) + 1e-6))
        for g, w in zip(grads, wide):
            assert float((g.double() - factor * w).norm()) <= 16 * 2.0 ** -9 * factor * float(w.norm())


def test_second_derivatives_are_refused(layer):
    # a gradient of a gradient has terms that these functions do not make: an error, not a wrong number
    x = torch.randn(6, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(2, 64, 64, device="cuda").bfloat16().requires_grad_()
    n = torch.ones(64, device="cuda").bfloat16().requires_grad_()
    starts = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    for y, leaves in ((layer.Experts.apply(x, w, starts), (x, w)), (layer.Norm.apply(x, n), (x, n))):
        with pytest.raises(RuntimeError):
            first = torch.autograd.grad((y.float() ** 2).sum(), leaves, create_graph=True)
            penalty = sum(g.float().pow(2).sum() for g in first) + sum(t.float().pow(2).sum() for t in leaves)
            torch.autograd.grad(penalty, leaves)


def test_only_the_gradients_that_are_asked_for(layer, monkeypatch):
    x, w = torch.randn(6, 64, device="cuda").bfloat16(), torch.randn(2, 64, 64, device="cuda").bfloat16()
    starts = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    made, call = [], layer.tm.tm_gemm_experts_bwd

    def spy(*a):
        made.append((a[6] is not None, a[8] is not None))
        return call(*a)
    monkeypatch.setattr(layer.tm, "tm_gemm_experts_bwd", spy)
    grads = []
    for rows, weights in ((True, True), (True, False), (False, True)):
        leaves = [t.clone().requires_grad_(need) for t, need in ((x, rows), (w, weights))]
        layer.Experts.apply(*leaves, starts).float().sum().backward()
        grads.append([t.grad for t in leaves])
        assert made[-1] == (rows, weights)
    assert grads[1][1] is None and grads[2][0] is None
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[2][1])
    made.clear()
    norm, back = [], layer.tm.tm_rmsnorm_bwd
    monkeypatch.setattr(layer.tm, "tm_rmsnorm_bwd", lambda *a: (norm.append(a[10] is not None), back(*a))[1])
    for weights in (True, False):
        g, n = x.clone().requires_grad_(), torch.ones(64, device="cuda").bfloat16().requires_grad_(weights)
        layer.Norm.apply(g, n).float().sum().backward()
        assert norm[-1] is weights and (n.grad is not None) is weights
        grads.append(g.grad)
    assert torch.equal(grads[-1], grads[-2])
