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
