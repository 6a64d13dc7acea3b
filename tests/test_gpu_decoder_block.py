"""The example that runs the block's operators together (examples/decoder_block.py)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("decoder_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


# The two ways see the same tokens, so they differ by fp32 roundings of the products (2^-20 of an
# output of about 1) and, where such a rounding carries a key or value over the border between
# two codes, by one step of one dimension: a 15th of a vector's range (about 5 for 64 normal
# numbers) in one of the lens >= 7 tokens averaged, a third, through a weight of 1/sqrt(512) in
# the output product: below 0.01 each.  Few such borders are met: 0.05 leaves room for several.
@pytest.mark.parametrize("prompts,steps,Hq,Hkv,D", [((5, 130, 1, 64), 6, 8, 2, 64), ((31,), 1, 4, 4, 128),
                                                    ((300, 17), 3, 16, 1, 64)])
def test_served_tokens_equal_their_prompt(block, prompts, steps, Hq, Hkv, D):
    graph, whole = block.serve(prompts=prompts, steps=steps, Hq=Hq, Hkv=Hkv, D=D)
    assert graph.shape == whole.shape == (len(prompts), 256)
    assert torch.isfinite(whole).all()
    assert float((graph - whole).abs().max()) <= 0.05
    assert float(whole.abs().max()) > 0.1


# The quotient's own errors: fp32 losses rounded at 2^-22 of sums of about sqrt(T H D) products
# of size 1, over 2 e = 2^-6, and the third derivative's e^2 / 6: together below 1e-3 of
# sqrt(T E).  sqrt(37 * 256) is 97, the size of the derivative itself.
@pytest.mark.parametrize("T,E,H,D", [(37, 256, 4, 64), (1, 64, 1, 128), (130, 96, 3, 64)])
def test_gradient_equals_difference(block, T, E, H, D):
    slope, quotient = block.train(T=T, E=E, H=H, D=D)
    assert abs(slope - quotient) <= 1e-2 * (T * E) ** 0.5
