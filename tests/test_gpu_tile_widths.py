"""The products by expert at sizes that take tiles of each width (64, 128 and 256 along the narrow extent; in 8 bits also
of 128 by 128), among them calls with more tiles than SMs hold at once and tiles that end after one row or one column."""
import pytest
import torch

from masking_tm_affine_gb300 import tm
from test_gpu_e4m3 import Case as Case8
from test_gpu_experts import Case

pytestmark = pytest.mark.gpu

# rows of each expert, N, K
SHAPES = [([900, 800, 333, 5, 0, 700], 1000, 330), ([900, 800, 333, 5, 0, 700], 500, 330), ([129] * 50, 200, 72), ([65] * 60, 256, 136),
          ([33] * 70, 130, 264), ([257] * 48, 100, 200), ([64, 65, 63, 1, 129, 128, 127], 257, 129), ([3000], 264, 1000),
          ([1025], 1025, 512), ([255, 257, 513], 72, 1032), ([2000, 1, 2000], 260, 64), ([127, 0, 0, 300, 40, 1], 1000, 136),
          ([100] * 20, 1100, 200), ([34, 128, 0, 129, 1], 136, 1160)]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_16_bits(cuda, counts, N, K, out):
    Case(counts, N, K, "bf16", seed=N + K, ints=True, behind=3, gap=1).check_all(out)
    Case(counts, N, K, "bf16", seed=N + K).check_all(out)


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("out,group", [("bf16", 128), ("f32", 0)])
def test_8_bits(cuda, counts, N, K, out, group):
    for ints in (True, False):
        c = Case8(counts, N, K, group, seed=N, ints=ints, behind=3)
        for ldc in (N, N + 3):
            y = c.run(out, ldc)
            tm.tm_check()
            c.check(y, out)


@pytest.mark.parametrize("counts", [[700], [300, 400], [150] * 4])
@pytest.mark.parametrize("K", [2040, 2048, 2200])
def test_sums_on_both_sides_of_a_rule(cuda, counts, K):
    # long sums over few tiles go to the kernel that cuts them: the results are the definition's either way
    Case(counts, 256, K, "f16", seed=K, ints=True).check_all("f32")
    c = Case8(counts, 256, K, 128, seed=K, ints=True)
    y, again = c.run("f32"), c.run("f32")
    tm.tm_check()
    c.check(y, "f32")
    assert torch.equal(y, again)
