"""The forms of the 8-bit products at sizes that reach each of them, against the float64
definitions. Tolerances as in test_gpu_fp8.py."""
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8
from tests.test_gpu_fp8 import _built, check_product, operands, rand  # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


def test_launches_back_to_back_keep_their_results():
    # (a product's CTAs hand their shared memory to the next launch's while others still run:
    # pairs of CTAs, clusters and single ones in turn, each right every time)
    shapes = [(2048, 1024, 384), (4, 512, 2048), (1500, 2048, 128), (40, 640, 1024), (100, 256, 1024), (700, 4096, 256)]
    ops = [operands(*shape, seed=i) for i, shape in enumerate(shapes)]
    first = [fp8.matmul(*o) for o in ops]
    for out, o in zip(first, ops):
        check_product(out, *o)
    for _ in range(40):
        outs = [fp8.matmul(*o) for o in ops]
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    assert fp8.status() == 0
