"""Nothing of the first product's sums is lost on their way into the second one.

The values are whole numbers of which every sum is below 2^23 whatever its order: x and a up
to 127 over at most 512 columns, so that sum |a| |x| < 2^23, and three entries of a row of b,
1 or -1, where the sums of a[l] x stay below 2^21.3. All products and sums are then exact in 24
bits, whether a matrix unit rounds or cuts off, and the result is the whole number rounded once
to the output's type: no tolerance. The sums have more than 16 bits, and addends that cancel
the adapter's term show the last of them."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import lora
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def problem(M, K, N, r, L, seed):
    rng = np.random.default_rng(seed)
    most = 127 if K <= 256 else 90
    x, a = rng.integers(0, most + 1, (M, K)), rng.integers(0, most + 1, (L, r, K))
    b = np.zeros((L, N, r), np.int64)
    for _ in range(min(3, r)):  # (two may fall on one entry: the later one stands)
        at = rng.integers(0, r, (L, N, 1))
        np.put_along_axis(b, at, rng.choice([-1, 1], (L, N, 1)), 2)
    index = rng.integers(-1, L, M).astype(np.int32)
    v = np.einsum("mk,mrk->mr", x, a[np.maximum(index, 0)])
    term = np.einsum("mr,mnr->mn", v, b[np.maximum(index, 0)]) * (index >= 0)[:, None]
    assert v.max() < 2 ** 21.3 and v.max() > 2 ** 18 and K * most * most < 2 ** 23 and np.abs(term).max() < 2 ** 23
    return x, a, b, index, term, rng


SIZES = [(1, 256, 40, 8, 1), (20, 512, 136, 16, 3), (70, 264, 72, 64, 8), (300, 512, 128, 128, 2), (700, 256, 64, 32, 5),
         (40, 257, 33, 3, 4), (900, 250, 41, 12, 3),                                  # (value by value, several launches)
         (800, 512, 136, 16, 3), (1200, 256, 264, 64, 2), (1000, 264, 128, 128, 4), (1600, 512, 128, 24, 9), (2500, 256, 136, 72, 3)]


@pytest.mark.parametrize("M,K,N,r,L", SIZES)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_sums_enter_the_second_product_whole(M, K, N, r, L, out_type):
    x, a, b, index, term, rng = problem(M, K, N, r, L, M + r)
    t = lambda v: dev(v.astype(np.float32)).to(BF16)  # noqa: E731
    near = rng.integers(-100, 101, term.shape) - term
    for add in (None, dev(near.astype(np.float32)), t(-term)):
        plus = 0 if add is None else add.double().cpu().numpy().astype(np.int64)
        want = torch.from_numpy((term + plus).astype(np.float32)).to(out_type)
        got = lora.apply(t(x), t(a), t(b), dev(index), add=add, out_dtype=out_type).cpu()
        assert torch.equal(got, want), ((got.double() - want.double()).abs().max(), (got != want).sum(), got.numel())
