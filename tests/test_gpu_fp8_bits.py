"""The bytes that the quantisers write, signs of zeros among them, and SwiGLU's stated error."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8
from oracle import ops_oracle as oo
from tests.test_gpu_fp8 import _built, np64, rand  # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


def nearest_bytes(x, s):
    """e4m3 bytes of x / s, the quotient a 32-bit number; a zero keeps its sign."""
    quotient = (x / s).astype(np.float32)
    v = oo.e4m3_round(quotient.astype(np.float64))
    grid = oo.e4m3_values(np.arange(127, dtype=np.uint8))
    return (np.searchsorted(grid, np.abs(v)) | np.where(np.signbit(quotient), 0x80, 0)).astype(np.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** 60, 2.0 ** -120, 2.0 ** 110])
@pytest.mark.parametrize("K", [512, 300])
def test_bytes_and_signs_of_zeros(dtype, scale, K):
    x = rand((200, K), K, 1.0, torch.float32)
    x[:, ::5] = -0.0
    x[:, 1::5] = 0.0
    x[:, 2::5] *= 1e-4  # (rounds to a zero of its sign, in part)
    x[7], x[8] = -0.0, 0.0
    x = (x * scale).to(dtype)
    for call, rows in ((fp8.quantize, 1), (fp8.quantize_weight, 128)):
        q, s = call(x)
        s64 = np.repeat(np.repeat(s.cpu().numpy().astype(np.float64), rows, 0)[:200], 128, 1)[:, :K]
        np.testing.assert_array_equal(q.view(torch.uint8).cpu().numpy(), nearest_bytes(np64(x), s64))
