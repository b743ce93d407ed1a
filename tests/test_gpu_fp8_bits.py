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


@pytest.mark.parametrize("lo,hi,u", [(-1, 1, 1.0), (-20, -10, 1e5), (-87, -60, 1e30), (20, 87, 1.0)])
def test_swiglu_error_over_the_range_of_gates(lo, hi, u):
    # The scale is amax / 448 of one h: |error| <= 2^-21 + |g| 2^-23 of it, the stated bound
    # (the largest h of a block is within that of its computed one), and its own rounding, 2^-24;
    # the values are within half an e4m3 step of h / s more.
    rng = np.random.default_rng(int(hi) + 100)
    M, N = 300, 256
    g = rng.uniform(lo, hi, (M, N)).astype(np.float32)
    x = np.concatenate([g, (rng.uniform(0.5, 1, (M, N)) * u).astype(np.float32)], 1)
    q, s = fp8.swiglu_quantize(torch.from_numpy(x).cuda())
    h = oo.silu(x[:, :N]) * x[:, N:].astype(np.float64)
    rel = 2.0 ** -21 + max(abs(lo), abs(hi)) * 2.0 ** -23 + 2.0 ** -24
    want = np.abs(h).reshape(M, 2, 128).max(2) / 448.0
    np.testing.assert_allclose(s.cpu().numpy().astype(np.float64), want, rtol=rel)
    sp = np.repeat(s.cpu().numpy().astype(np.float64), 128, 1)
    got = oo.e4m3_values(q.view(torch.uint8).cpu().numpy()) * sp
    assert (np.abs(got - h) <= (2.0 ** -4 + 2 * rel) * np.abs(h) + 2.0 ** -10 * sp).all()


def test_swiglu_far_below_is_zero():
    g = torch.tensor([-87.4, -88.5, -100.0, -1e4, -3e38] * 32, device="cuda")
    q, s = fp8.swiglu_quantize(torch.cat([g, torch.ones_like(g)])[None, :])
    assert not (q.view(torch.uint8) & 0x7F).any() and (s == 2.0 ** -126).all()
