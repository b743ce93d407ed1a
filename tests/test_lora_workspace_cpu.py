"""A workspace is asked for only where the kernel that uses it runs. The host code on the fake
CUDA runtime, which has no memory pool: a call that takes memory from one fails there."""
import pytest

from tests.test_host_code_dispatch_cpu import BF16, BUF, BUF2, ODD, ODD2, launched, lib, library, lora  # noqa: F401 (fixtures)

CUDA_ERROR, WORKSPACE = -4, -3


@pytest.mark.parametrize("M", [1537, 5000, 100000])
@pytest.mark.parametrize("kw", [dict(K=513), dict(N=514), dict(r=3), dict(r=12), dict(r=100, N=514), dict(x=ODD), dict(out=ODD2),
                                dict(add=ODD)], ids=str)
def test_rows_that_no_order_is_made_of_take_none(lib, M, kw):  # noqa: F811
    assert lora(lib, M, ws=None, **kw) == 0
    assert all("lora_few" in name for _, name, *_ in launched(lib))
    if not {"x", "out", "add"} & set(kw):  # (addresses, which the size does not know)
        sizes = dict(K=512, N=512, r=16) | kw
        assert lib.moe_w4a16_lora_workspace_size(M, sizes["K"], sizes["N"], sizes["r"], 4) == 0
    # one that is too small for an order is not refused either
    assert lib.moe_w4a16_lora(kw.get("x", BUF), kw.get("K", 512), BUF, BUF, BUF, BUF, kw.get("add", BUF), BF16, kw.get("out", BUF2), BF16, M,
                              kw.get("K", 512), kw.get("N", 512), kw.get("r", 16), 4, BUF, 1, None) == 0


@pytest.mark.parametrize("M", [1537, 5000])
def test_an_order_takes_what_the_size_says(lib, M):  # noqa: F811
    need = lib.moe_w4a16_lora_workspace_size(M, 512, 512, 16, 4)
    assert need >= 4 * M and lora(lib, M, ws=None) == CUDA_ERROR

    def given(size):
        return lib.moe_w4a16_lora(BUF, 512, BUF, BUF, BUF, BUF, BUF, BF16, BUF2, BF16, M, 512, 512, 16, 4, BUF, size, None)

    assert given(need) == 0 and given(need - 1) == WORKSPACE
    assert lora(lib, 1536, ws=None) == 0 and lib.moe_w4a16_lora_workspace_size(1536, 512, 512, 16, 4) == 0
