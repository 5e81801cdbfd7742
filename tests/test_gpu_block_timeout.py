"""Waits that run out in the FP8 linear layer and the cross attention: the call
ends by itself, the status word tells, and the next call is right.

Nothing is stuck: with the wait bound at its smallest (10^6 cycles, about 0.5 ms)
the epilogue's wait for a long tile, which is legitimate and takes some
milliseconds, is what gives up.  Every wait is bounded, and the kernels drain
their copies and products before they return.
"""
import pytest

pytestmark = pytest.mark.gpu

TIMEOUT_STATUS = -7       # W4A4_ERR_DEVICE_TIMEOUT
SHORT_BOUND = 1_000_000   # SM cycles


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_diffusion_transformer_nvfp4_b200 as w
    w.lib()
    return w


def runs_out_and_recovers(w4, call, want):
    import torch
    torch.cuda.synchronize()
    assert w4.w4a4_device_status(reset=True) == 0
    w4.w4a4_set_wait_bound(SHORT_BOUND)
    try:
        call()
        torch.cuda.synchronize()
        assert w4.w4a4_last_error() == TIMEOUT_STATUS
        assert w4.w4a4_device_status(reset=True) == TIMEOUT_STATUS
    finally:
        w4.w4a4_set_wait_bound(0)
    out = call()
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0
    assert bool((out.float() == want).all())


def test_cross_attention(w4):
    """148 work tiles of 4096 key tiles each, some 7 ms."""
    import torch
    keys, rows = 1 << 19, 256 * 37
    k = torch.zeros(keys, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 2.0)
    q = torch.zeros(rows, 4 * 128, dtype=torch.bfloat16, device="cuda")
    runs_out_and_recovers(w4, lambda: w4.cross_attention(q, k, v, heads=4, kv_heads=1), 2.0)


@pytest.mark.parametrize("residual", [False, True])
def test_linear_of_many_rows(w4, residual):
    """Two or three tiles a CTA pair of 8192 K steps each, some 3 ms a tile."""
    import torch
    M, N, K = 2048, 5120, 1 << 20
    a = w4.Fp8Rows(torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.ones(M, device="cuda"))
    w = w4.PackedWeightFp8(torch.zeros(N, K, dtype=torch.uint8, device="cuda"), torch.ones(N, device="cuda"),
                           torch.full((N,), 0.5, dtype=torch.bfloat16, device="cuda"))
    r = torch.full((M, N), 1.5, dtype=torch.bfloat16, device="cuda") if residual else None
    runs_out_and_recovers(w4, lambda: w4.linear_fp8(a, w, residual=r), 2.0 if residual else 0.5)


def test_linear_of_few_rows(w4):
    """A weight of 20 GB past one token, some 3 ms."""
    import torch
    N, K = 148 * 128, 1 << 20
    a = w4.Fp8Rows(torch.zeros(1, K, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"))
    w = w4.PackedWeightFp8(torch.zeros(N, K, dtype=torch.uint8, device="cuda"), torch.ones(N, device="cuda"),
                           torch.full((N,), 0.5, dtype=torch.bfloat16, device="cuda"))
    runs_out_and_recovers(w4, lambda: w4.linear_fp8(a, w), 0.5)
