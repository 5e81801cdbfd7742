"""GPU parity of every kernel of the FP8 linear layer and both forms of the
cross attention, at sizes that are known (on the CPU) to reach them, against
64-bit references.

Linear: the codes are 0, +-0.5, +-1 and +-2, so every partial sum is exact in
fp32 on the GPU and in the reference (products of whole numbers up to 16, sums
below 2^24); what is left is four fp32 operations, the hardware exponential of
the GELU (2^-20 of its argument's terms) and the output's bf16 rounding, 2^-8.
Attention: as for the ordinary cases (weights rounded to bf16, 2^-8, an
exponential good to 2^-13, the output's own 2^-8).
"""
import math

import numpy as np
import pytest

from helpers import from_dev_bf16, to_dev_bf16, to_dev_f32
from oracle import block as oblock
from plan_shapes import ATTENTION, PRODUCTS
from synth import bf16_round, rng

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
CODES = np.array([0x00, 0x30, 0x38, 0x40, 0xB0, 0xB8, 0xC0], np.uint8)  # 0, +-0.5, +-1, +-2


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_diffusion_transformer_nvfp4_b200 as w
    w.lib()
    return w


@pytest.fixture(autouse=True)
def clean_status(w4):
    import torch
    yield
    torch.cuda.synchronize()
    assert w4.w4a4_device_status() == 0


def doubled(codes):
    """Twice the codes' values, whole numbers, in fp32."""
    return (2 * oblock.decode(codes)).astype(np.float32)


@pytest.mark.parametrize("M,N,K", [p[:3] for p in PRODUCTS])
def test_linear_of_every_kernel(w4, M, N, K):
    """All four of GELU or none, with and without residual, in turn with and
    without bias; rows and columns behind the output stay."""
    import torch
    g = rng(M * 5 + N + K)
    a, w = CODES[g.integers(0, 7, (M, K))], CODES[g.integers(0, 7, (N, K))]
    s_a = np.exp(0.5 * g.standard_normal(M)).astype(np.float32)
    s_w = (np.exp(0.5 * g.standard_normal(N)) / math.sqrt(K)).astype(np.float32)
    b = bf16_round(g.standard_normal(N).astype(np.float32))
    r = bf16_round(g.standard_normal((M, N)).astype(np.float32))
    t = (doubled(a) @ doubled(w).T).astype(np.float64) / 4 * s_a[:, None].astype(np.float64) * s_w[None, :]
    A = w4.Fp8Rows(torch.from_numpy(a).cuda(), to_dev_f32(s_a))
    codes, scales, B, R = torch.from_numpy(w).cuda(), to_dev_f32(s_w), to_dev_bf16(b), to_dev_bf16(r)
    for gelu, residual, bias in ((False, False, True), (True, False, False), (False, True, False), (True, True, True)):
        want = t + b if bias else t.copy()
        size = np.abs(t) + (np.abs(b) if bias else 0.0) + (np.abs(r) if residual else 0.0)
        if gelu:
            want = oblock.gelu_tanh(want)
        if residual:
            want = want + r
        base = torch.full((M + 1, N + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        w4.linear_fp8(A, w4.PackedWeightFp8(codes, scales, B if bias else None), residual=R if residual else None,
                      activation=w4.EPI_GELU_TANH if gelu else w4.EPI_NONE, Y=base[:M, :N])
        err = np.abs(from_dev_bf16(base[:M, :N].contiguous()) - want)
        bound = BF16 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -133
        assert np.all(err <= bound), (gelu, residual, np.max(err / bound))
        assert bool((base[M:] == 3.0).all()) and bool((base[:, N:] == 3.0).all())


@pytest.mark.parametrize("batch,kv_batch,sq,sk,heads,kv_heads,d", [a[:7] for a in ATTENTION])
@pytest.mark.parametrize("what", ["all", "length", "mask", "both", "none"])
def test_cross_attention_of_shared_states(w4, batch, kv_batch, sq, sk, heads, kv_heads, d, what):
    """Every sequence attends to the same keys, under one length and one mask."""
    import torch
    g = rng(sq + sk + d)
    q = bf16_round((1.5 * g.standard_normal((batch * sq, heads * d))).astype(np.float32))
    k, v = (bf16_round(g.standard_normal((kv_batch * sk, kv_heads * d)).astype(np.float32)) for _ in range(2))
    n = np.array([sk - 77], np.int32) if what in ("length", "both") else None
    if what == "none":
        n = np.array([0], np.int32)
    mask = g.random((1, sk)) < 0.6 if what in ("mask", "both") else None
    kd, vd = k.copy(), v.copy()
    gone = np.zeros(sk, bool)
    if n is not None:
        gone |= np.arange(sk) >= n[0]
    if mask is not None:
        mask[0, 128:256] = False
        gone |= ~mask[0]
    kd[gone], vd[gone] = np.nan, np.inf
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(vd), heads=heads, kv_heads=kv_heads, batch=batch,
                           kv_batch=kv_batch, kv_len=None if n is None else torch.from_numpy(n).cuda(),
                           key_mask=None if mask is None else torch.from_numpy(mask).cuda())
    want, avg = oblock.cross_attention(q, k, v, heads, kv_heads, batch, kv_batch, kv_len=n, key_mask=mask)
    err = np.abs(from_dev_bf16(O) - want)
    bound = BF16 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * avg
    assert np.all(err <= bound)


def test_norm_is_what_a_w4a4_layer_reads(w4):
    """A W4A4 layer behind the norm, against the same layer behind the oracle's
    norm in bf16.

    The kernel's norm is off by at most 2^-18 before its rounding, so it can
    differ from the oracle's bf16 only where that lies within 2^-18 of a
    border between values 2^-8 apart: fewer than one element in 256, by one
    step.  Such an element moves its code by one step at most and, as the
    largest of its block, the scale of 16: with half of the value each, the
    outputs are off by less than sqrt(16 / 256) / 2 = 1/8 of their norm.  A norm
    without its weight (here from 0.1 to 10) or with a wrong row factor is off
    by about all of it.
    """
    import torch
    g = rng(57)
    x = bf16_round((g.standard_normal((300, 512)) * np.exp(g.standard_normal((300, 1)))).astype(np.float32))
    r = bf16_round(g.standard_normal((300, 512)).astype(np.float32))
    nw = bf16_round((10.0 ** g.uniform(-1, 1, 512)).astype(np.float32))
    normed = torch.empty(300, 512, dtype=torch.bfloat16, device="cuda")
    w4.rms_norm_fp8(to_dev_bf16(x), to_dev_bf16(nw), residual=to_dev_bf16(r), normed=normed)
    want = bf16_round(oblock.rms_norm(x, r, nw)[1].astype(np.float32))
    off = from_dev_bf16(normed) != want
    assert np.mean(off) < 1 / 256
    np.testing.assert_allclose(from_dev_bf16(normed), want, rtol=2 * BF16)
    w = w4.pack_weight(to_dev_f32((0.05 * g.standard_normal((256, 512))).astype(np.float32)))
    y = from_dev_bf16(w4.gemm(w4.quantize_act(normed), w)).astype(np.float64)
    ref = from_dev_bf16(w4.gemm(w4.quantize_act(to_dev_bf16(want)), w)).astype(np.float64)
    plain = from_dev_bf16(w4.gemm(w4.quantize_act(to_dev_bf16(bf16_round((x + r).astype(np.float32)))), w))
    assert np.linalg.norm(y - ref) <= np.linalg.norm(ref) / 8
    assert np.linalg.norm(plain - ref) >= np.linalg.norm(ref) / 2  # (the test can tell)
