"""Host-side checks of the layers around the W4A4 ones: sizes, strides,
pointers and enums are rejected before a GPU is touched."""
import ctypes

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import block as oblock
from synth import rng

P = 1 << 20  # aligned fake device address, never dereferenced
NO_GPU = not __import__("torch").cuda.is_available()


@pytest.fixture(scope="module")
def so():
    from bit_diffusion_transformer_nvfp4_b200 import build
    build.build()
    import bit_diffusion_transformer_nvfp4_b200 as w
    return w.lib()


def test_rows_arguments(so):
    def call(X=P, rows=4, cols=256, ldx=256, codes=P, ldo=256, scales=P):
        return so.fp8_quantize_rows(X, rows, cols, ldx, codes, ldo, scales, None)
    if NO_GPU:
        assert call() == -4
        assert call(cols=32768, ldx=32768, ldo=32768) == -4
    assert call(cols=32776, ldx=32776, ldo=32776) == -2
    assert call(cols=250) == -2
    assert call(cols=0) == -2
    assert call(ldx=248) == -2
    assert call(ldx=260) == -2
    assert call(ldo=248) == -2
    assert call(rows=-1) == -2
    assert call(X=None) == -1
    assert call(codes=None) == -1
    assert call(scales=None) == -1
    assert call(X=P + 8) == -3
    assert call(codes=P + 8) == -3
    assert call(scales=P + 2) == -3
    assert call(rows=0, X=None, codes=None, scales=None) == 0


def test_norm_arguments(so):
    def call(X=P, rows=4, cols=256, ldx=256, R=None, ldr=0, w=None, eps=1e-6, hidden=None, ldh=0, normed=None, ldn=0,
             codes=P, ldo=256, scales=P):
        return so.rmsnorm_fp8(X, rows, cols, ldx, R, ldr, w, ctypes.c_float(eps), hidden, ldh, normed, ldn, codes, ldo,
                              scales, None)
    if NO_GPU:
        assert call() == -4
        assert call(codes=None, scales=None, ldo=0, normed=P, ldn=256) == -4
    assert call(R=P, ldr=248) == -2
    assert call(hidden=P, ldh=250) == -2
    assert call(normed=P, ldn=0) == -2
    assert call(codes=None, scales=None) == -1
    assert call(scales=None) == -1
    assert call(eps=-1.0) == -8
    assert call(eps=float("nan")) == -8
    assert call(eps=float("inf")) == -8
    assert call(w=P + 4) == -3
    assert call(R=P + 4, ldr=256) == -3
    assert call(hidden=P + 4, ldh=256) == -3
    assert call(rows=0, X=None, codes=None, scales=None) == 0


def test_gemm_arguments(so):
    def call(A=P, lda=256, s_a=P, per_row=1, M=8, N=64, K=256, W=P, ldw=256, s_w=P, bias=None, epi=0, R=None, ldr=0,
             Y=P, ldy=64):
        return so.fp8_gemm(A, lda, s_a, per_row, M, N, K, W, ldw, s_w, bias, epi, R, ldr, Y, ldy, None)
    if NO_GPU:
        assert call() == -4
        assert call(K=16, lda=16, ldw=16) == -4
        assert call(M=1 << 20, R=P, ldr=64) == -4
    assert call(K=250) == -2
    assert call(K=0) == -2
    assert call(K=(1 << 20) + 16, lda=1 << 21, ldw=1 << 21) == -2
    assert call(N=60) == -2
    assert call(N=0) == -2
    assert call(lda=240) == -2
    assert call(ldw=264) == -2
    assert call(ldy=56) == -2
    assert call(R=P, ldr=56) == -2
    assert call(M=-1) == -2
    assert call(M=1 << 30, N=1 << 30, ldy=1 << 30) == -2
    assert call(epi=2) == -8
    assert call(per_row=2) == -8
    for name in ("A", "s_a", "W", "s_w", "Y"):
        assert call(**{name: None}) == -1, name
    for name in ("A", "W", "s_w", "Y", "bias"):
        assert call(**{name: P + 8}) == -3, name
    assert call(R=P + 8, ldr=64) == -3
    assert call(s_a=P + 2) == -3
    assert call(M=0, A=None, s_a=None, W=None, s_w=None, Y=None) == 0


def test_cross_attention_arguments(so):
    def call(Q=P, ldq=256, K=P, ldk=128, V=P, ldv=128, batch=2, kv_batch=2, Sq=10, Skv=20, heads=4, kv_heads=2, d=64,
             kv_len=None, mask=None, ldm=0, c=0.125, O=P, ldo=256):
        return so.cross_attention_bf16(Q, ldq, K, ldk, V, ldv, batch, kv_batch, Sq, Skv, heads, kv_heads, d, kv_len,
                                       mask, ldm, ctypes.c_float(c), O, ldo, None)
    if NO_GPU:
        assert call() == -4
        assert call(kv_batch=1) == -4
        assert call(mask=P + 1, ldm=21) == -4
        assert call(Skv=0, Q=None, K=None, V=None) == -4
    assert call(d=4) == -2
    assert call(d=60) == -2
    assert call(d=136, ldq=1024, ldk=1024, ldv=1024, ldo=1024) == -2
    assert call(kv_heads=3) == -2
    assert call(kv_heads=0) == -2
    assert call(kv_batch=3) == -2
    assert call(ldq=248) == -2
    assert call(ldk=120) == -2
    assert call(ldv=132) == -2
    assert call(ldo=128) == -2
    assert call(Sq=(1 << 24) + 1) == -2
    assert call(Skv=(1 << 24) + 1) == -2
    assert call(Sq=1 << 24, ldq=1 << 20) == -2     # the batch stride leaves its field
    assert call(mask=P, ldm=19) == -2
    assert call(batch=40000, kv_batch=1, heads=40000, kv_heads=1, d=8, Sq=1, ldq=320000, ldo=320000) == -2  # tile count
    for c in (0.0, -1.0, float("nan"), float("inf"), 2.5e38):
        assert call(c=c) == -8
    for name in ("Q", "K", "V", "O"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 8}) == -3, name
    assert call(kv_len=P + 2) == -3
    assert call(batch=0, kv_batch=1, Q=None, K=None, V=None, O=None) == 0
    assert call(Sq=0, Q=None, K=None, V=None, O=None) == 0


def test_python_wrappers_refuse_what_the_kernels_would_misread():
    import torch
    import bit_diffusion_transformer_nvfp4_b200 as w4
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        w4.quantize_rows_fp8(x)                                 # not bf16
    with pytest.raises(ValueError):
        w4.quantize_rows_fp8(x.bfloat16())                      # not on a GPU
    with pytest.raises(ValueError):
        w4.rms_norm_fp8(x.bfloat16().reshape(2, 2, 64))         # not a matrix
    with pytest.raises(ValueError):
        w4.cross_attention(x.bfloat16(), x.bfloat16(), x.bfloat16(), heads=1)


def test_oracle_row_codes_are_the_tensor_quantisers():
    x = rng(1).standard_normal((3, 40)).astype(np.float32)
    codes, s = oblock.quantize_rows(x)
    for i in range(3):
        c, si = oatt.fp8_quantize(x[i:i + 1])
        assert np.array_equal(codes[i:i + 1], c) and s[i] == si


def test_oracle_norm_and_linear_by_hand():
    h, y = oblock.rms_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), eps=0.0)
    np.testing.assert_allclose(y, np.array([[3.0, 8.0]]) / np.sqrt(12.5))
    np.testing.assert_allclose(h, [[3.0, 4.0]])
    y = oblock.linear(np.array([[1.0, 2.0]]), [2.0], np.array([[1.0, 1.0], [0.5, -1.0]]), [1.0, 3.0],
                      bias=[1.0, 0.0], residual=np.array([[10.0, 20.0]]))
    np.testing.assert_allclose(y, [[2 * 3 + 1 + 10, 2 * -1.5 * 3 + 20]])


def test_oracle_attention_against_the_square_one_and_by_hand():
    g = rng(2)
    q, k, v = (g.standard_normal((6, 256)) for _ in range(3))
    o, _ = oblock.cross_attention(q, k, v, 2, 2, 1, 1)
    np.testing.assert_allclose(o, oatt.attention(q, k, v, 2), rtol=1e-12, atol=1e-13)
    # one key: its value, whatever the score; no key: zero
    o, a = oblock.cross_attention(q, k[:3], v[:3], 2, 2, 2, 1, kv_len=[1])
    np.testing.assert_allclose(o, np.repeat(v[:1], 6, axis=0))
    np.testing.assert_allclose(a, np.abs(o))
    assert not oblock.cross_attention(q, k, v, 2, 2, 1, 1, kv_len=[0])[0].any()
    # a shared head and a mask: the same as the head repeated and the keys left out
    keep = np.array([True, False, True, True, False, True])
    o, _ = oblock.cross_attention(q, k[:, :128], v[:, :128], 2, 1, 1, 1, key_mask=keep[None])
    kk, vv = np.tile(k[keep, :128], (1, 2)), np.tile(v[keep, :128], (1, 2))
    np.testing.assert_allclose(o, oblock.cross_attention(q, kk, vv, 2, 2, 1, 1)[0], rtol=1e-12)
