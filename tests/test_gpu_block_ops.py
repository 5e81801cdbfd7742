"""GPU parity of the layers around the W4A4 ones: row codes, RMS norm, the FP8
linear layer and cross attention, against the 64-bit oracle.

Tolerances count roundings (half a step of bf16 is 2^-8 of the value, of E4M3
2^-4 or 2^-10 of the scale below its normal range):

* row codes: the oracle repeats the fp32 steps, bytes and scales are equal.
* norm: the row factor sums up to 2^15 squares in fp32 along chains of at most
  32 + 10 additions (half of that error after the root) with six more
  operations behind it: below 32 x 2^-24 = 2^-19, doubled.  A code is off by half
  its step, hidden and normed by half a bf16 step.
* linear: with integer codes every partial sum is exact in fp32, so what is
  left is four fp32 operations, the hardware exponential of the GELU (2^-20)
  and the bf16 rounding.  On random codes the sum itself is rounded too; the
  norm of the error stays below one bf16 half-step of the norm of the result.
* attention: each weight is rounded to bf16 (2^-8) after an exponential good to
  2^-13 (its polynomial part: 7.5e-5), so an output is off by (2^-8 + 2^-12) times
  the same average over |v|, the factor's 2^-12 covering the fp32 scores too
  (|c s| <= 64 here: 64 x 2^-24 each), plus its own bf16 rounding.
"""
import math

import numpy as np
import pytest

from helpers import from_dev_bf16, to_dev_bf16, to_dev_f32
from oracle import block as oblock
from synth import bf16_round, rng

pytestmark = pytest.mark.gpu

BF16, E4M3 = 2.0 ** -8, 2.0 ** -4
NORM = 2.0 ** -18


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


def values(g, rows, cols, spread=1.0):
    return bf16_round((g.standard_normal((rows, cols)) * np.exp(spread * g.standard_normal(cols))).astype(np.float32))


def padded(x, pad, fill=7.0):
    """A device view of x inside rows `pad` columns longer, and its base."""
    import torch
    base = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=torch.bfloat16, device="cuda")
    base[:, :x.shape[1]] = to_dev_bf16(x)
    return base[:, :x.shape[1]], base


# ------------------------------------------------------------------ row codes

@pytest.mark.parametrize("rows,cols,pad", [(1, 8, 0), (3, 64, 8), (33, 72, 0), (129, 128, 0), (5, 264, 16), (40, 520, 0),
                                           (9, 1024, 0), (7, 1032, 8), (65, 4104, 0), (3, 16392, 0), (2, 32768, 0)])
def test_rows_bytes(w4, rows, cols, pad):
    x = values(rng(rows * 40000 + cols), rows, cols)
    X, _ = padded(x, pad)
    a = w4.quantize_rows_fp8(X)
    codes, scales = oblock.quantize_rows(x)
    np.testing.assert_array_equal(a.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(a.codes.cpu().numpy(), codes)


def test_rows_of_zeros_infinities_and_nan(w4):
    import torch
    x = values(rng(5), 5, 1032)
    x[0] = 0.0
    x[1, 5] = np.inf
    x[2, 7] = np.nan
    x[3] = 1e-38          # the scale would be subnormal
    X = to_dev_bf16(x)
    for cols in (1032, 256):   # a block and a warp per row
        a = w4.quantize_rows_fp8(X[:, :cols])
        codes, s = a.codes.cpu().numpy(), a.scales.cpu().numpy()
        assert s[0] == 1.0 and not codes[0].any()
        assert s[1] == 1.0 and codes[1, 5] == 0x7E          # saturated
        rest = np.delete(x[2, :cols], 7)
        want, ws = oblock.quantize_rows(rest[None, :])
        assert s[2] == ws[0] and codes[2, 7] & 0x7F == 0x7F
        np.testing.assert_array_equal(np.delete(codes[2], 7), want[0])
        assert s[3] == 1.0 and not codes[3].any()
        want, ws = oblock.quantize_rows(x[4:5, :cols])
        np.testing.assert_array_equal(codes[4], want[0])
        assert s[4] == ws[0]


def test_rows_leave_the_padding_alone(w4):
    import torch
    x = values(rng(6), 20, 200)
    codes = torch.full((21, 256), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((21,), -1.0, device="cuda")
    w4.quantize_rows_fp8(to_dev_bf16(x), codes=codes[:20, :200], scales=scales[:20])
    assert bool((codes[:, 200:] == 0xAB).all()) and bool((codes[20] == 0xAB).all()) and float(scales[20]) == -1.0
    np.testing.assert_array_equal(codes[:20, :200].cpu().numpy(), oblock.quantize_rows(x)[0])


# ------------------------------------------------------------------ norm

def check_codes(a, y):
    s = np.max(np.abs(y), axis=1) / 448.0
    s = np.where(s >= 1.17549435e-38, s, 1.0)
    got = a.scales.cpu().numpy().astype(np.float64)
    np.testing.assert_allclose(got, s, rtol=NORM)
    d = oblock.decode(a.codes.cpu().numpy()) * got[:, None]
    # (the code of the largest element may saturate by the scale's own error)
    bound = (E4M3 + 2 * NORM) * np.abs(y) + 2.0 ** -10 * got[:, None] * (1 + NORM)
    assert np.all(np.abs(d - y) <= bound), np.max(np.abs(d - y) - bound)


@pytest.mark.parametrize("rows,cols,residual,weight,pad",
                         [(1, 8, True, True, 0), (2, 128, False, True, 0), (37, 136, True, False, 8),
                          (9, 1000, True, True, 0), (3, 1032, False, False, 8), (130, 2056, True, True, 0),
                          (5, 6144, True, True, 16), (2, 16392, True, True, 0), (2, 32768, True, True, 0)])
def test_norm(w4, rows, cols, residual, weight, pad):
    import torch
    g = rng(cols * 3 + rows)
    x = values(g, rows, cols)
    r = values(g, rows, cols, 0.3) if residual else None
    w = bf16_round((1.0 + 0.3 * g.standard_normal(cols)).astype(np.float32)) if weight else None
    X, _ = padded(x, pad)
    R = padded(r, 2 * pad)[0] if residual else None
    W = to_dev_bf16(w) if weight else None
    normed = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    a, hidden = w4.rms_norm_fp8(X, W, residual=R, normed=normed)
    h, y = oblock.rms_norm(x, r, w)
    check_codes(a, y)
    if residual:
        # one fp32 addition, then bf16
        np.testing.assert_array_equal(from_dev_bf16(hidden), bf16_round(x + r))
    else:
        assert hidden is None
    np.testing.assert_allclose(from_dev_bf16(normed), y, rtol=BF16 + NORM, atol=0)


def test_norm_in_place_and_without_codes(w4):
    import torch
    g = rng(81)
    for cols in (512, 3080):
        x, r = values(g, 70, cols), values(g, 70, cols)
        want_h = bf16_round(x + r)
        for which in ("x", "r"):
            X, R = to_dev_bf16(x), to_dev_bf16(r)
            a, hidden = w4.rms_norm_fp8(X, residual=R, hidden=X if which == "x" else R)
            np.testing.assert_array_equal(from_dev_bf16(X if which == "x" else R), want_h)
            np.testing.assert_array_equal(from_dev_bf16(R if which == "x" else X), r if which == "x" else x)
            check_codes(a, oblock.rms_norm(x, r)[1])
        Y = torch.zeros(70, cols, dtype=torch.bfloat16, device="cuda")
        w4.rmsnorm_fp8(to_dev_bf16(x), 70, cols, cols, None, 0, None, 1e-5, None, 0, Y, cols, None, 0, None)
        np.testing.assert_allclose(from_dev_bf16(Y), oblock.rms_norm(x, eps=1e-5)[1], rtol=BF16 + NORM)


def test_norm_of_extreme_products(w4):
    """h * weight near either end of fp32, the norm itself well inside."""
    g = rng(83)
    for cols in (264, 2056):
        for top, scale, eps in ((2.0 ** 30, 2.0 ** 95, 1e-6), (2.0 ** -34, 2.0 ** -90, 0.0)):
            h = bf16_round((g.uniform(1.0, 2.0, (4, cols)) * g.choice([-top, top], (4, cols))).astype(np.float32))
            w = bf16_round((g.uniform(1.0, 2.0, cols) * scale).astype(np.float32))
            a, _ = w4.rms_norm_fp8(to_dev_bf16(h), to_dev_bf16(w), eps=eps)
            y = oblock.rms_norm(h, None, w, eps)[1]
            check_codes(a, y)
            assert np.all(np.abs(y) > 0) and a.codes.cpu().numpy().any(axis=1).all()


def test_norm_of_zero_rows_and_large_offsets(w4):
    """A zero row gives zeros and scale 1; rows beyond 2^31 elements are found."""
    import torch
    x = np.zeros((3, 256), np.float32)
    x[1] = values(rng(3), 1, 256)[0]
    a, _ = w4.rms_norm_fp8(to_dev_bf16(x))
    assert a.scales.cpu().numpy()[[0, 2]].tolist() == [1.0, 1.0] and not a.codes.cpu().numpy()[[0, 2]].any()
    check_codes(a, oblock.rms_norm(x)[1])
    ld = 1 << 30  # row 3 starts at 3 x 2^30 elements
    base = torch.empty(3 * ld + 256, dtype=torch.bfloat16, device="cuda")
    view = base.as_strided((4, 256), (ld, 1))
    y = values(rng(4), 4, 256)
    view.copy_(to_dev_bf16(y))
    a = w4.quantize_rows_fp8(view)
    np.testing.assert_array_equal(a.codes.cpu().numpy(), oblock.quantize_rows(y)[0])


# ------------------------------------------------------------------ linear

SMALL_CODES = np.array([0x00, 0x30, 0x38, 0x40, 0xB0, 0xB8, 0xC0], np.uint8)  # 0, +-0.5, +-1, +-2


def integer_case(g, M, N, K, residual, bias):
    a = SMALL_CODES[g.integers(0, 7, (M, K))]
    w = SMALL_CODES[g.integers(0, 7, (N, K))]
    s_a = np.exp(0.5 * g.standard_normal(M)).astype(np.float32)
    s_w = (np.exp(0.5 * g.standard_normal(N)) / math.sqrt(K)).astype(np.float32)
    b = bf16_round(g.standard_normal(N).astype(np.float32)) if bias else None
    r = bf16_round(g.standard_normal((M, N)).astype(np.float32)) if residual else None
    return a, s_a, w, s_w, b, r


def dev_u8(a, pad=0):
    import torch
    base = torch.full((a.shape[0], a.shape[1] + pad), 0x7F, dtype=torch.uint8, device="cuda")
    base[:, :a.shape[1]] = torch.from_numpy(a).cuda()
    return base[:, :a.shape[1]]


def linear_bound(y, a, s_a, w, s_w, b, r):
    """Elementwise: the result's bf16 rounding, and fp32 steps relative to the terms."""
    t = np.abs((a @ w.T) * s_a[:, None].astype(np.float64) * s_w[None, :])
    t = t + (0 if b is None else np.abs(b)) + (0 if r is None else np.abs(r))
    return BF16 * np.abs(y) + 2.0 ** -19 * t + 2.0 ** -133


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 1000, 4112), (2, 136, 64), (15, 128, 128), (17, 264, 1040),
                                   (32, 2056, 256), (33, 72, 2064), (64, 512, 8192), (65, 384, 272), (128, 264, 1024),
                                   (129, 64, 48), (200, 1000, 528), (256, 256, 1024), (300, 2056, 400),
                                   (1100, 2312, 912), (2500, 4608, 160)])
@pytest.mark.parametrize("gelu,bias,residual", [(False, False, False), (True, True, False), (False, True, True),
                                                (True, False, True)])
def test_linear_exact_sums(w4, M, N, K, gelu, bias, residual):
    g = rng(M * 7 + N * 3 + K + gelu)
    a, s_a, w, s_w, b, r = integer_case(g, M, N, K, residual, bias)
    A = w4.Fp8Rows(dev_u8(a, 16), to_dev_f32(s_a))
    W = w4.PackedWeightFp8(dev_u8(w, 32), to_dev_f32(s_w), None if b is None else to_dev_bf16(b))
    R = None if r is None else padded(r, 8)[0]
    Y = w4.linear_fp8(A, W, activation=w4.EPI_GELU_TANH if gelu else w4.EPI_NONE, residual=R)
    da, dw = oblock.decode(a), oblock.decode(w)
    want = oblock.linear(da, s_a, dw, s_w, b, gelu, r)
    err = np.abs(from_dev_bf16(Y) - want)
    bound = linear_bound(want, da, s_a, dw, s_w, b, r)
    assert np.all(err <= bound), (np.max(err / bound), np.unravel_index(np.argmax(err / bound), err.shape))


@pytest.mark.parametrize("M,N,K", [(1100, 2312, 4112), (1000, 9400, 2064), (2000, 9400, 2064),
                                   (1100, 520, 65536), (300, 264, 131072)])
def test_linear_wide_tiles(w4, M, N, K):
    """256-column tiles: one, two and four a CTA pair, ragged on both sides;
    rows so long that the row tiles are swept in groups of two and one."""
    g = rng(M + N)
    a, s_a, w, s_w, b, r = integer_case(g, M, N, K, True, True)
    A = w4.Fp8Rows(dev_u8(a), to_dev_f32(s_a))
    W = w4.PackedWeightFp8(dev_u8(w), to_dev_f32(s_w), to_dev_bf16(b))
    Y = w4.linear_fp8(A, W, activation=w4.EPI_GELU_TANH, residual=to_dev_bf16(r))
    # codes of whole and half units: fp32 products of 2 a and 2 w are exact below 2^24
    acc = (2 * oblock.decode(a)).astype(np.float32) @ (2 * oblock.decode(w)).astype(np.float32).T
    t = acc.astype(np.float64) / 4 * s_a[:, None].astype(np.float64) * s_w[None, :]
    want = oblock.gelu_tanh(t + b) + r
    bound = BF16 * np.abs(want) + 2.0 ** -19 * (np.abs(t) + np.abs(b) + np.abs(r)) + 2.0 ** -133
    err = np.abs(from_dev_bf16(Y) - want)
    assert np.all(err <= bound), np.max(err / bound)


@pytest.mark.parametrize("M,N,K", [(1, 768, 3328), (48, 520, 2048), (500, 776, 4096), (1500, 2048, 1552)])
def test_linear_random_codes(w4, M, N, K):
    g = rng(M + N + K)
    x, wt = values(g, M, K), bf16_round((g.standard_normal((N, K)) / math.sqrt(K)).astype(np.float32))
    A = w4.quantize_rows_fp8(to_dev_bf16(x))
    W = w4.pack_weight_fp8(to_dev_bf16(wt))
    y = from_dev_bf16(w4.linear_fp8(A, W))
    ca, sa = oblock.quantize_rows(x)
    cw, sw = oblock.quantize_rows(wt)
    want = oblock.linear(oblock.decode(ca), sa, oblock.decode(cw), sw)
    rel = np.linalg.norm(y - want) / np.linalg.norm(want)
    assert rel <= BF16, rel


def test_linear_takes_a_tensor_scale(w4):
    g = rng(12)
    for M in (40, 400):
        x, wt = values(g, M, 512, 0.2), bf16_round((0.05 * g.standard_normal((264, 512))).astype(np.float32))
        A = w4.quantize_fp8(to_dev_bf16(x))
        W = w4.pack_weight_fp8(to_dev_bf16(wt))
        y = from_dev_bf16(w4.linear_fp8(A, W))
        cw, sw = oblock.quantize_rows(wt)
        want = oblock.linear(oblock.decode(A.codes.cpu().numpy()), A.scale.cpu().numpy(), oblock.decode(cw), sw)
        assert np.linalg.norm(y - want) <= BF16 * np.linalg.norm(want)
        with pytest.raises(ValueError):
            w4.linear_fp8(w4.quantize_fp8(to_dev_bf16(values(g, 512, 512)), transpose=True), W)


@pytest.mark.parametrize("M", [5, 700])
def test_linear_residual_in_place_and_padding(w4, M):
    """Y may be the residual itself; columns and rows behind Y stay."""
    import torch
    g = rng(90 + M)
    a, s_a, w, s_w, b, r = integer_case(g, M, 328, 288, True, True)
    A, W = w4.Fp8Rows(dev_u8(a), to_dev_f32(s_a)), w4.PackedWeightFp8(dev_u8(w), to_dev_f32(s_w), to_dev_bf16(b))
    base = torch.full((M + 2, 344), 3.0, dtype=torch.bfloat16, device="cuda")
    base[:M, :328] = to_dev_bf16(r)
    Y = base[:M, :328]
    w4.linear_fp8(A, W, residual=Y, Y=Y)
    want = oblock.linear(oblock.decode(a), s_a, oblock.decode(w), s_w, b, False, r)
    assert np.all(np.abs(from_dev_bf16(Y.contiguous()) - want) <=
                  linear_bound(want, oblock.decode(a), s_a, oblock.decode(w), s_w, b, r))
    assert bool((base[:, 328:] == 3.0).all()) and bool((base[M:] == 3.0).all())


@pytest.mark.parametrize("M", [1, 100, 900])
def test_linear_repeats_bit_for_bit(w4, M):
    import torch
    g = rng(M)
    A = w4.quantize_rows_fp8(to_dev_bf16(values(g, M, 4096)))
    W = w4.pack_weight_fp8(to_dev_bf16(values(g, 1032, 4096, 0.1)))
    first = w4.linear_fp8(A, W)
    for _ in range(5):
        assert torch.equal(first, w4.linear_fp8(A, W))


# ------------------------------------------------------------------ cross attention

def attention_case(g, batch, kv_batch, sq, sk, heads, kv_heads, d, spread=1.5):
    q = bf16_round((spread * g.standard_normal((batch * sq, heads * d))).astype(np.float32))
    k = bf16_round(g.standard_normal((kv_batch * sk, kv_heads * d)).astype(np.float32))
    v = bf16_round(g.standard_normal((kv_batch * sk, kv_heads * d)).astype(np.float32))
    return q, k, v


def check_attention(got, want, avg):
    err = np.abs(got - want)
    bound = BF16 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * avg
    assert np.all(err <= bound), (np.max(err[bound > 0] / bound[bound > 0]), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("batch,kv_batch,sq,sk,heads,kv_heads,d",
                         [(1, 1, 1, 1, 1, 1, 8), (1, 1, 1, 300, 2, 2, 64), (2, 2, 5, 77, 3, 3, 128),
                          (3, 1, 17, 130, 4, 2, 72), (2, 2, 1, 1500, 8, 2, 128), (1, 1, 1, 2049, 6, 1, 64),
                          (1, 1, 130, 512, 2, 2, 96), (2, 1, 300, 129, 6, 2, 40), (2, 2, 513, 333, 4, 1, 128),
                          (1, 1, 1000, 1025, 3, 3, 64), (1, 1, 256, 128, 1, 1, 128), (1, 1, 40, 3000, 64, 2, 16),
                          (5, 5, 600, 257, 32, 16, 64), (4, 4, 700, 640, 30, 30, 128)])
def test_cross_attention(w4, batch, kv_batch, sq, sk, heads, kv_heads, d):
    g = rng(sq * 3 + sk + d)
    q, k, v = attention_case(g, batch, kv_batch, sq, sk, heads, kv_heads, d)
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=heads, kv_heads=kv_heads, batch=batch,
                           kv_batch=kv_batch)
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, heads, kv_heads, batch, kv_batch))


@pytest.mark.parametrize("sq", [1, 60, 700])
@pytest.mark.parametrize("lens", [(0, 1, 128, 400), (400, 129, 0, 127), (0, 0, 0, 0), (-5, 1000, 257, 400)])
def test_cross_attention_lengths(w4, sq, lens):
    """Lengths per prompt, none at all among them; values outside the range
    count as the nearest.  What lies behind a length is NaN and infinity."""
    import torch
    g = rng(sq + lens[1])
    batch, sk, heads, d = 4, 400, 4, 128
    q, k, v = attention_case(g, batch, batch, sq, sk, heads, 2, d)
    n = np.clip(np.array(lens), 0, sk)
    kd, vd = k.copy(), v.copy()
    for b in range(batch):
        kd[b * sk + n[b]:(b + 1) * sk] = np.nan
        vd[b * sk + n[b]:(b + 1) * sk] = np.inf
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(vd), heads=heads, kv_heads=2, batch=batch,
                           kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    got = from_dev_bf16(O)
    check_attention(got, *oblock.cross_attention(q, k, v, heads, 2, batch, batch, kv_len=n))
    for b in range(batch):
        if n[b] == 0:
            assert not got[b * sq:(b + 1) * sq].any()


@pytest.mark.parametrize("sq,sk", [(1, 1000), (50, 385), (600, 300)])
@pytest.mark.parametrize("shared", [False, True])
def test_cross_attention_key_mask(w4, sq, sk, shared):
    """Masks with holes, whole tiles and whole rows masked, with NaN keys and
    values in the masked places; together with lengths."""
    import torch
    g = rng(sq + sk + shared)
    batch, heads, d = 3, 2, 64
    kv_batch = 1 if shared else batch
    q, k, v = attention_case(g, batch, kv_batch, sq, sk, heads, heads, d)
    mask = g.random((kv_batch, sk)) < 0.6
    mask[0, :200] = False
    if not shared:
        mask[1] = False
    n = np.array([sk - 40] * kv_batch, np.int32)
    kd, vd = k.copy(), v.copy()
    kd[~mask.reshape(-1)] = np.inf
    vd[~mask.reshape(-1)] = np.nan
    M = torch.zeros(kv_batch, sk + 13, dtype=torch.bool, device="cuda")
    M[:, :sk] = torch.from_numpy(mask).cuda()
    Q, K, V = to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(vd)
    O = w4.cross_attention(Q, K, V, heads=heads, batch=batch, kv_batch=kv_batch, key_mask=M[:, :sk])
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, heads, heads, batch, kv_batch, key_mask=mask))
    O = w4.cross_attention(Q, K, V, heads=heads, batch=batch, kv_batch=kv_batch, key_mask=M.to(torch.uint8)[:, :sk],
                           kv_len=torch.from_numpy(n).cuda())
    check_attention(from_dev_bf16(O),
                    *oblock.cross_attention(q, k, v, heads, heads, batch, kv_batch, kv_len=n, key_mask=mask))


@pytest.mark.parametrize("sq", [3, 500])
def test_cross_attention_views(w4, sq):
    """Keys and values from one projection, queries and outputs inside wider
    rows; rows and columns behind the output stay as they were."""
    import torch
    g = rng(sq)
    batch, sk, heads, kv_heads, d = 2, 200, 4, 2, 64
    q, k, v = attention_case(g, batch, batch, sq, sk, heads, kv_heads, d)
    Q, _ = padded(q, 24)
    KV = to_dev_bf16(np.concatenate([k, v], axis=1))
    base = torch.full((batch * sq + 3, heads * d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    O = base[:batch * sq, :heads * d]
    w4.cross_attention(Q, KV[:, :kv_heads * d], KV[:, kv_heads * d:], heads=heads, kv_heads=kv_heads, batch=batch, O=O,
                       softmax_scale=0.2)
    check_attention(from_dev_bf16(O.contiguous()),
                    *oblock.cross_attention(q, k, v, heads, kv_heads, batch, batch, scale=0.2))
    assert bool((base[batch * sq:] == 5.0).all()) and bool((base[:, heads * d:] == 5.0).all())


@pytest.mark.parametrize("sq", [4, 400])
def test_cross_attention_moves_its_offset(w4, sq):
    """Scores that grow from tile to tile by far more than the slack, and one
    key that outweighs all others."""
    g = rng(17 + sq)
    sk, d = 900, 128
    q, k, v = attention_case(g, 1, 1, sq, sk, 2, 2, d, spread=0.05)
    q[:, 0] = q[:, d] = 8.0
    grow = bf16_round((np.arange(sk) // 128 * 6.0 + g.standard_normal(sk)).astype(np.float32))
    k[:, 0] = grow
    k[:, d] = grow[::-1]
    k[450, 0] = 80.0
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=2)
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 2, 2, 1, 1))


@pytest.mark.parametrize("sq", [4, 400])
def test_cross_attention_scores_of_minus_infinity(w4, sq):
    """Scores that overflow below weigh nothing, over a whole tile too; a row
    of nothing else is 0."""
    g = rng(29 + sq)
    sk, d = 400, 64
    q, k, v = attention_case(g, 1, 1, sq, sk, 2, 2, d)
    q[:, 0] = 2.0 ** 70
    gone = g.random(sk) < 0.4
    gone[:130] = True
    k[:, 0] = np.where(gone, -2.0 ** 70, 0.0)
    O = from_dev_bf16(w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=2))
    want, avg = oblock.cross_attention(q, k, v, 2, 2, 1, 1)
    check_attention(O, want, avg)
    k[:, 0] = -2.0 ** 70
    O = from_dev_bf16(w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=2))
    assert not O[:, :d].any()
    check_attention(O[:, d:], want[:, d:], avg[:, d:])


@pytest.mark.parametrize("sq", [4, 400])
def test_cross_attention_nan_scores_show(w4, sq):
    """A NaN key that counts makes its head's rows NaN wherever it lies; the
    other head is untouched; an infinite score likewise."""
    g = rng(23 + sq)
    sk, d = 300, 64
    q, k, v = attention_case(g, 1, 1, sq, sk, 2, 2, d)
    want, avg = oblock.cross_attention(q, k, v, 2, 2, 1, 1)
    for j in (0, 1, 2, 3, 140, 299):
        for bad in (np.nan, np.inf):
            kd = k.copy()
            kd[j, 3] = bad
            got = from_dev_bf16(w4.cross_attention(to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(v), heads=2))
            check_attention(got[:, d:], want[:, d:], avg[:, d:])
            hit = np.isnan(bad) | (q[:, 3] > 0)
            assert np.all(np.isnan(got[hit, :d])) and np.all(np.isfinite(got[~hit, :d]))


@pytest.mark.parametrize("d", [64, 120])
@pytest.mark.parametrize("what", ["lengths", "mask", "offset", "nan"])
def test_cross_attention_many_rows(w4, d, what):
    """The same with enough sequences, heads and queries that every SM takes
    several tiles of 256 rows, prompts without keys between others."""
    import torch
    g = rng(300 + d)
    batch, sq, sk, heads, kv_heads = 6, 520, 390, 60, 30
    q, k, v = attention_case(g, batch, batch, sq, sk, heads, kv_heads, d)
    kd, vd, n, mask, bad = k.copy(), v.copy(), None, None, None
    if what == "lengths":
        n = np.array([390, 0, 1, 129, 0, 256], np.int32)
        for b in range(batch):
            kd[b * sk + n[b]:(b + 1) * sk] = np.inf
            vd[b * sk + n[b]:(b + 1) * sk] = np.nan
    elif what == "mask":
        mask = g.random((batch, sk)) < 0.5
        mask[2] = False
        mask[3, :128] = False
        kd[~mask.reshape(-1)] = np.nan
        vd[~mask.reshape(-1)] = np.inf
    elif what == "offset":
        grow = bf16_round((np.arange(batch * sk) % sk // 64 * 3.0).astype(np.float32))
        k[:, ::d] = grow[:, None]
        q[:, ::d] = 4.0
        kd = k
    else:
        kd[sk + 7, 2 * d + 5] = np.nan
        bad = (slice(sq, 2 * sq), slice(4 * d, 6 * d))
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(vd), heads=heads, kv_heads=kv_heads, batch=batch,
                           kv_len=None if n is None else torch.from_numpy(n).cuda(),
                           key_mask=None if mask is None else torch.from_numpy(mask).cuda())
    got = from_dev_bf16(O)
    want, avg = oblock.cross_attention(q, k, v, heads, kv_heads, batch, batch, kv_len=n, key_mask=mask)
    if bad is not None:
        assert np.all(np.isnan(got[bad]))
        got[bad] = want[bad]
    check_attention(got, want, avg)


def test_cross_attention_no_keys_at_all(w4):
    import torch
    base = torch.full((10, 72), 2.0, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w4.cross_attention(base[:, :64].clone(), k, k, heads=1, O=base[:, :64])
    assert not bool(base[:, :64].any()) and bool((base[:, 64:] == 2.0).all())


def test_cross_attention_far_keys(w4):
    """Keys beyond 2^31 elements of a wide projection."""
    import torch
    g = rng(31)
    sk, ld = 300, 1 << 23
    q, k, v = attention_case(g, 1, 1, 20, sk, 1, 1, 128)
    base = torch.empty(sk * ld, dtype=torch.bfloat16, device="cuda")
    K, V = base.as_strided((sk, 128), (ld, 1)), base.as_strided((sk, 128), (ld, 1), 256)
    K.copy_(to_dev_bf16(k))
    V.copy_(to_dev_bf16(v))
    O = w4.cross_attention(to_dev_bf16(q), K, V, heads=1)
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 1, 1, 1, 1))


# ------------------------------------------------------------------ together

def sublayer(w4, x, r, norm_w, wq, wo, K, V, n, batch, heads, activation=0):
    a, h = w4.rms_norm_fp8(x, norm_w, residual=r)
    q = w4.linear_fp8(a, wq)
    o = w4.cross_attention(q, K, V, heads=heads, batch=batch, kv_len=n)
    return w4.linear_fp8(w4.quantize_rows_fp8(o), wo, activation=activation, residual=h), h, q, o


@pytest.mark.parametrize("sq", [1, 90, 640])
def test_conditioned_sublayer(w4, sq):
    """Norm, query projection, attention to a ragged prompt, output projection
    onto the residual stream: each step against the oracle on the inputs it
    was given, also from another stream and from a replayed graph."""
    import torch
    g = rng(1000 + sq)
    batch, sk, heads, d = 2, 150, 4, 64
    D = heads * d
    x, r = values(g, batch * sq, D, 0.4), values(g, batch * sq, D, 0.4)
    nw = bf16_round((1 + 0.1 * g.standard_normal(D)).astype(np.float32))
    wq, wo = (bf16_round((g.standard_normal((D, D)) / 16).astype(np.float32)) for _ in range(2))
    _, k, v = attention_case(g, batch, batch, 1, sk, heads, heads, d)
    lens = np.array([sk, 70], np.int32)
    args = [to_dev_bf16(t) for t in (x, r, nw)]
    Wq, Wo = w4.pack_weight_fp8(to_dev_bf16(wq)), w4.pack_weight_fp8(to_dev_bf16(wo))
    K, V, n = to_dev_bf16(k), to_dev_bf16(v), torch.from_numpy(lens).cuda()

    def call():
        return sublayer(w4, *args, Wq, Wo, K, V, n, batch, heads)

    y, h, q, o = call()
    oq = from_dev_bf16(q)
    want, avg = oblock.cross_attention(oq, k, v, heads, heads, batch, batch, kv_len=lens)
    check_attention(from_dev_bf16(o), want, avg)
    oo, hh = from_dev_bf16(o), from_dev_bf16(h)
    co, so = oblock.quantize_rows(oo)
    cw, sw = oblock.quantize_rows(wo)
    full = oblock.linear(oblock.decode(co), so, oblock.decode(cw), sw, residual=hh)
    assert np.linalg.norm(from_dev_bf16(y) - full) <= BF16 * np.linalg.norm(full)
    _, ny = oblock.rms_norm(x, r, nw)
    cq, sq_ = oblock.quantize_rows(wq)
    # the norm's codes: each off by half a step (2^-4) at most, at random, so
    # the sum over 256 of them is off by far less than 2^-4 of its norm
    qq = oblock.linear(ny, np.ones(1), oblock.decode(cq), sq_)
    assert np.linalg.norm(oq - qq) <= E4M3 * np.linalg.norm(qq)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[0], y)

    graphs = []
    for _ in range(2):  # two captures of the same calls: they share nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out))
    args[0].copy_(args[0].flip(0))
    n.copy_(n.flip(0))
    y2 = call()[0]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out[0], y2)


def test_norm_feeds_a_w4a4_layer(w4):
    """normed is what the W4A4 quantiser takes."""
    import torch
    g = rng(55)
    x = values(g, 300, 512)
    X = to_dev_bf16(x)
    normed = torch.empty_like(X)
    w4.rms_norm_fp8(X, normed=normed)
    qa = w4.quantize_act(normed)
    w = w4.pack_weight(to_dev_f32((0.05 * g.standard_normal((256, 512))).astype(np.float32)))
    y = from_dev_bf16(w4.gemm(qa, w))
    again = w4.gemm(w4.quantize_act(to_dev_bf16(from_dev_bf16(normed))), w)
    np.testing.assert_array_equal(from_dev_bf16(again), y)
    assert np.all(np.isfinite(y)) and np.any(y)
