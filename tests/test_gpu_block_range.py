"""GPU parity of the layers around the W4A4 ones at the ends of their range:
scores and rows whose magnitudes leave fp32's comfortable middle, against the
64-bit oracle.

Tolerances are those of the ordinary cases (a weight of the attention rounded
to bf16, 2^-8, after an exponential good to 2^-13, and the output's own 2^-8).
Scores: the queries and keys below have one term that carries the magnitude,
a product of powers of two and small integers, so that the scores are exact in
fp32 and the oracle's weights are the operator's.  Of the differences that
decide the weights, c s is off by three roundings (c, the difference, the
product): below 2^-22 of a difference that matters (at most 32 binades), far
below the 2^-12 that the bound holds for it.
"""
import numpy as np
import pytest

from helpers import from_dev_bf16, to_dev_bf16
from oracle import block as oblock
from synth import bf16_round, rng

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


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


def check_attention(got, want, avg):
    err = np.abs(got - want)
    bound = BF16 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * avg
    assert np.all(err <= bound), (np.max(err[bound > 0] / bound[bound > 0]), np.argwhere(~(err <= bound))[:4])


# ------------------------------------------------------------------ cross attention

def large_scores(g, sq, sk, heads, d, top, sign):
    """Scores +-top * (128 + i) / 2 for whole i, eight keys a value at least:
    keys that share the row's largest score share the weight, the others have none
    (or, for the smallest tops, little)."""
    q = np.zeros((sq, heads * d), np.float32)
    k = np.zeros((sk, heads * d), np.float32)
    for h in range(heads):
        q[:, h * d] = top
        k[:, h * d] = sign * (128 + g.integers(0, max(1, min(sk // 8, 128)), sk)) / 2
    v = bf16_round(g.standard_normal((sk, heads * d)).astype(np.float32))
    return q, k, v


@pytest.mark.parametrize("sq", [3, 300])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("log2_top", [10, 17, 20, 24, 27, 31, 40, 80, 118])
def test_cross_attention_of_large_scores(w4, sq, sign, log2_top):
    g = rng(log2_top * 2 + sq)
    for sk, d in ((64, 64), (700, 128)):
        q, k, v = large_scores(g, sq, sk, 2, d, 2.0 ** log2_top, sign)
        O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=2, softmax_scale=0.125)
        check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 2, 2, 1, 1, scale=0.125))


@pytest.mark.parametrize("sq", [3, 300])
@pytest.mark.parametrize("value", [-2.0 ** 33, 2.0 ** 33, -2.0 ** 100, 2.0 ** 121])
def test_cross_attention_of_one_large_score(w4, sq, value):
    """Every score the same large number (a feature used as a mask that stops
    short of overflow): the average of the values."""
    g = rng(51 + sq)
    sk, d = 333, 64
    q = np.zeros((sq, d), np.float32)
    k = np.zeros((sk, d), np.float32)
    q[:, 3], k[:, 3] = 2.0 ** 4, value / 2.0 ** 4
    v = bf16_round(g.standard_normal((sk, d)).astype(np.float32))
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=1)
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 1, 1, 1, 1))


@pytest.mark.parametrize("sq", [3, 300])
def test_cross_attention_of_rows_far_apart(w4, sq):
    """Rows of ordinary and of large scores in one warp, and rows whose scores
    grow from ordinary to large ones and back from tile to tile."""
    g = rng(57 + sq)
    sk, d = 900, 128
    q = bf16_round((0.5 * g.standard_normal((sq, 2 * d))).astype(np.float32))
    k = bf16_round(g.standard_normal((sk, 2 * d)).astype(np.float32))
    v = bf16_round(g.standard_normal((sk, 2 * d)).astype(np.float32))
    # head 0: every third row is large.  Its other products are cleared: beside
    # 2^40 they would be lost in the fp32 score, not in the oracle's
    q[::3, :d] = 0.0
    q[::3, 0] = 2.0 ** 40
    k[:, 0] = g.integers(0, 9, sk) - 4
    # head 1: whole scores of -2^27 .. 2^27 by key tile, several at the top
    q[:, d:] = 0.0
    q[:, d] = 2.0 ** 20
    steps = np.array([-128.0, -1.0, -0.5, 0.0, 2.0 ** -20, 2.0 ** -17, 1.0, 128.0])
    k[:, d] = steps[np.minimum(np.arange(sk) // 128, 7)]
    for flip in (False, True):
        if flip:
            k[:, d] = k[::-1, d].copy()
        O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(v), heads=2)
        check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 2, 2, 1, 1))


@pytest.mark.parametrize("sq", [3, 300])
def test_cross_attention_of_large_scores_under_a_mask(w4, sq):
    """Keys that do not count are NaN, among large scores."""
    import torch
    g = rng(61 + sq)
    sk, d = 400, 64
    q, k, v = large_scores(g, sq, sk, 2, d, 2.0 ** 60, -1.0)
    mask = g.random((1, sk)) < 0.5
    mask[0, 128:256] = False
    kd, vd = k.copy(), v.copy()
    kd[~mask[0]] = np.nan
    vd[~mask[0]] = np.inf
    O = w4.cross_attention(to_dev_bf16(q), to_dev_bf16(kd), to_dev_bf16(vd), heads=2,
                           key_mask=torch.from_numpy(mask).cuda(), kv_len=torch.tensor([390], dtype=torch.int32).cuda())
    check_attention(from_dev_bf16(O), *oblock.cross_attention(q, k, v, 2, 2, 1, 1, kv_len=[390], key_mask=mask))


# ------------------------------------------------------------------ norm
#
# The row factor sums up to 2^15 squares in fp32: at most 8 vectors of 8 a
# thread, 5 + 5 additions over lanes and warps, so chains of 74; half of that
# error after the root and six more operations: 43 x 2^-24 < 2^-18.  Scaling by
# a power of two adds none.

NORM, E4M3 = 2.0 ** -18, 2.0 ** -4


def check_norm(w4, x, r, w, eps, in_place=None):
    import torch
    X = to_dev_bf16(x)
    R = None if r is None else to_dev_bf16(r)
    normed = torch.empty_like(X)
    hidden = {None: None, "x": X, "r": R, "own": torch.empty_like(X)}[in_place]
    a, hidden = w4.rms_norm_fp8(X, None if w is None else to_dev_bf16(w), residual=R, eps=eps, hidden=hidden,
                                normed=normed)
    _, y = oblock.rms_norm(x, r, w, np.float64(np.float32(eps)))
    s = np.max(np.abs(y), axis=1) / 448.0
    s = np.where(s >= 1.17549435e-38, s, 1.0)
    got = a.scales.cpu().numpy().astype(np.float64)
    np.testing.assert_allclose(got, s, rtol=NORM)
    d = oblock.decode(a.codes.cpu().numpy()) * got[:, None]
    bound = (E4M3 + 2 * NORM) * np.abs(y) + 2.0 ** -10 * got[:, None] * (1 + NORM)
    assert np.all(np.abs(d - y) <= bound), np.max(np.abs(d - y) / bound)
    # (half a step of a bf16 below its normal range: 2^-134)
    np.testing.assert_allclose(from_dev_bf16(normed), y, rtol=BF16 + NORM, atol=2.0 ** -134)
    if r is not None or in_place is not None:
        h = x if r is None else x + r  # one fp32 addition
        np.testing.assert_array_equal(from_dev_bf16(hidden), bf16_round(h))


def rows_of(g, rows, cols, log2):
    with np.errstate(under="ignore"):
        return bf16_round((g.uniform(1.0, 2.0, (rows, cols)) * g.choice([-1.0, 1.0], (rows, cols))
                           * 2.0 ** float(log2)).astype(np.float32))


@pytest.mark.parametrize("cols", [8, 128, 264, 1000, 2056, 16392, 32768])
@pytest.mark.parametrize("log2", [-130, -120, -90, -60, -50, -44, -30, 28, 45, 53, 60, 64, 90, 125])
def test_norm_of_far_rows(w4, cols, log2):
    """Rows whose squares leave fp32's range at either end, with and without a
    residual, a weight, and hidden in place."""
    g = rng(cols + 1000 + log2)
    rows = 5 if cols > 4096 else 33
    x, r = rows_of(g, rows, cols, log2), rows_of(g, rows, cols, log2 - 1)
    w = bf16_round((1.0 + 0.3 * g.standard_normal(cols)).astype(np.float32))
    w[::7] = 0.0
    eps = 0.0 if log2 < 0 else 1e-6
    check_norm(w4, x, None, None, eps)
    check_norm(w4, x, None, w, eps, "own")
    for in_place in (None, "x", "r"):
        check_norm(w4, x, r, w, eps, in_place)


@pytest.mark.parametrize("cols", [128, 512, 2056, 24576])
@pytest.mark.parametrize("in_place", [None, "x", "r"])
def test_norm_of_mixed_rows(w4, cols, in_place):
    """Far and ordinary rows side by side, and rows that hold both kinds of
    elements: one huge among ordinary ones, magnitudes that rise and fall
    along the row, zeros among tiny ones."""
    g = rng(cols + 7)
    rows = 40 if cols < 4096 else 9
    x, r = rows_of(g, rows, cols, 0), rows_of(g, rows, cols, -2)
    x[1] = rows_of(g, 1, cols, 70)
    x[2, cols // 3] = 2.0 ** 80
    x[3] = rows_of(g, 1, cols, 0) * 2.0 ** np.linspace(-60, 100, cols).astype(np.float32).round()
    x[4] = rows_of(g, 1, cols, 0) * 2.0 ** np.linspace(100, -60, cols).astype(np.float32).round()
    x[5], r[5] = rows_of(g, 1, cols, -70), 0.0
    x[6], r[6] = 0.0, 0.0
    x[6, 5] = 2.0 ** -100
    x[7], r[7] = rows_of(g, 1, cols, -40), 0.0
    x[8, -1] = 2.0 ** 57
    for eps in (1e-38, 1e-30, 1e-26, 1e-6, 1.0, 1e37):
        check_norm(w4, x, r, None, eps, in_place)


def test_norm_of_rows_that_are_not_numbers(w4):
    """Zero rows with eps 0, NaN and infinities: the row NaN (the scale 1), the
    others as they are; an infinite element NaN among zeros."""
    import torch
    g = rng(91)
    for cols in (256, 4096):
        x = rows_of(g, 12, cols, 0)
        x[1] = 0.0
        x[3, 17] = np.nan
        x[5, cols - 1] = np.inf
        x[7] = rows_of(g, 1, cols, 80)
        X = to_dev_bf16(x)
        X[9, 3] = float("-inf")
        normed = torch.empty_like(X)
        a, _ = w4.rms_norm_fp8(X, eps=0.0, normed=normed)
        y, s, codes = from_dev_bf16(normed), a.scales.cpu().numpy(), a.codes.cpu().numpy()
        for i in (1, 3):
            assert np.all(np.isnan(y[i])) and s[i] == 1.0 and np.all((codes[i] & 0x7F) == 0x7F)
        for i, j in ((5, cols - 1), (9, 3)):
            assert np.isnan(y[i, j]) and not np.delete(y[i], j).any() and s[i] == 1.0
        rest = [0, 2, 4, 6, 7, 8, 10, 11]
        np.testing.assert_allclose(y[rest], oblock.rms_norm(x[rest], eps=0.0)[1], rtol=BF16 + NORM)


@pytest.mark.parametrize("sq,ld", [(1, 72), (3, 72), (700, 72), (2, (1 << 30) + 8)])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 1)])
def test_cross_attention_without_keys(w4, sq, ld, heads, kv_heads):
    """No keys at all: zeros, whatever the output's stride, and nothing beside them."""
    import torch
    d = 64 // heads
    base = torch.full((2 * sq, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    O = base
    if ld > 72:
        far = torch.empty(ld * (2 * sq - 1) + 72, dtype=torch.bfloat16, device="cuda")
        O = far.as_strided((2 * sq, 72), (ld, 1))
        O.copy_(base)
    none = torch.empty(0, kv_heads * d, dtype=torch.bfloat16, device="cuda")
    q = torch.full((2 * sq, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    for kv_len in (None, torch.tensor([5, -1], dtype=torch.int32, device="cuda")):
        w4.cross_attention(q, none, none, heads=heads, kv_heads=kv_heads, batch=2, O=O[:, :64], kv_len=kv_len)
        assert not bool(O[:, :64].any()) and bool((O[:, 64:] == 3.0).all())
        O.fill_(3.0)
