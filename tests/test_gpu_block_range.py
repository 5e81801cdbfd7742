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
