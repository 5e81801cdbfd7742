"""The cases on which the block operators around the quantised linear layers are measured.

Four operators of a conditioned transformer block, in the order a block runs them:

* ``norm``    residual addition and root-mean-square norm, out in E4M3 with one scale per row
* ``rows``    E4M3 codes with one scale per row of a tensor as it stands (weights, attention outputs)
* ``linear``  the product of such codes with bias, activation and residual in its epilogue
* ``cross``   attention of image tokens to an encoder's states of another length

``run`` computes a case in elementary torch operations, or, with ``own`` set, through the package.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 1.17549435e-38  # the smallest normal fp32 number


def listed():
    return [
        # one modulation vector's norm: a single row, where only latency counts
        dict(name="norm_1x6144", op="norm", rows=1, cols=6144, residual=True, weight=True),
        # a 1024px sequence (4096 image and 512 text tokens) at hidden size 6144
        dict(name="norm_4608x6144", op="norm", rows=4608, cols=6144, residual=True, weight=True),
        # a batch of per-head query norms of an odd token count: short rows, no residual
        dict(name="norm_heads_36888x128", op="norm", rows=36888, cols=128, residual=False, weight=True),
        # a ragged prompt's encoder states on their way to the key projection
        dict(name="rows_333x4096", op="rows", rows=333, cols=4096),
        # the attention output of a 2048px sequence before its projection
        dict(name="rows_16896x6144", op="rows", rows=16896, cols=6144),
        # the modulation layer of one image: one token times six hidden sizes, weight streaming
        dict(name="linear_1x36864x6144", op="linear", m=1, n=36864, k=6144, act="none", bias=True, residual=False),
        # a prompt's first projection, odd sizes, with its activation
        dict(name="linear_333x2056x4112", op="linear", m=333, n=2056, k=4112, act="gelu", bias=True, residual=False),
        # the attention output projection of a 1024px sequence, added to the residual stream
        dict(name="linear_4608x6144x6144", op="linear", m=4608, n=6144, k=6144, act="none", bias=True, residual=True),
        # the up projection of a 2048px sequence
        dict(name="linear_16896x18432x6144", op="linear", m=16896, n=18432, k=6144, act="gelu", bias=True,
             residual=False),
        # one pooled query per image against a long encoder output, query heads in groups of four
        dict(name="cross_4x1x4109", op="cross", batch=4, kv_batch=4, q=1, kv=4109, heads=32, kv_heads=8, d=128,
             ragged=True),
        # two images against their own prompts of up to 512 tokens
        dict(name="cross_2x4096x512", op="cross", batch=2, kv_batch=2, q=4096, kv=512, heads=48, kv_heads=48, d=128,
             ragged=True),
        # a 2048px image against a reference image's tokens, all of them seen
        dict(name="cross_1x16384x4096", op="cross", batch=1, kv_batch=1, q=16384, kv=4096, heads=16, kv_heads=16,
             d=128, ragged=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "rows", "linear", "cross"])
    if op == "norm":
        cols = _log(rng, 64, 16384, 8)
        return dict(op=op, rows=_log(rng, 1, min(1 << 17, (16896 * 6144) // cols)), cols=cols,
                    residual=rng.random() < 0.6, weight=rng.random() < 0.8)
    if op == "rows":
        cols = _log(rng, 64, 24576, 8)
        return dict(op=op, rows=_log(rng, 1, min(1 << 17, (16896 * 6144) // cols)), cols=cols)
    if op == "linear":
        n, k = _log(rng, 256, 18432, 8), _log(rng, 256, 12288, 16)
        return dict(op=op, m=_log(rng, 1, 9216), n=n, k=k, act=rng.choice(["none", "gelu"]),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 3, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4])
    batch = rng.choice([1, 2, 3, 4])
    d = rng.choice([64, 72, 96, 128])
    kv = _log(rng, 16, 4096)
    # queries up to the largest listed case's number of scores
    most = (16 * 16384 * 4096) // (batch * kv_heads * group * kv)
    return dict(op=op, batch=batch, kv_batch=rng.choice([1, batch]), q=_log(rng, 1, min(16384, most)), kv=kv,
                heads=kv_heads * group, kv_heads=kv_heads, d=d, ragged=rng.random() < 0.7)


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _channels(g, cols):
    """Per-channel magnitudes of a transformer's activations: log-normal, one in a hundred far out."""
    mag = torch.exp(0.5 * _normal(g, cols))
    far = torch.rand(cols, device="cuda", generator=g) < 0.01
    return torch.where(far, 20.0 * mag, mag)


def _codes(x):
    """E4M3 codes of the rows of x, as bytes, and their scales: what such a program holds before a product."""
    s = x.float().abs().amax(1) / E4M3_MAX
    s = torch.where(s >= TINY, s, torch.ones_like(s))
    return (x.float() * (1.0 / s)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "rows"):
        m, d = case["rows"], case["cols"]
        s["x"] = (_normal(g, m, d) * _channels(g, d)).bfloat16()
        if op == "norm":
            s["r"] = (2.0 * _normal(g, m, d)).bfloat16() if case["residual"] else None
            s["w"] = (1.0 + 0.2 * _normal(g, d)).bfloat16() if case["weight"] else None
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _codes((_normal(g, m, k) * _channels(g, k)).bfloat16())
        s["b"], s["sb"] = _codes((_normal(g, n, k) / math.sqrt(k)).bfloat16())
        s["bias"] = (0.1 * _normal(g, n)).bfloat16() if case["bias"] else None
        s["res"] = _normal(g, m, n).bfloat16() if case["residual"] else None
    else:
        b, kb, hd, kd = case["batch"], case["kv_batch"], case["heads"] * case["d"], case["kv_heads"] * case["d"]
        s["query"] = (1.5 * _normal(g, b * case["q"], hd)).bfloat16()
        kv = _normal(g, kb * case["kv"], 2 * kd).bfloat16()  # one projection gives keys and values
        s["key"], s["value"] = kv[:, :kd], kv[:, kd:]
        s["len"] = None
        if case["ragged"]:
            # prompts fill between a quarter and all of the padded length
            s["len"] = torch.randint(max(1, case["kv"] // 4), case["kv"] + 1, (kb,), device="cuda", generator=g,
                                     dtype=torch.int32)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import bit_diffusion_transformer_nvfp4_b200 as w4
    if s["op"] == "norm":
        a, hidden = w4.rms_norm_fp8(s["x"], s["w"], residual=s["r"], eps=1e-6)
        return {"codes": a.codes.view(E4M3), "scales": a.scales, "hidden": hidden}
    if s["op"] == "rows":
        a = w4.quantize_rows_fp8(s["x"])
        return {"codes": a.codes.view(E4M3), "scales": a.scales}
    if s["op"] == "linear":
        a = w4.Fp8Rows(s["a"], s["sa"])
        w = w4.PackedWeightFp8(s["b"], s["sb"], s["bias"])
        act = w4.EPI_GELU_TANH if s["act"] == "gelu" else w4.EPI_NONE
        return {"y": w4.linear_fp8(a, w, activation=act, residual=s["res"])}
    return {"o": w4.cross_attention(s["query"], s["key"], s["value"], heads=s["heads"], kv_heads=s["kv_heads"],
                                    batch=s["batch"], kv_batch=s["kv_batch"], kv_len=s["len"])}


def _run_plain(s):
    if s["op"] in ("norm", "rows"):
        y = s["x"].float()
        hidden = None
        if s["op"] == "norm":
            if s["r"] is not None:
                y = y + s["r"].float()
                hidden = y.bfloat16()
            y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + 1e-6)
            if s["w"] is not None:
                y = y * s["w"].float()
        scale = y.abs().amax(1) / E4M3_MAX
        scale = torch.where(scale >= TINY, scale, torch.ones_like(scale))
        codes = (y * (1.0 / scale)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        out = {"codes": codes, "scales": scale}
        return {**out, "hidden": hidden} if s["op"] == "norm" else out
    if s["op"] == "linear":
        y = s["a"].view(E4M3).float() @ s["b"].view(E4M3).float().t()
        y = y * s["sa"][:, None] * s["sb"]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if s["act"] == "gelu":
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.bfloat16()}
    b, kb, hk, d = s["batch"], s["kv_batch"], s["kv_heads"], s["d"]
    group = s["heads"] // hk
    q = s["query"].float().view(b, s["q"], hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * s["q"], d)
    k = s["key"].float().view(kb, s["kv"], hk, d).permute(0, 2, 3, 1)
    v = s["value"].float().view(kb, s["kv"], hk, d).permute(0, 2, 1, 3)
    p = (q @ k) / math.sqrt(d)
    if s["len"] is not None:
        seen = torch.arange(s["kv"], device=p.device) < s["len"][:, None]
        p = p.masked_fill(~seen[:, None, None, :], -math.inf)
    p = torch.exp(p - p.amax(3, keepdim=True))
    o = (p @ v) / p.sum(3, keepdim=True)
    return {"o": o.view(b, hk, group, s["q"], d).permute(0, 3, 1, 2, 4).reshape(b * s["q"], s["heads"] * d).bfloat16()}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("norm", "rows"):
        # codes are compared as the unrounded values they round
        h = s["x"].to(f64)
        hidden = None
        if case["op"] == "norm":
            if s["r"] is not None:
                h = hidden = h + s["r"].to(f64)
            rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + 1e-6)
            h = h / rms[:, None]
            if s["w"] is not None:
                h = h * s["w"].to(f64)[None, :]
        top = torch.linalg.vector_norm(h, ord=math.inf, dim=1)
        scale = torch.where(top / E4M3_MAX < TINY, torch.ones_like(top), top / E4M3_MAX)
        out = {"codes": h / scale[:, None], "scales": scale}
        return {**out, "hidden": hidden} if case["op"] == "norm" else out
    if case["op"] == "linear":
        a = s["a"].view(E4M3).to(f64) * s["sa"].to(f64)[:, None]
        w = s["b"].view(E4M3).to(f64) * s["sb"].to(f64)[:, None]
        y = torch.einsum("mk,nk->mn", a, w)
        if s["bias"] is not None:
            y += s["bias"].to(f64)
        if case["act"] == "gelu":
            y = y / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
        if s["res"] is not None:
            y += s["res"].to(f64)
        return {"y": y}
    b, sq, sk, d = case["batch"], case["q"], case["kv"], case["d"]
    group = case["heads"] // case["kv_heads"]
    o = torch.empty(b * sq, case["heads"] * d, dtype=f64, device="cuda")
    for i in range(b):
        j = i if case["kv_batch"] > 1 else 0
        n = sk if s["len"] is None else int(s["len"][j])
        for h in range(case["heads"]):
            hk = h // group
            keys = s["key"][j * sk:j * sk + n, hk * d:(hk + 1) * d].to(f64)
            values = s["value"][j * sk:j * sk + n, hk * d:(hk + 1) * d].to(f64)
            scores = s["query"][i * sq:(i + 1) * sq, h * d:(h + 1) * d].to(f64) @ keys.t()
            o[i * sq:(i + 1) * sq, h * d:(h + 1) * d] = torch.softmax(scores / math.sqrt(d), 1) @ values
    return {"o": o}


def _keys_seen(case):
    """Keys a query attends to on average: the prompts' lengths are even between a quarter and all."""
    return 0.625 * case["kv"] if case["ragged"] else float(case["kv"])


def work(case):
    op = case["op"]
    if op in ("norm", "rows"):
        m, d = case["rows"], case["cols"]
        moved = 3 * m * d + 4 * m
        if op == "norm":
            moved += (4 * m * d if case["residual"] else 0) + (2 * d if case["weight"] else 0)
        return {"bytes": moved, "flops": (8 if op == "norm" else 3) * m * d}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        moved = m * k + n * k + 4 * (m + n) + 2 * m * n
        moved += (2 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": moved, "flops": 2 * m * n * k}
    seen = _keys_seen(case)
    queries = case["batch"] * case["q"] * case["heads"] * case["d"]
    return {"bytes": 4 * queries + 4 * case["kv_batch"] * seen * case["kv_heads"] * case["d"],
            "flops": 4 * queries * seen}
