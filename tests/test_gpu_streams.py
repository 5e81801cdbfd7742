"""The helpers' ``stream`` argument, a stream that is not the current one: the
whole call runs there, and its outputs and workspaces are that stream's memory.

A block that the current stream has given up goes back to the current stream's
pool while its kernels may still use it, so a call on another stream that took
its outputs from there would write into memory in use.  Each case frees a block
of its output's size on the current stream and looks where the output lies; the
results equal those of a call on the current stream.
"""
import pytest

pytestmark = pytest.mark.gpu

M, K, N, HEADS = 1536, 1024, 2048, 8  # outputs of a megabyte and more: blocks of their own


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_diffusion_transformer_nvfp4_b200 as w
    w.lib()
    return w


@pytest.fixture(scope="module")
def made(w4):
    """Inputs of every helper."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()

    d = {"x": normal(M, K), "r": normal(M, K), "w": normal(N, K)}
    d["qa"], d["pw"] = w4.quantize_act(d["x"]), w4.pack_weight(d["w"])
    d["fa"], d["fw"] = w4.quantize_rows_fp8(d["x"]), w4.pack_weight_fp8(d["w"])
    d["q8"], d["vt"] = w4.quantize_fp8(d["x"]), w4.quantize_fp8(d["x"], transpose=True)
    d["rope"] = torch.rand(M, 128, device="cuda", generator=g)
    d["next_t"] = torch.full((1,), 0.01, device="cuda")
    return d


CALLS = {
    "quantize_act": lambda w4, d, s: [getattr(w4.quantize_act(d["x"], stream=s), n) for n in ("Xq", "Xsf", "t_x")],
    "pack_weight": lambda w4, d, s: [getattr(w4.pack_weight(d["w"], stream=s), n) for n in ("Wq", "Wsf", "t_w")],
    "gemm": lambda w4, d, s: [w4.gemm(d["qa"], d["pw"], stream=s)],
    "gemm_swiglu": lambda w4, d, s: list(w4.gemm_swiglu(d["qa"], d["pw"], 1024, stream=s)),
    "gemm_rope": lambda w4, d, s: [w4.gemm_rope(d["qa"], d["pw"], d["rope"], 1024, 128, stream=s)[0]],
    "gemm_quantize_next": lambda w4, d, s: [t for t in w4.gemm_quantize_next(d["qa"], d["pw"], d["next_t"], stream=s)
                                            if t is not None],
    "linear": lambda w4, d, s: [w4.linear(d["x"], d["pw"], stream=s)],
    "sf_rowmajor": lambda w4, d, s: [w4.sf_rowmajor(d["qa"].Xsf, M, K, stream=s)],
    "quantize_fp8": lambda w4, d, s: [getattr(w4.quantize_fp8(d["x"], stream=s), n) for n in ("codes", "scale")],
    "attention": lambda w4, d, s: [w4.attention(d["q8"], d["q8"], d["vt"], HEADS, stream=s)],
    "quantize_rows_fp8": lambda w4, d, s: [getattr(w4.quantize_rows_fp8(d["x"], stream=s), n)
                                           for n in ("codes", "scales")],
    "rms_norm_fp8": lambda w4, d, s: (lambda a, h: [a.codes, a.scales, h])(
        *w4.rms_norm_fp8(d["x"], residual=d["r"], stream=s)),
    "pack_weight_fp8": lambda w4, d, s: [getattr(w4.pack_weight_fp8(d["w"], stream=s), n) for n in ("codes", "scales")],
    "linear_fp8": lambda w4, d, s: [w4.linear_fp8(d["fa"], d["fw"], stream=s)],
    "cross_attention": lambda w4, d, s: [w4.cross_attention(d["x"], d["r"], d["r"], HEADS, stream=s)],
}


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_outputs_belong_to_the_given_stream(w4, made, name, kind):
    import torch
    call = CALLS[name]
    want = call(w4, made, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = {torch.empty_like(t).data_ptr() for t in want}  # blocks of the outputs' sizes, given up at once
    got = call(w4, made, side if kind == "stream" else side.cuda_stream)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    side.synchronize()
    assert not freed & {t.data_ptr() for t in got}
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert w4.w4a4_device_status() == 0


def test_a_chain_on_another_stream_while_this_one_works(w4, made):
    """Temporaries of a busy current stream are not what the other one writes."""
    import torch
    side = torch.cuda.Stream()

    def chain(s):
        a, h = w4.rms_norm_fp8(made["x"], residual=made["r"], stream=s)
        y = w4.linear_fp8(a, made["fw"], stream=s)
        o = w4.cross_attention(y, y, y, heads=2 * HEADS, stream=s)
        return [a.codes, h, y, o]

    want = chain(None)
    torch.cuda.synchronize()
    for _ in range(5):
        busy = made["x"].float()
        for _ in range(20):  # each step gives its input's block back while the kernel that reads it is queued
            busy = busy * 1.5 - 0.5 * busy
        got = chain(side)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        torch.testing.assert_close(busy, made["x"].float())


def test_default_stream_by_its_handles(w4, made):
    import torch
    want = w4.quantize_rows_fp8(made["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (0, 1):
        with torch.cuda.stream(side):
            a = w4.quantize_rows_fp8(made["x"], stream=handle)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert torch.equal(a.codes, want.codes) and torch.equal(a.scales, want.scales)
