"""Corners of the training and MXFP4 operators on the GPU (marked gpu): values next to a clip's bound,
addresses and pointers that only the C ABI can be given, waits that run out with many tiles under way."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


# products and sums that are exact in fp32, so that the sign of g is beyond doubt: (x, w, bias, g), g too small for
# bf16 (its smallest value is 2^-133) in all but the last two
TINY_GATES = [(2.0 ** -70, -2.0 ** -70, 0.0, -2.0 ** -140), (2.0 ** -70, 2.0 ** -70, 0.0, 2.0 ** -140),
              (2.0 ** -60 * (1 + 2.0 ** -7), -2.0 ** -73, 2.0 ** -133, -2.0 ** -140),
              (2.0 ** -67, -2.0 ** -67, 0.0, -2.0 ** -134), (0.0, 0.0, 0.0, 0.0), (1.0, -2.0 ** -133, 0.0, -2.0 ** -133),
              (1.0, -1.0, 0.0, -1.0)]


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("x0,w0,b0,g", TINY_GATES)
def test_gate_next_to_its_lower_bound(api, x0, w0, b0, g, act):
    """A negative g is stored as a negative number even where bf16 would round it to -0, so that the clip at 0 stops
    its gradient as the forward pass clipped it; without that clip (SiLU) it is rounded to nearest."""
    D = F = 16
    x = torch.zeros(1, D, dtype=BF16, device="cuda")
    x[0, 0] = x0
    wg = torch.zeros(1, F, D, dtype=BF16, device="cuda")
    wg[:, :, 0] = w0
    ones = lambda *s: torch.ones(s, dtype=BF16, device="cuda")  # noqa: E731
    w = api.ExpertWeights(wg, ones(1, F, D), ones(1, D, F), ones(1, F) * b0, ones(1, F), None)
    cfg = api.make_config(D, F, 1, 1)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    gu, h, _ = api.expert_ffn_train(cfg, x, off, w, act=act)
    _, gr = api.expert_ffn_backward(cfg, x, off, w, gu, h, ones(1, D), act=act)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    got = gu[0, 0].double()
    if act == "swiglu" and g < 0:
        assert (got < 0).all()
        assert (got - g).abs().max().item() <= 2.0 ** -133          # at most a step of bf16's smallest values
        assert (gr.b_gate == 0).all() and (gr.w_gate == 0).all()
    else:
        assert (got == torch.tensor(g, dtype=F32).to(BF16).double().item()).all()
        assert (gr.b_gate != 0).all()                               # f'(0) = 1/2; f' > 0 at -1 as well


def test_waits_that_run_out_with_several_tiles_a_pair(api):
    """With a wait limit of 1 ns every kernel that has several tiles a CTA pair gives up: the calls return soon, the
    error word says so, and the next calls on the same buffers have the right bits."""
    import time
    from mixture_experts_ffn_12_b200 import _lib
    from train_util import Block
    b = Block([700, 0, 1300, 345, 90], 2880, 2048, BF16, True, seed=11)
    cfg, w = b.config(api), b.weights(api)
    gen = torch.Generator("cuda").manual_seed(11)
    codes = torch.randint(0, 256, (5, 2048, 2880), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(119, 128, (5, 2048, 180), dtype=torch.uint8, device="cuda", generator=gen)
    mw = api.mxfp4_weights(codes, scales)
    x2 = torch.randn(b.R, 5760, device="cuda", generator=gen).to(BF16)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, w)

    def forward():
        return list(api.expert_ffn_train(cfg, b.x, b.off_gpu, w))

    def backward():
        dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
        return [dx, gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down]

    def linear():
        return [api.mxfp4_linear(x2, mw, None, b.off_gpu)]
    for call in (forward, backward, linear):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        assert api.last_device_error() == 0
        api.set_wait_limit_ns(1)
        t0 = time.monotonic()
        try:
            call()
            torch.cuda.synchronize()
            status = api.last_device_error()
        finally:
            api.set_wait_limit_ns(0)
        assert status == _lib.MOE_ERR_TIMEOUT, call.__name__
        assert time.monotonic() - t0 < 30          # three launches, each drained within a few seconds
        got = call()
        torch.cuda.synchronize()
        assert api.last_device_error() == 0
        for a, c in zip(got, want):
            assert torch.equal(a, c), call.__name__
