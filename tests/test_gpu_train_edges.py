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


def _shifted(t, nbytes=16):
    """The tensor's values in an allocation of its own, nbytes from its start; guard bytes behind it."""
    n = t.numel() * t.element_size()
    flat = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    view = flat[nbytes:nbytes + n].view(t.dtype).view(t.shape)
    view.copy_(t)
    return view, flat


def _guards_kept(view, flat, nbytes=16):
    n = view.numel() * view.element_size()
    return bool((flat[:nbytes] == 0xA5).all() and (flat[nbytes + n:] == 0xA5).all())


def _p(t):
    import ctypes
    return ctypes.c_void_p(t.data_ptr())


def _here():
    import ctypes
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (37, 160), (129, 2880)])
def test_mxfp4_rows_16_bytes_off(api, rows, K, dtype):
    """quantize of an x, and dequantize to an out, that begin 16 bytes off a 32-byte boundary: the same bits."""
    from mixture_experts_ffn_12_b200 import _lib
    L = _lib.load()
    x = torch.randn(rows, K, device="cuda", generator=torch.Generator("cuda").manual_seed(rows)).to(dtype)
    codes, scales = api.quantize_mxfp4(x)
    (xs, _), dt = _shifted(x), _lib.MOE_BF16 if dtype == BF16 else _lib.MOE_F32
    assert xs.data_ptr() % 32 == 16
    c, s = api.quantize_mxfp4(xs)
    assert torch.equal(c, codes) and torch.equal(s, scales)
    (c, cf), (s, sf), (out, of) = _shifted(torch.zeros_like(codes)), _shifted(torch.zeros_like(scales)), _shifted(x * 0)
    assert L.moe_quantize_mxfp4(rows, K, dt, _p(xs), _p(c), _p(s), _here()) == 0
    assert L.moe_dequantize_mxfp4(rows, K, _p(c), _p(s), dt, _p(out), _here()) == 0
    torch.cuda.synchronize()
    assert torch.equal(c, codes) and torch.equal(s, scales)
    assert torch.equal(out, api.dequantize_mxfp4(codes, scales, dtype))
    assert _guards_kept(c, cf) and _guards_kept(s, sf) and _guards_kept(out, of)


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("counts,N,K", [([5], 48, 96), ([70, 0, 333], 400, 1312), ([2600, 2500], 272, 1312)])
def test_linear_16_bytes_off(api, counts, N, K, out_f32):
    """Every tensor of the product 16 bytes off: the bits of aligned ones, nothing written beside y."""
    from train_util import offsets
    G, R = len(counts), sum(counts)
    gen = torch.Generator("cuda").manual_seed(N)
    codes = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(119, 130, (G, N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    x = torch.randn(R, K, device="cuda", generator=gen).to(BF16)
    b = torch.randn(G, N, device="cuda", generator=gen).to(BF16)
    off = offsets(counts)[1]
    w = api.mxfp4_weights(codes, scales)
    want = api.mxfp4_linear(x, w, b, off, out_f32=out_f32)
    ws, wsf = _shifted(torch.zeros(_ws_bytes(G, R, N, K), dtype=torch.uint8, device="cuda"))
    y, yf = _shifted(torch.zeros_like(want))
    tiles, tf = _shifted(torch.zeros_like(w.tiles))
    from mixture_experts_ffn_12_b200 import _lib
    assert _lib.load().moe_mxfp4_weight_tiles(G, N, K, _p(_shifted(scales)[0]), _p(tiles), _here()) == 0
    sw = api.Mxfp4Weights(_shifted(codes)[0], tiles)
    api.mxfp4_linear(_shifted(x)[0], sw, _shifted(b)[0], _shifted(off)[0], out_f32=out_f32, y=y, ws=ws)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert torch.equal(y, want) and torch.equal(tiles, w.tiles)
    assert _guards_kept(y, yf) and _guards_kept(ws, wsf) and _guards_kept(tiles, tf)


def _ws_bytes(G, R, N, K):
    from mixture_experts_ffn_12_b200 import _lib
    return _lib.load().moe_mxfp4_linear_workspace_size(G, R, N, K)


@pytest.mark.parametrize("dtype,grad_f32", [(BF16, False), (BF16, True), (F32, True)], ids=["bf16", "bf16_f32_grads", "f32"])
def test_training_outputs_16_bytes_off(api, dtype, grad_f32):
    """Outputs, gradients and the workspace of the training pass 16 bytes off, through the C ABI: the bits of aligned
    ones, nothing written beside them."""
    import ctypes
    from mixture_experts_ffn_12_b200 import _lib
    from train_util import Block
    L = _lib.load()
    b = Block([37, 0, 190, 300], 176, 208, dtype, True, seed=12)
    cfg, w = b.config(api), b.weights(api)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, w)
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, grad_f32=grad_f32)
    (gu2, guf), (h2, hf), (y2, yf) = (_shifted(torch.zeros_like(t)) for t in (gu, h, y))
    wst = w.c_struct()
    assert L.moe_expert_ffn_train(ctypes.byref(cfg), 0, b.R, _p(b.x), _p(b.off_gpu), ctypes.byref(wst), _p(gu2), _p(h2),
                                  _p(y2), _here()) == 0
    names = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")
    grads = [_shifted(torch.zeros_like(getattr(gr, n))) for n in names]
    gst = api.ExpertGrads(*(g for g, _ in grads)).c_struct()
    n = L.moe_expert_ffn_backward_workspace_size(ctypes.byref(cfg), b.R)
    ws, wsf = _shifted(torch.zeros(n, dtype=torch.uint8, device="cuda"))
    dx2, dxf = _shifted(torch.zeros_like(dx))
    assert L.moe_expert_ffn_backward(ctypes.byref(cfg), 0, b.R, _p(b.x), _p(b.off_gpu), ctypes.byref(wst), _p(gu2), _p(h2),
                                     _p(b.dy), _p(dx2), ctypes.byref(gst), _p(ws), n, _here()) == 0
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    for a, c, f in [(gu, gu2, guf), (h, h2, hf), (y, y2, yf), (dx, dx2, dxf)] + [
            (getattr(gr, name), g, f) for name, (g, f) in zip(names, grads)]:
        assert torch.equal(a, c) and _guards_kept(c, f)
    assert _guards_kept(ws, wsf)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_combine_backward_16_bytes_off(api, dtype):
    T, k, D = 21, 3, 208
    gen = torch.Generator("cuda").manual_seed(3)
    dy, yp = torch.randn(T, D, device="cuda", generator=gen).to(dtype), torch.randn(T * k, D, device="cuda", generator=gen).to(dtype)
    row = torch.randperm(T * k, device="cuda", generator=gen).to(torch.int32).view(T, k)
    tw = torch.rand(T, k, device="cuda", generator=gen)
    cfg = api.make_config(D, 16, 4, k, dtype="bf16" if dtype == BF16 else "f32")
    want = api.combine_backward(cfg, dy, yp, row, tw)
    got = api.combine_backward(cfg, *(_shifted(t)[0] for t in (dy, yp, row, tw)))
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert all(torch.equal(a, c) for a, c in zip(want, got))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("wanted", [(), ("w_down",), ("w_gate", "b_gate"), ("w_up", "w_down", "b_down")], ids=str)
def test_some_gradients_only(api, wanted, dtype):
    """The gradients that `grads` has buffers for, and dx or not: the bits of the whole pass, and no launch for what is
    not wanted (dH, dX and the weights' gradients are one each)."""
    from mixture_experts_ffn_12_b200 import _lib
    from train_util import Block
    b = Block([37, 0, 190], 96, 112, dtype, True, seed=13)
    cfg, w = b.config(api), b.weights(api)
    gu, h, _ = api.expert_ffn_train(cfg, b.x, b.off_gpu, w)
    dx, full = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
    names = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")
    for need_dx in (True, False):
        some = api.ExpertGrads(*(torch.full_like(getattr(full, n), 7.0) if n in wanted else None for n in names))
        before = _lib.load().moe_launch_count()
        dx2, got = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, need_dx=need_dx, grads=some)
        dh = need_dx or "w_gate" in wanted or "w_up" in wanted
        assert _lib.load().moe_launch_count() - before == dh + need_dx + bool(wanted)
        torch.cuda.synchronize()
        assert api.last_device_error() == 0
        assert torch.equal(dx, dx2) if need_dx else dx2 is None
        for n in names:
            assert torch.equal(getattr(got, n), getattr(full, n)) if n in wanted else getattr(got, n) is None
