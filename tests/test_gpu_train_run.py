"""The training and MXFP4 operators as they are used (marked gpu): one step of an expert layer end to end, on
streams, in captured graphs, two at a time, at odd addresses, and with waits that run out."""
import ctypes

import numpy as np
import pytest

import workloads as W
from oracle import moe_oracle as MO
from oracle import train as O
from parity_util import TOL_Y, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_util import HALF, Block, backward_ws, sum_bound, values, within  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


def _ok(api):
    torch.cuda.synchronize()
    assert api.last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_then_mxfp4(api, dtype):
    """Router and dispatch, the block forward, combine; combine and block backward, dx summed over the slots;
    a step on the weights; the stepped weights in MXFP4 through the layer and through mxfp4_linear."""
    T, D, E, k, F = 170, 64, 5, 2, 96
    spec = W.tiny_spec(T=T, D=D, E=E, k=k, F=F, dtype=dtype, cfg_id=821, router_w_std=0.2)
    layer = W.make_layer(spec, seed=0, logits_fn=lambda l: MO.router_logits(l["x"], l["w_router"], l["b_router"]))
    d = api.upload_layer(layer)
    cfg, w = api.config_from_spec(spec), api.expert_weights_from(d)
    dt = api.torch_dtype(cfg)
    half = HALF[dt]
    ids, tw = api.router_topk(cfg, d["x"], d["w_router"], d["b_router"])
    p = api.permute(cfg, ids, d["x"])
    off = p["expert_off"].cpu().numpy()
    gu, h, y_perm = api.expert_ffn_train(cfg, p["x_perm"], p["expert_off"], w)
    y = api.combine(cfg, y_perm, p["row_of_slot"], tw)
    # the block's output against the plain layer of the same weights (the layer's own bound)
    ref = MO.layer_tokens(layer, np.arange(T), k, spec.limit, spec.alpha)["y"]
    rms = np.sqrt(np.mean(ref ** 2))
    assert np.max(np.abs(f64(y) - ref)) / rms <= TOL_Y[dtype] + half * np.max(np.abs(ref)) / rms
    dy = torch.randn(T, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dt)
    dy_perm, dtw = api.combine_backward(cfg, dy, y_perm, p["row_of_slot"], tw)
    dx_perm, gr = api.expert_ffn_backward(cfg, p["x_perm"], p["expert_off"], w, gu, h, dy_perm)
    dx = api.combine(cfg, dx_perm, p["row_of_slot"], torch.ones_like(tw))     # the slots' gradients, summed
    _ok(api)
    row, twv = p["row_of_slot"].cpu().numpy(), values(tw)
    rdyp, rdw = O.combine_backward(values(dy), values(y_perm), row, twv)
    within("dy_perm", values(dy_perm), rdyp, np.abs(rdyp) * (half + 2.0 ** -23) + 1e-40)
    within("dtopk_w", values(dtw), rdw, sum_bound(D, O.combine_backward(np.abs(values(dy)), np.abs(values(y_perm)), row, twv)[1]))
    xp, dyp, hv = values(p["x_perm"]), values(dy_perm), values(h)
    want = O.outer_sums(dyp, hv, off)
    err = sum_bound(T * k, O.outer_sums(np.abs(dyp), np.abs(hv), off))
    within("dw_down", values(gr.w_down), want, err + half * (np.abs(want) + err))
    dxv = values(dx_perm)[row]                                                 # [T, k, D]
    within("dx", values(dx), dxv.sum(1), np.abs(dxv).sum(1) * (k * 2.0 ** -23) + half * np.abs(dxv.sum(1)) + 1e-40)
    assert np.all(xp == values(d["x"])[p["slot_of_row"].cpu().numpy() // k])
    # a step, then the weights in MXFP4
    new = api.ExpertWeights(*((t.float() - 1e-3 * g.float()).to(BF16) for t, g in
                              ((w.w_gate, gr.w_gate), (w.w_up, gr.w_up), (w.w_down, gr.w_down))),
                            *(b.to(BF16) for b in (w.b_gate, w.b_up, w.b_down)))
    bcfg = api.make_config(D, F, E, k, spec.limit, spec.alpha)
    qcfg, q = api.quantize_experts(bcfg, new)
    x16, wr, br = d["x"].to(BF16), d["w_router"].to(BF16), d["b_router"].to(BF16)
    yq = api.layer_forward(qcfg, x16, wr, br, q)
    _ok(api)
    vals = {n: f64(api.dequantize_mxfp4(getattr(q, "w_" + n), getattr(q, "s_" + n))) for n in ("gate", "up", "down")}
    bits = lambda t: W.f32_to_bf16_bits(f64(t).astype(np.float32))  # noqa: E731
    qlayer = dict(x=bits(x16), w_router=bits(wr), b_router=bits(br), b_gate=bits(new.b_gate), b_up=bits(new.b_up),
                  b_down=bits(new.b_down), **{"w_" + n: W.f32_to_bf16_bits(v.astype(np.float32)) for n, v in vals.items()})
    qref = MO.layer_tokens(qlayer, np.arange(T), k, spec.limit, spec.alpha)["y"]
    rms = np.sqrt(np.mean(qref ** 2))
    assert np.max(np.abs(f64(yq) - qref)) / rms <= TOL_Y["mxfp4"]
    # the down projection of the same weights, 4 bits x 4 bits
    h16 = h.to(BF16)
    lin = api.mxfp4_linear(h16, api.mxfp4_weights(q.w_down, q.s_down), new.b_down, p["expert_off"], out_f32=True)
    _ok(api)
    hq = O.mxfp4_values(*O.quantize_mxfp4(values(h16)))
    e = O.per_row(off, T * k)
    want = O.rows_times(hq, vals["down"], off) + f64(new.b_down)[e]
    mags = O.rows_times(np.abs(hq), np.abs(vals["down"]), off) + np.abs(f64(new.b_down))[e]
    within("linear", values(lin), want, sum_bound(F, mags) + HALF[F32] * np.abs(want))


def _ops(api, seed):
    """Each operator as (call on static inputs, outputs): the inputs' tensors are returned to be refilled."""
    b = Block([70, 0, 33, 150], 96, 112, BF16, True, seed=seed)
    f = Block([20, 45], 48, 64, F32, True, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    cfg, fcfg = b.config(api), f.config(api)
    w, fw = b.weights(api), f.weights(api)
    codes = torch.randint(0, 256, (4, 112, 48), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(119, 128, (4, 112, 3), dtype=torch.uint8, device="cuda", generator=gen)
    mw = api.mxfp4_weights(codes, scales)
    ccfg = api.make_config(96, 16, 8, 2)
    y_perm = torch.randn(52, 96, device="cuda", generator=gen).to(BF16)
    row = torch.randperm(52, device="cuda", generator=gen).to(torch.int32).view(26, 2)
    tw = torch.rand(26, 2, device="cuda", generator=gen)
    dy = torch.randn(26, 96, device="cuda", generator=gen).to(BF16)

    def block(bl, c, ww):
        gu, h, y = api.expert_ffn_train(c, bl.x, bl.off_gpu, ww)
        dx, gr = api.expert_ffn_backward(c, bl.x, bl.off_gpu, ww, gu, h, bl.dy)
        return [gu, h, y, dx, gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down]

    def quant():
        c, s = api.quantize_mxfp4(b.x)
        return [c, s, api.dequantize_mxfp4(c, s)]
    calls = dict(block=lambda: block(b, cfg, w), block_f32=lambda: block(f, fcfg, fw), quantize=quant,
                 linear=lambda: [api.mxfp4_linear(b.x, mw, None, b.off_gpu)],
                 combine=lambda: list(api.combine_backward(ccfg, dy, y_perm, row, tw)))
    return calls, [b.x, b.dy, f.x, f.dy, y_perm, dy]


NAMES = ["block", "block_f32", "quantize", "linear", "combine"]


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(api, name):
    """Captured on a side stream, replayed on new values in the same buffers: the eager call's bits."""
    calls, inputs = _ops(api, 1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls[name]()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = calls[name]()
    for t in inputs:
        t.copy_(torch.randn(t.shape, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    want = calls[name]()
    _ok(api)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_at_once(api):
    """Every operator on two streams at a time, many calls in flight: each result is that of a quiet call."""
    sets = [_ops(api, 3)[0], _ops(api, 4)[0]]
    want = [{n: [o.clone() for o in c[n]()] for n in NAMES} for c in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for n in NAMES:
                    got[i].append((n, sets[i][n]()))
    _ok(api)
    for i in range(2):
        for n, outs in got[i]:
            for a, b in zip(outs, want[i][n]):
                assert torch.equal(a, b), (i, n)


def test_addresses_16_bytes_off(api):
    """Tensors that begin 16 bytes into their allocation are taken and give the same bits; 8 bytes are refused."""
    def shifted(t, nbytes):
        flat = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
        view = flat[nbytes:nbytes + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view
    b = Block([37, 90], 96, 112, BF16, True, seed=5)
    cfg, w = b.config(api), b.weights(api)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, w)
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
    sw = api.ExpertWeights(*(shifted(t, 16) for t in (b.wg, b.wu, b.wd, b.bg, b.bu, b.bd)))
    x, dy, off = shifted(b.x, 16), shifted(b.dy, 16), shifted(b.off_gpu, 16)
    gu2, h2, y2 = api.expert_ffn_train(cfg, x, off, sw)
    dx2, gr2 = api.expert_ffn_backward(cfg, x, off, sw, shifted(gu, 16), shifted(h, 16), dy)
    _ok(api)
    for a, c in ((gu, gu2), (h, h2), (y, y2), (dx, dx2), (gr.w_gate, gr2.w_gate), (gr.b_up, gr2.b_up)):
        assert torch.equal(a, c)
    c, s = api.quantize_mxfp4(b.x)
    c2, s2 = api.quantize_mxfp4(x)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    assert torch.equal(api.dequantize_mxfp4(shifted(c, 16), shifted(s, 16)), api.dequantize_mxfp4(c, s))
    with pytest.raises(api.MoeError):
        api.quantize_mxfp4(shifted(b.x, 8))
    with pytest.raises(api.MoeError):
        api.expert_ffn_train(cfg, shifted(b.x, 8), b.off_gpu, w)


def test_one_gradient_through_the_abi(api):
    """Only the down projection's gradient is asked for, through the C ABI: no other is computed or written."""
    from mixture_experts_ffn_12_b200 import _lib
    for dtype in (BF16, F32):
        b = Block([40, 77], 64, 80, dtype, True, seed=6)
        cfg, w = b.config(api), b.weights(api)
        gu, h, _ = api.expert_ffn_train(cfg, b.x, b.off_gpu, w)
        _, want = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
        out = torch.zeros_like(want.w_down)
        g = _lib.MoeExpertGrads(None, None, out.data_ptr(), None, None, None, 1 if dtype == F32 else 0)
        ws, _ = backward_ws(cfg, b)
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        before = _lib.load().moe_launch_count()
        assert _lib.load().moe_expert_ffn_backward(
            ctypes.byref(cfg), 0, b.R, p(b.x), p(b.off_gpu), ctypes.byref(w.c_struct()), p(gu), p(h), p(b.dy), None,
            ctypes.byref(g), p(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        _ok(api)
        assert _lib.load().moe_launch_count() - before == 1
        assert torch.equal(out, want.w_down)


def test_offsets_out_of_range_are_reported(api):
    """expert_off with an entry beyond the rows, and one that is not ascending: reported, no access out of range."""
    from mixture_experts_ffn_12_b200 import _lib
    b = Block([40, 30, 58], 64, 80, BF16, True, seed=7)
    f = Block([40, 30, 58], 64, 80, F32, True, seed=7)
    codes = torch.zeros((3, 80, 32), dtype=torch.uint8, device="cuda")
    mw = api.mxfp4_weights(codes, torch.full((3, 80, 2), 127, dtype=torch.uint8, device="cuda"))
    for bad in ([0, 40, 1000, 128], [0, 100, 30, 128], [-5, 40, 70, 128]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for bl in (b, f):
            cfg, w = bl.config(api), bl.weights(api)
            gu, h, _ = api.expert_ffn_train(cfg, bl.x, off, w)
            torch.cuda.synchronize()
            assert api.last_device_error() == _lib.MOE_ERR_DEVICE_BOUNDS
            api.expert_ffn_backward(cfg, bl.x, off, w, torch.zeros_like(gu), torch.zeros_like(h), bl.dy)
            torch.cuda.synchronize()
            assert api.last_device_error() == _lib.MOE_ERR_DEVICE_BOUNDS
        api.mxfp4_linear(b.x, mw, None, off)
        torch.cuda.synchronize()
        assert api.last_device_error() == _lib.MOE_ERR_DEVICE_BOUNDS
    assert api.last_device_error() == 0


def test_zz_waits_that_run_out_are_reported(api):
    """With a wait limit of 1 ns the pipelines give up: the error word says so, and the next calls are right."""
    from mixture_experts_ffn_12_b200 import _lib
    calls, _ = _ops(api, 8)
    want = {n: [o.clone() for o in calls[n]()] for n in ("block", "linear")}
    _ok(api)
    for n in ("block", "linear"):
        api.set_wait_limit_ns(1)
        try:
            calls[n]()
            torch.cuda.synchronize()
            status = api.last_device_error()
        finally:
            api.set_wait_limit_ns(0)
        assert status == _lib.MOE_ERR_TIMEOUT
        got = calls[n]()
        _ok(api)
        for a, c in zip(got, want[n]):
            assert torch.equal(a, c)
