"""Refusals of the training-pass and MXFP4 entry points (no GPU): the C ABI's before any launch, the binding's
before any library call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from mixture_experts_ffn_12_b200 import _lib, api, build  # noqa: E402

OK, INV, UNS, WS = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
P = ctypes.c_void_p
A = P(4096)          # an aligned address that no rejected call reads
ODD = P(4096 + 8)    # a misaligned one


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def cfg(**kw):
    base = dict(hidden_size=64, intermediate_size=96, num_local_experts=4, num_experts_per_tok=2, swiglu_limit=7.0,
                swiglu_alpha=1.702, dtype=_lib.MOE_BF16, wfmt=_lib.MOE_W_DENSE)
    base.update(kw)
    return ctypes.byref(_lib.MoeConfig(**base))


@pytest.mark.parametrize("args,want", [
    ((0, 64, 1, None, None, None), OK),                  # no rows
    ((-1, 64, 1, A, A, A), INV), (((1 << 31) + 1, 64, 1, A, A, A), INV),
    ((4, 0, 1, A, A, A), INV), ((4, 48, 1, A, A, A), INV), ((4, -32, 1, A, A, A), INV), ((4, (1 << 20) + 32, 1, A, A, A), INV),
    ((4, 64, 2, A, A, A), INV), ((4, 64, 1, None, A, A), INV), ((4, 64, 1, ODD, A, A), INV),
    ((4, 64, 1, A, ODD, A), INV), ((4, 64, 1, A, A, None), INV),
])
def test_quantize(lib, args, want):
    rows, K, dt, x, c, s = args
    assert lib.moe_quantize_mxfp4(rows, K, dt, x, c, s, None) == want
    assert lib.moe_dequantize_mxfp4(rows, K, c, s, dt, x, None) == want


@pytest.mark.parametrize("G,N,K,ok", [(1, 16, 32, True), (256, 2880, 2880, True), (0, 16, 32, False), (257, 16, 32, False),
                                      (1, 8, 32, False), (1, 0, 32, False), (1, 24, 32, False), (1, 16, 48, False),
                                      (1, (1 << 20) + 16, 32, False)])
def test_weight_tile_sizes(lib, G, N, K, ok):
    n = lib.moe_mxfp4_weight_tiles_size(G, N, K)
    assert n == (G * ((N + 127) // 128) * (2 * ((K + 255) // 256)) * 512 if ok else _lib.SIZE_INVALID)
    if not ok:
        assert lib.moe_mxfp4_weight_tiles(G, N, K, A, A, None) == INV
        assert lib.moe_mxfp4_linear_workspace_size(G, 4, N, K) == _lib.SIZE_INVALID
    assert lib.moe_mxfp4_weight_tiles(G, N, K, None, A, None) == INV
    assert lib.moe_mxfp4_weight_tiles(G, N, K, A, ODD, None) == INV


def test_linear(lib):
    def call(G=2, R=3, N=32, K=64, x=A, off=A, wc=A, wt=A, bias=A, f32=0, out=A, ws=A, n=1 << 20):
        return lib.moe_mxfp4_linear(G, R, N, K, x, off, wc, wt, bias, f32, out, ws, n, None)
    assert call(R=0, x=None, out=None, ws=None) == OK
    for bad in (dict(G=0), dict(N=8), dict(K=16), dict(R=-1), dict(R=1 << 31), dict(f32=2), dict(off=None), dict(off=ODD),
                dict(x=None), dict(x=ODD), dict(wc=None), dict(wt=ODD), dict(bias=ODD), dict(out=None)):
        assert call(**bad) == INV, bad
    need = lib.moe_mxfp4_linear_workspace_size(2, 3, 32, 64)
    for bad in (dict(ws=None), dict(ws=ODD), dict(n=need - 1)):
        assert call(**bad) == WS, bad
    assert lib.moe_mxfp4_linear_workspace_size(2, 0, 32, 64) == 0
    assert lib.moe_mxfp4_linear_workspace_size(2, -1, 32, 64) == _lib.SIZE_INVALID


def weights(**kw):
    w = _lib.MoeExpertWeights(*([4096] * 9))
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.byref(w)


def test_train_forward(lib):
    def call(c=None, act=0, T=3, x=A, off=A, w=None, gu=A, h=A, y=A):
        return lib.moe_expert_ffn_train(c or cfg(), act, T, x, off, w or weights(), gu, h, y, None)
    assert call(T=0, x=None, off=None, gu=None, h=None, y=None) == OK
    for bad in (dict(act=2), dict(act=-1), dict(T=-1), dict(T=1 << 30), dict(x=None), dict(x=ODD), dict(off=None), dict(gu=ODD),
                dict(h=None), dict(y=ODD), dict(c=cfg(hidden_size=24)), dict(w=weights(w_gate=None)),
                dict(w=weights(w_down=4104)), dict(w=weights(b_up=4104))):
        assert call(**bad) == INV, bad
    assert lib.moe_expert_ffn_train(cfg(), 0, 3, A, A, None, A, A, A, None) == INV
    for bad in (dict(c=cfg(wfmt=_lib.MOE_W_MXFP4)), dict(c=cfg(h_split=1))):
        assert call(**bad) == UNS, bad


def test_backward(lib):
    def grads(**kw):
        g = _lib.MoeExpertGrads(*([4096] * 6), 0)
        for k, v in kw.items():
            setattr(g, k, v)
        return ctypes.byref(g)

    def call(c=None, act=0, T=3, x=A, off=A, w=None, gu=A, h=A, dy=A, dx=A, g=None, ws=A, n=1 << 30):
        return lib.moe_expert_ffn_backward(c or cfg(), act, T, x, off, w or weights(), gu, h, dy, dx, g or grads(), ws, n, None)
    for bad in (dict(act=7), dict(T=-1), dict(x=None), dict(off=ODD), dict(gu=None), dict(h=ODD), dict(dy=None), dict(dx=ODD),
                dict(w=weights(w_up=None)), dict(g=grads(w_gate=4104)), dict(g=grads(grad_f32=2)),
                dict(g=grads(w_down=None))):        # a bias gradient without its weight's
        assert call(**bad) == INV, bad
    assert lib.moe_expert_ffn_backward(cfg(), 0, 3, A, A, weights(), A, A, A, A, None, A, 1 << 30, None) == INV
    for bad in (dict(c=cfg(wfmt=_lib.MOE_W_MXFP4)), dict(c=cfg(h_split=1))):
        assert call(**bad) == UNS, bad
    need = lib.moe_expert_ffn_backward_workspace_size(cfg(), 3)
    # dgu, rounded up to 256 bytes, then the bias sums of up to ceil(R / 64) + E row tiles, two halves each, and
    # a counter
    assert need == 2304 + (1 + 4) * 2 * 2 * 96 * 4 + 16
    assert lib.moe_expert_ffn_backward_workspace_size(cfg(dtype=_lib.MOE_F32), 3) == 6 * 2 * 96 * 4
    assert lib.moe_expert_ffn_backward_workspace_size(cfg(h_split=1), 3) == _lib.SIZE_INVALID
    for bad in (dict(ws=None), dict(ws=ODD), dict(n=need - 1)):
        assert call(**bad) == WS, bad


def test_combine_backward(lib):
    def call(c=None, T=3, dy=A, yp=A, row=A, w=A, dyp=A, dw=A):
        return lib.moe_combine_backward(c or cfg(), T, dy, yp, row, w, dyp, dw, None)
    assert call(T=0, dy=None) == OK
    for bad in (dict(T=-1), dict(dy=None), dict(yp=ODD), dict(row=None), dict(w=ODD), dict(dyp=None), dict(dw=ODD),
                dict(c=cfg(num_experts_per_tok=9))):
        assert call(**bad) == INV, bad


def test_struct_layout():
    assert ctypes.sizeof(_lib.MoeExpertGrads) == 56 and _lib.MoeExpertGrads.grad_f32.offset == 48


# ---- the binding -------------------------------------------------------------------------------------------
BF16 = torch.bfloat16


def refused(fn, *a, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_mxfp4(lib):
    x = torch.zeros(4, 64, dtype=BF16)
    refused(api.quantize_mxfp4, x.half(), match="bf16 or fp32")
    refused(api.quantize_mxfp4, torch.zeros(4, 40), match="multiple of 32")
    refused(api.quantize_mxfp4, torch.zeros(4, 0), match="multiple of 32")
    refused(api.quantize_mxfp4, torch.zeros(64, 64).t(), match="contiguous")
    refused(api.quantize_mxfp4, x, match="CUDA")
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    refused(api.dequantize_mxfp4, c.int(), s, match="uint8")
    refused(api.dequantize_mxfp4, c, s[:, :1], match="shape")
    refused(api.dequantize_mxfp4, c, s, torch.float16, match="bf16 or fp32")
    wc, ws = torch.zeros(2, 32, 32, dtype=torch.uint8), torch.zeros(2, 32, 2, dtype=torch.uint8)
    refused(api.mxfp4_weights, wc[0], ws, match="uint8")
    refused(api.mxfp4_weights, wc, ws[:1], match="shape")
    w = api.Mxfp4Weights(wc, torch.zeros(lib.moe_mxfp4_weight_tiles_size(2, 32, 64), dtype=torch.uint8))
    off = torch.zeros(3, dtype=torch.int32)
    assert api.check_mxfp4_linear_args(x, w, torch.zeros(2, 32, dtype=BF16), off) == 4
    refused(api.check_mxfp4_linear_args, x, w, match="group_off")
    refused(api.check_mxfp4_linear_args, x.float(), w, None, off, match="dtype")
    refused(api.check_mxfp4_linear_args, x[:, :32].contiguous(), w, None, off, match="shape")
    refused(api.check_mxfp4_linear_args, x, w, torch.zeros(2, 32), off, match="dtype")
    refused(api.check_mxfp4_linear_args, x, w, None, off.long(), match="dtype")
    refused(api.check_mxfp4_linear_args, x, w, None, off, torch.zeros(4, 32), match="dtype")
    refused(api.check_mxfp4_linear_args, x, api.Mxfp4Weights(wc, w.tiles[:-1]), None, off, match="shape")
    cf = api.make_config(64, 96, 2, 1)
    refused(api.quantize_experts, api.make_config(64, 96, 2, 1, dtype="f32"), None, match="bf16")
    refused(api.quantize_experts, cf, None, "int4", match="wfmt")


def test_binding_train(lib):
    E, R, D, F = 2, 6, 32, 48
    z = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    cf = api.make_config(D, F, E, 2)
    off = torch.zeros(E + 1, dtype=torch.int32)
    w = api.ExpertWeights(z(E, F, D), z(E, F, D), z(E, D, F), None, None, z(E, D))
    assert api.check_ffn_train_args(cf, z(R, D), off, w) == 3
    assert api.check_ffn_train_args(cf, z(R, D), off, w, z(R, 2, F), z(R, F), z(R, D)) == 3
    refused(api.check_ffn_train_args, cf, z(5, D), off, w, match="multiple of k")
    refused(api.check_ffn_train_args, cf, z(R, D), off[:2], w, match="shape")
    refused(api.check_ffn_train_args, cf, z(R, D), off, api.ExpertWeights(z(E, F, D), z(E, F, D), z(E, F, D), None, None, None),
            match="w_down")
    refused(api.check_ffn_train_args, cf, z(R, D), off, w, z(R, F, 2), z(R, F), z(R, D), match="gu")
    refused(api.check_ffn_train_args, cf, z(R, D), off, w, z(R, 2, F), None, z(R, D), match="h is required")
    refused(api.check_ffn_train_args, api.make_config(D, 64, E, 2, wfmt="mxfp4"), z(R, D), off, w, match="dense")
    refused(api.expert_ffn_train, cf, z(R, D), off, w, act="gelu", match="act")
    refused(api.expert_ffn_train, cf, z(R, D), off, w, match="CUDA")
    refused(api.expert_ffn_backward, cf, z(R, D), off, w, z(R, 2, F), z(R, F), None, match="dy_perm")
    bad = api.ExpertGrads(z(E, F, D), z(E, F, D), z(E, F, D))
    refused(api.expert_ffn_backward, cf, z(R, D), off, w, z(R, 2, F), z(R, F), z(R, D), grads=bad, match="grads.w_down")
    refused(api.expert_ffn_backward, cf, z(R, D), off, w, z(R, 2, F), z(R, F), z(R, D), ws=z(64, 64).t(), match="contiguous")
    ros, tw = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    refused(api.combine_backward, cf, z(3, D).float(), z(R, D), ros, tw, match="dy: dtype")
    refused(api.combine_backward, cf, z(3, D), z(R, D), ros, tw, match="CUDA")
