"""MXFP4 quantization and the MXFP4 x MXFP4 linear layer on the GPU (marked gpu) against the fp64 oracle.

Codes, scales and dequantized values are bit-exact.  The product's operands are then exact numbers, so its
error is that of fp32 sums (``sum_bound``) and one rounding of the output.
"""
import numpy as np
import pytest

from oracle import train as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_util import HALF, offsets, sum_bound, values, within  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


def _rows(rows, K, dtype, seed):
    rng = np.random.default_rng(seed)
    a = rng.normal(0, 1, (max(rows, 4), K)) * np.exp2(rng.integers(-30, 30, (max(rows, 4), 1)))
    a[0, :32] = 0.0
    a[1, :32] = np.resize([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -6.0], 32) * 2.0 ** -9   # ties
    a[2, :32] = 2.0 ** -130                                    # below the smallest scale's range
    a[3, :32] = np.ldexp(1.0, np.arange(-16, 16))              # one block over many binades
    a[0, 40 % K], a[1, 50 % K] = 2.0 ** -127, -(2.0 ** -126)   # subnormal values at the smallest scale, and next to it
    if K >= 96:
        a[0, 32:64] = 2.0 ** -127 * np.resize([1, 2, 3, 0.5, -1, 0.25], 32)   # a block of them
        a[2, 32:64] = 2.5e38                                   # largest magnitudes
        a[3, 40], a[3, 70] = np.inf, np.nan
    return torch.from_numpy(a[:rows].astype(np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (129, 160), (37, 2880)])
def test_quantize_and_back_bit_exact(api, rows, K, dtype):
    x = _rows(rows, K, dtype, rows)
    codes, scales = api.quantize_mxfp4(x)
    torch.cuda.synchronize()
    c, s = O.quantize_mxfp4(values(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), O.pack(c))
    for out in (BF16, F32):
        v = api.dequantize_mxfp4(codes, scales, out)
        assert v.dtype == out and np.array_equal(values(v), O.mxfp4_values(c, s), equal_nan=True)


def test_quantize_shapes(api):
    x = _rows(24, 64, BF16, 0).view(2, 3, 4, 64)
    codes, scales = api.quantize_mxfp4(x)
    assert codes.shape == (2, 3, 4, 32) and scales.shape == (2, 3, 4, 2)
    assert api.quantize_mxfp4(x[:0])[0].shape == (0, 3, 4, 32)
    assert api.dequantize_mxfp4(codes[:0], scales[:0]).shape == (0, 3, 4, 64)


@pytest.mark.parametrize("G,N,K", [(1, 16, 32), (2, 144, 96), (3, 272, 288), (1, 128, 2880)])
def test_weight_tiles(api, G, N, K):
    s = np.random.default_rng(N).integers(0, 256, (G, N, K // 32)).astype(np.uint8)
    codes = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda")
    w = api.mxfp4_weights(codes, torch.from_numpy(s).cuda())
    assert np.array_equal(w.tiles.cpu().numpy(), O.scale_tiles(s))


def _weights(G, N, K, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (G, N, K // 2)).astype(np.uint8)
    scales = rng.integers(119, 130, (G, N, K // 32)).astype(np.uint8)
    return codes, scales, O.mxfp4_values(O.unpack(codes), scales)


def _check_linear(api, counts, N, K, bias, out_f32, group=True, seed=0):
    G, R = len(counts), int(sum(counts))
    rng = np.random.default_rng(seed + 1)
    codes, scales, wv = _weights(G, N, K, seed)
    off, off_gpu = offsets(counts)
    x = torch.from_numpy((rng.normal(0, 1, (R, K)) * np.exp2(rng.integers(-4, 4, (R, 1)))).astype(np.float32)).cuda().to(BF16)
    b = torch.from_numpy(rng.normal(0, 3, (G, N)).astype(np.float32)).cuda().to(BF16) if bias else None
    w = api.mxfp4_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    y = api.mxfp4_linear(x, w, b, off_gpu if group else None, out_f32=out_f32)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert y.dtype == (F32 if out_f32 else BF16)
    xq = O.mxfp4_values(*O.quantize_mxfp4(values(x)))
    want, mags = O.rows_times(xq, wv, off), O.rows_times(np.abs(xq), np.abs(wv), off)
    if bias:
        e = O.per_row(off, R)
        want, mags = want + values(b)[e], mags + np.abs(values(b)[e])
    err = sum_bound(K, mags)
    within("y", values(y), want, err + HALF[y.dtype] * (np.abs(want) + err))


# every second 192-column tile starts inside a 128-row scale chunk; K ends inside the 256-element stages
LINEAR = [([1], 16, 32), ([1], 208, 64), ([7], 192, 256), ([130], 400, 288), ([129], 576, 544), ([300], 2880, 96),
          ([3], 48, 2880), ([0, 1, 127, 0, 128, 129, 300, 5, 0], 336, 416), ([2, 0, 5, 1], 2880, 2880)]


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("counts,N,K", LINEAR, ids=[f"G{len(c)}_R{sum(c)}_N{n}_K{k}" for c, n, k in LINEAR])
def test_linear(api, counts, N, K, out_f32):
    _check_linear(api, counts, N, K, bias=True, out_f32=out_f32, seed=N + K)


def test_linear_without_groups_or_bias(api):
    _check_linear(api, [77], 320, 352, bias=False, out_f32=True, group=False)


def test_linear_empty_and_rows_of_no_group(api):
    codes, scales, _ = _weights(2, 32, 64, 5)
    w = api.mxfp4_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    off = torch.tensor([0, 3, 5], dtype=torch.int32).cuda()
    assert api.mxfp4_linear(torch.empty((0, 64), dtype=BF16, device="cuda"), w, None, off * 0).shape == (0, 32)
    x = torch.randn(9, 64, device="cuda").to(BF16)
    y = torch.full((9, 32), 5.0, dtype=BF16, device="cuda")
    api.mxfp4_linear(x, w, None, off, y=y)
    torch.cuda.synchronize()
    assert (y[5:] == 5.0).all()
    assert torch.equal(y[:5], api.mxfp4_linear(x[:5].contiguous(), w, None, off))


def test_linear_non_finite_row_stays_alone(api):
    """A row with an infinity and one with a NaN read as NaN (their blocks' scale is the E8M0 NaN); all
    others keep their bits."""
    codes, scales, _ = _weights(1, 224, 288, 6)
    w = api.mxfp4_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = torch.randn(140, 288, device="cuda").to(BF16)
    clean = api.mxfp4_linear(x, w)
    x[3, 287], x[130, 0] = float("inf"), float("nan")
    got = api.mxfp4_linear(x, w)
    torch.cuda.synchronize()
    assert torch.isnan(got[3]).all() and torch.isnan(got[130]).all()
    keep = [i for i in range(140) if i not in (3, 130)]
    assert torch.equal(got[keep], clean[keep])


def test_quantized_layer(api):
    """MoELayer.quantized(): the layer whose weights are the values of the quantized ones, bit for bit."""
    import workloads as W
    from parity_util import layer_for
    spec = W.tiny_spec(T=130, D=64, E=6, k=2, F=96, dtype="bf16", cfg_id=811)
    layer = layer_for(spec)
    d = api.upload_layer(layer)
    dense = api.MoELayer(api.config_from_spec(spec), d["w_router"], d["b_router"], api.expert_weights_from(d))
    q = dense.quantized()
    values_of = lambda c, s: api.dequantize_mxfp4(c, s)  # noqa: E731
    e = q.experts
    same = api.ExpertWeights(values_of(e.w_gate, e.s_gate), values_of(e.w_up, e.s_up), values_of(e.w_down, e.s_down),
                             e.b_gate, e.b_up, e.b_down)
    ref = api.MoELayer(dense.cfg, d["w_router"], d["b_router"], same)
    y, yr = q(d["x"]), ref(d["x"])
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    rms = yr.float().square().mean().sqrt()
    # same operands; the two GEMM kernels add in another order, and h and y are rounded to bf16 in each
    assert ((y.float() - yr.float()).abs().max() / rms).item() < 2e-2
