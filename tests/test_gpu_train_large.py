"""The training and MXFP4 calls on tensors of more than 2^32 elements (marked gpu): their last rows against calls on
those rows alone, whose bits they must have (a row's sums do not depend on the rows beside it), and the weight
gradients against fp64."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_check import within  # noqa: E402
from train_util import HALF, offsets, sum_bound  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    yield A
    torch.cuda.empty_cache()


def _ok(api):
    torch.cuda.synchronize()
    assert api.last_device_error() == 0


def _randn(seed, *shape, dtype=BF16):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=gen, dtype=dtype)


def test_mxfp4(api):
    R, K, N, last = 1_500_001, 2880, 32, 777
    x = _randn(1, R, K)
    codes, scales = api.quantize_mxfp4(x)
    values = api.dequantize_mxfp4(codes, scales)
    c, s = api.quantize_mxfp4(x[-last:])
    assert torch.equal(codes[-last:], c) and torch.equal(scales[-last:], s)
    assert torch.equal(values[-last:], api.dequantize_mxfp4(c, s))
    assert torch.equal(values[:last], api.dequantize_mxfp4(*api.quantize_mxfp4(x[:last])))
    del values
    gen = torch.Generator("cuda").manual_seed(2)
    w = api.mxfp4_weights(torch.randint(0, 256, (3, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen),
                          torch.randint(119, 128, (3, N, K // 32), dtype=torch.uint8, device="cuda", generator=gen))
    y = api.mxfp4_linear(x, w, None, offsets([700_000, 1, R - 700_001])[1])
    tail = api.mxfp4_linear(x[-last:], w, None, offsets([0, 0, last])[1])
    _ok(api)
    assert torch.equal(y[-last:], tail)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_expert_block(api, dtype):
    # gu and (dg, du) have 2 R F elements
    D, F, last = (64, 2048, 700) if dtype == BF16 else (16, 2048, 300)
    counts = [400_001, 0, 700_000 - last, last]
    R = sum(counts)
    x, dy = _randn(3, R, D, dtype=dtype), _randn(4, R, D, dtype=dtype)
    E = len(counts)
    wg, wu = (_randn(i, E, F, D, dtype=dtype) * D ** -0.5 for i in (5, 6))
    w = api.ExpertWeights(wg, wu, _randn(7, E, D, F, dtype=dtype) * F ** -0.5, *(_randn(i, E, n, dtype=dtype) * 0.2 for i, n in
                                                                                 ((8, F), (9, F), (10, D))))
    cfg = api.make_config(D, F, E, 1, 2.0, dtype="bf16" if dtype == BF16 else "f32")
    off = offsets(counts)[1]
    gu, h, y = api.expert_ffn_train(cfg, x, off, w)
    dx, gr = api.expert_ffn_backward(cfg, x, off, w, gu, h, dy, grad_f32=True)
    # the last expert's rows, in a call on them alone: the same tiles of at most 256 (128) rows, or others
    at = slice(R - last, R)
    one = offsets([0, 0, 0, last])[1]
    gu1, h1, y1 = api.expert_ffn_train(cfg, x[at], one, w)
    dx1, gr1 = api.expert_ffn_backward(cfg, x[at], one, w, gu1, h1, dy[at], grad_f32=True)
    _ok(api)
    for a, b in ((gu[at], gu1), (h[at], h1), (y[at], y1), (dx[at], dx1)):
        assert torch.equal(a, b)
    for n in ("w_gate", "w_up", "w_down", "b_down"):
        assert torch.equal(getattr(gr, n)[3], getattr(gr1, n)[3])
        assert (getattr(gr, n)[1] == 0).all()
    # dy^T h of the largest expert
    want, mags = torch.zeros(D, F, dtype=torch.float64, device="cuda"), torch.zeros(D, F, dtype=torch.float64, device="cuda")
    for r in range(counts[0], R - last, 50_000):
        c = slice(r, min(r + 50_000, R - last))
        a, b = dy[c].double(), h[c].double()
        want += a.T @ b
        mags += a.abs().T @ b.abs()
    err = sum_bound(counts[2], mags)
    within("w_down", gr.w_down[2], want, err + HALF[F32] * (want.abs() + err))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_combine_backward(api, dtype):
    T, k, D, last = 380_000, 4, 2880, 500
    dy, yp = _randn(11, T, D, dtype=dtype), _randn(12, T * k, D, dtype=dtype)
    row = torch.arange(T * k, device="cuda", dtype=torch.int32).flip(0).view(T, k)      # the last tokens at the first rows
    tw = torch.rand(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(13))
    cfg = api.make_config(D, 16, 8, k, dtype="bf16" if dtype == BF16 else "f32")
    dyp, dw = api.combine_backward(cfg, dy, yp, row, tw)
    for part in (slice(0, last), slice(T - last, T)):
        r = row[part].long()
        own = r - r.min()
        dyp1, dw1 = api.combine_backward(cfg, dy[part], yp[r.min():r.max() + 1], own.to(torch.int32), tw[part])
        _ok(api)
        assert torch.equal(dw[part], dw1) and torch.equal(dyp[r.min():r.max() + 1], dyp1)
