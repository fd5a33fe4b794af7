"""MXFP4 on the GPU (marked gpu) with many tiles a CTA pair, every tile width, 256 groups, and more blocks than one
grid covers.  A tile is 256 output columns by at most 192 of a group's rows, split evenly in steps of 16; K runs in
stages of 256 elements.  The product is compared with fp64 on the values of the quantized operands (the quantizer
and its inverse are bit-exact, test_gpu_mxfp4.py), with the bounds of that file."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_check import within  # noqa: E402
from train_util import HALF, offsets, sum_bound  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


# 72 row tiles, the splits' edges among them; with 12 column tiles eleven tiles a pair
EDGES = [191, 192, 193, 385, 0, 384, 1, 577, 576, 1000, 33, 208, 900, 640, 383, 0, 961, 15, 1537, 17, 1152, 129, 1300, 768]
CASES = {
    "eleven_tiles_a_pair": (EDGES, 2880, 2880, True, False),
    "eleven_tiles_a_pair_f32": (EDGES, 2848, 2848, True, True),      # the last column tile, block of rows and stage not full
    "one_group": ([11000], 1456, 1120, False, True),
    "widths": ([16 * i - (i & 1) for i in range(1, 13)], 528, 544, True, False),
    "widths_over": ([16 * i + 1 for i in range(12)], 272, 800, False, True),
    "256_groups": ([int(n) for n in np.random.default_rng(3).integers(0, 20, 256)], 144, 160, True, False),
    "skewed": ([3] * 40 + [2500] + [7] * 60 + [900, 0, 0], 1008, 416, True, True),
}


@pytest.mark.parametrize("case", CASES)
def test_linear(api, case):
    counts, N, K, bias, out_f32 = CASES[case]
    G, R = len(counts), sum(counts)
    off, off_gpu = offsets(counts)
    gen = torch.Generator("cuda").manual_seed(N + K)
    codes = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(119, 130, (G, N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    x = torch.randn(R, K, device="cuda", generator=gen)
    x = (x * torch.exp2(torch.randint(-4, 4, (R, 1), device="cuda", generator=gen).float())).to(BF16)
    b = (3 * torch.randn(G, N, device="cuda", generator=gen)).to(BF16) if bias else None
    w = api.mxfp4_weights(codes, scales)
    args = (x, w, b, off_gpu if G > 1 else None)
    y = api.mxfp4_linear(*args, out_f32=out_f32)
    again = api.mxfp4_linear(*args, out_f32=out_f32)
    xq = api.dequantize_mxfp4(*api.quantize_mxfp4(x), F32)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert torch.equal(y, again)
    for g in range(G):
        at = slice(int(off[g]), int(off[g + 1]))
        if at.start == at.stop:
            continue
        a, v = xq[at].double(), api.dequantize_mxfp4(codes[g], scales[g], F32).double()
        want, mags = a @ v.T, a.abs() @ v.abs().T
        if bias:
            want, mags = want + b[g].double(), mags + b[g].double().abs()
        err = sum_bound(K, mags)
        within(f"y of group {g}", y[at], want, err + HALF[y.dtype] * (want.abs() + err))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_more_blocks_than_one_grid(api, dtype):
    """Rows beyond what one grid covers at once have the codes, scales and values of calls on a few of them."""
    rows, K, part = 7001, 2880, 500
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(rows, K, device="cuda", generator=gen)
    x = (x * torch.exp2(torch.randint(-60, 60, (rows, 1), device="cuda", generator=gen).float())).to(dtype)
    x[rows - 1, K - 1] = float("inf")
    codes, scales = api.quantize_mxfp4(x)
    values = {t: api.dequantize_mxfp4(codes, scales, t) for t in (BF16, F32)}
    for r in range(0, rows, part):
        c, s = api.quantize_mxfp4(x[r:r + part])
        assert torch.equal(codes[r:r + part], c) and torch.equal(scales[r:r + part], s)
        for t, v in values.items():
            assert torch.equal(v[r:r + part].nan_to_num(7.0), api.dequantize_mxfp4(c, s, t).nan_to_num(7.0))
    assert scales[rows - 1, K // 32 - 1] == 255 and values[BF16][rows - 1, K - 32:].isnan().all()
