"""The expert block's training pass on the GPU (marked gpu) with many tiles a CTA pair, every tile width, many and
unevenly loaded experts: accumulators and ring slots used again, tiles taken from the counter, tables of 256 groups."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_check import GpuBlock, run_checked  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
LIMIT = 2.0     # low enough that both clips are met often


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


def _zipf(E, R, s=1.1):
    """Rows of E experts, R in all, loaded as 1 / rank^s, the ranks shuffled."""
    p = 1.0 / np.arange(1, E + 1) ** s
    n = np.floor(R * p / p.sum()).astype(int)
    n[0] += R - n.sum()
    return [int(v) for v in np.random.default_rng(E).permutation(n)]


def _few(E, most, seed):
    """0 to `most` rows an expert, the first and the last without any."""
    n = np.random.default_rng(seed).integers(0, most + 1, E)
    n[0] = n[-1] = 0
    return [int(v) for v in n]


CASES = {
    # 38 row tiles of up to 256 and 12 column tiles: six tiles a pair in DOWN, DH and DX, twelve in GATEUP
    "six_tiles_a_pair": ([1500, 1490, 777, 0, 1024, 1203, 1640, 1361], 2880, 2880, BF16, "swiglu", True, False),
    "six_tiles_a_pair_silu_f32_grads": ([1537, 0, 2049, 1300, 255, 257, 1791, 900], 2848, 2896, BF16, "silu", True, True),
    # every width of the row tiles, 16 to 256, by one row less and one more
    "widths": ([16 * i - (i & 1) for i in range(1, 17)], 720, 752, BF16, "swiglu", True, False),
    "widths_over": ([16 * i + 1 for i in range(16)], 784, 720, BF16, "silu", False, True),
    # one expert with a quarter of the rows, most with a handful
    "zipf_128_experts": (_zipf(128, 6000), 576, 400, BF16, "swiglu", True, False),
    "zipf_64_experts": (_zipf(64, 9000, 1.6), 1440, 720, BF16, "silu", False, False),
    "256_experts": (_few(256, 15, 1), 64, 80, BF16, "swiglu", True, True),
    "256_experts_f32": (_few(256, 15, 2), 80, 64, F32, "swiglu", True, False),
    "40_experts_f32": (_zipf(40, 700), 272, 336, F32, "silu", True, False),
    "largest_f32": ([500, 0, 333, 191], 640, 640, F32, "swiglu", True, False),
}


@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(api, case):
    counts, D, F, dtype, act, bias, grad_f32 = CASES[case]
    run_checked(api, GpuBlock(counts, D, F, dtype, bias, seed=len(case)), act, LIMIT, grad_f32)


@pytest.mark.parametrize("case", ["six_tiles_a_pair", "zipf_128_experts", "256_experts_f32"])
def test_same_bits_again(api, case):
    """The same bits from call to call, other calls in between: whichever pair takes a tile from the counter."""
    counts, D, F, dtype, act, bias, grad_f32 = CASES[case]
    b, other = (GpuBlock(counts, D, F, dtype, bias, seed=s) for s in (21, 22))
    want = run_checked(api, b, act, LIMIT, grad_f32)

    def once(bl):
        cfg, w = bl.config(api, LIMIT), bl.weights(api)
        gu, h, y = api.expert_ffn_train(cfg, bl.x, bl.off_gpu, w, act=act)
        dx, gr = api.expert_ffn_backward(cfg, bl.x, bl.off_gpu, w, gu, h, bl.dy, act=act, grad_f32=grad_f32)
        return [gu, h, y, dx, gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down]
    for _ in range(6):
        once(other)
        for a, c in zip(once(b), want):
            assert torch.equal(a, c)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
