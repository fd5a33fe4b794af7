"""Training steps of a whole layer (marked gpu) as a program queues them, each call reading what the one before it
writes: without a wait between them, on two streams at once and captured, they have the bits of calls that were
waited for one by one."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


def _problem(api, T, D, F, E, k, dtype, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    mk = lambda std, *s: (torch.randn(s, device="cuda", generator=gen) * std).to(dtype)  # noqa: E731
    experts = api.ExpertWeights(mk(D ** -0.5, E, F, D), mk(D ** -0.5, E, F, D), mk(F ** -0.5, E, D, F), mk(0.1, E, F),
                                mk(0.1, E, F), mk(0.1, E, D))
    cfg = api.make_config(D, F, E, k, dtype="bf16" if dtype == BF16 else "f32")
    return cfg, mk(1.0, T, D), mk(D ** -0.5, E, D), mk(0.1, E), experts, mk(1.0, T, D)


def _steps(api, problem, wait):
    """Three training steps; after each, MXFP4 products with its gradients and the layer itself."""
    cfg, x, w_router, b_router, w, dy = problem
    outs = []

    def did(r):
        if wait:
            torch.cuda.synchronize()
        return r
    for _ in range(3):
        ids, tw = did(api.router_topk(cfg, x, w_router, b_router))
        p = did(api.permute(cfg, ids, x))
        row, off = p["row_of_slot"], p["expert_off"]
        gu, h, y = did(api.expert_ffn_train(cfg, p["x_perm"], off, w))
        dyp, dtw = did(api.combine_backward(cfg, dy, y, row, tw))
        dx, gr = did(api.expert_ffn_backward(cfg, p["x_perm"], off, w, gu, h, dyp))
        outs += [did(api.combine(cfg, y, row, tw)), dtw, did(api.combine(cfg, dx, row, torch.ones_like(tw))), gr.w_gate,
                 gr.w_up, gr.w_down, gr.b_gate, gr.b_down]
        if x.dtype == BF16:
            mw = did(api.mxfp4_weights(*did(api.quantize_mxfp4(gr.w_gate))))
            outs += [did(api.mxfp4_linear(p["x_perm"], mw, None, off)),
                     did(api.mxfp4_linear(dx, mw, gr.b_gate, off, out_f32=True))]
        outs.append(did(api.layer_forward(cfg, x, w_router, b_router, w)))
        names = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")
        w = did(api.ExpertWeights(*(getattr(w, n) - 0.01 * getattr(gr, n) for n in names)))
    return outs


# decode-sized, ragged and several tiles a pair; bf16 and fp32
PAIRS = [((3, 64, 96, 5, 2, BF16), (130, 32, 64, 33, 4, F32)), ((600, 1440, 736, 8, 4, BF16), (17, 256, 512, 8, 2, F32)),
         ((1500, 1024, 1312, 5, 4, BF16), (257, 2048, 320, 33, 2, BF16))]


@pytest.mark.parametrize("pair", PAIRS, ids=[f"{a[:5]}_{b[:5]}".replace(" ", "") for a, b in PAIRS])
def test_steps_without_waits(api, pair):
    problems = [_problem(api, *s, seed=i) for i, s in enumerate(pair)]
    want = [_steps(api, p, True) for p in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, _steps(api, problems[i], False)))
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _steps(api, problems[i], False)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        got.append((i, [o.clone() for o in outs]))
        del g
    assert api.last_device_error() == 0
    for i, outs in got:
        for n, (a, b) in enumerate(zip(outs, want[i])):
            assert torch.equal(a, b), (i, n)
