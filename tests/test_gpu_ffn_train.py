"""The expert block's training pass on the GPU (marked gpu), stage by stage against the fp64 oracle.

Each stage is compared on the values that the kernels themselves handed it (the stored gu and h, the dg and du
in the backward's workspace), so a bound counts that stage's own roundings only: fp32 sums (``sum_bound``), the
activation's exponential, and one rounding of the result.
"""
import numpy as np
import pytest

from oracle import train as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from train_util import HALF, Block, backward_ws, sum_bound, values, within  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api(cuda_ok):
    from mixture_experts_ffn_12_b200 import api as A, build
    build.build()
    return A


# rows per expert around the 16-row MMA steps, the 64-row stages and the 128-row tiles; experts without
# rows at the start, in the middle and at the end
EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 200, 0]
CASES = [
    (EDGES, 48, 80, BF16, "swiglu", True),
    (EDGES, 240, 256, BF16, "silu", False),
    ([1], 16, 16, BF16, "swiglu", True),
    ([300], 496, 272, BF16, "swiglu", False),
    ([0, 700, 3], 512, 720, BF16, "swiglu", True),
    ([40, 0, 513, 90], 1440, 336, BF16, "silu", True),
    # enough tiles that they keep their full height (128 and 256 rows)
    ([600, 0, 1030], 1440, 2880, BF16, "swiglu", True),
    ([530, 770], 2880, 1456, BF16, "silu", False),
    (EDGES, 48, 80, F32, "swiglu", True),
    ([1], 16, 16, F32, "silu", False),
    ([130, 0, 67], 272, 144, F32, "swiglu", False),
]
IDS = [f"E{len(c[0])}_R{sum(c[0])}_D{c[1]}_F{c[2]}_{'bf16' if c[3] == BF16 else 'f32'}_{c[4]}" for c in CASES]
LIMIT = 2.0     # low enough that both clips are met often


def _act_bounds(dh_err, dh, g, u, act):
    """Bounds of dg, du from an error of dh and the fp32 activation (its sigmoid to 2^-20)."""
    h, ag, au = O.activation(g, u, act, LIMIT)
    alpha = 1.0 if act == "silu" else 1.702
    gc, uc = O.clips(g, u, act, LIMIT)[:2]
    wobble = 2.0 ** -20
    dg = np.abs(ag) * dh_err + np.abs(dh * uc) * (1 + 2 * alpha * np.abs(gc)) * wobble
    du = np.abs(au) * dh_err + np.abs(dh * gc) * wobble
    return dg, du


def _forward(api, b, act):
    cfg = b.config(api, LIMIT)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, b.weights(api), act=act)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    return cfg, gu, h, y


@pytest.mark.parametrize("counts,D,F,dtype,act,bias", CASES, ids=IDS)
def test_forward(api, counts, D, F, dtype, act, bias):
    b = Block(counts, D, F, dtype, bias)
    _, gu, h, y = _forward(api, b, act)
    g, u, hw, _ = O.forward(b.val("x"), b.off, b.val("wg"), b.val("wu"), b.val("wd"), b.val("bg"), b.val("bu"),
                            b.val("bd"), act, LIMIT)
    got, half = values(gu), HALF[dtype]
    ax = np.abs(b.val("x"))
    err = {}
    for i, (name, want, w, bias_v) in enumerate((("g", g, "wg", b.val("bg")), ("u", u, "wu", b.val("bu")))):
        mags = O.rows_times(ax, np.abs(b.val(w)), b.off) + (0 if bias_v is None else np.abs(bias_v[O.per_row(b.off, b.R)]))
        err[name] = sum_bound(D, mags)
        # a value next to a clip bound may be rounded the other way: up to a whole step
        within(name, got[:, i], want, err[name] + 2 * half * (np.abs(want) + err[name]))
        if act == "swiglu":   # and it stays inside or outside the clip wherever the sum's own error leaves no doubt
            outside = (lambda v: v > LIMIT) if name == "g" else (lambda v: np.abs(v) > LIMIT)
            sure = np.abs(np.abs(want) - LIMIT) > err[name]
            assert np.array_equal(outside(got[:, i])[sure], outside(want)[sure])
    # |f'| <= 1.13 for every alpha-scaled sigmoid, |f(a)| <= |a|; the exponential to 2^-20
    gc, uc = O.clips(g, u, act, LIMIT)[:2]
    herr = 1.13 * np.abs(uc) * err["g"] + np.abs(gc) * err["u"] + np.abs(gc * uc) * 2.0 ** -20 + \
        1.13 * err["g"] * err["u"]
    within("h", values(h), hw, herr + half * (np.abs(hw) + herr))
    hk = values(h)
    yw = O.rows_times(hk, b.val("wd"), b.off)
    mags = O.rows_times(np.abs(hk), np.abs(b.val("wd")), b.off)
    if bias:
        e = O.per_row(b.off, b.R)
        yw, mags = yw + b.val("bd")[e], mags + np.abs(b.val("bd")[e])
    yerr = sum_bound(F, mags)
    within("y", values(y), yw, yerr + half * (np.abs(yw) + yerr))


@pytest.mark.parametrize("grad_f32", [False, True])
@pytest.mark.parametrize("counts,D,F,dtype,act,bias", CASES, ids=IDS)
def test_backward(api, counts, D, F, dtype, act, bias, grad_f32):
    b = Block(counts, D, F, dtype, bias, seed=1)
    cfg, gu, h, _ = _forward(api, b, act)
    ws, dgu_t = backward_ws(cfg, b)
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, b.weights(api), gu, h, b.dy, act=act, grad_f32=grad_f32, ws=ws)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    half, ghalf = HALF[dtype], HALF[F32 if grad_f32 else dtype]
    x, dy, hk, guv = b.val("x"), b.val("dy"), values(h), values(gu)
    wg, wu, wd = b.val("wg"), b.val("wu"), b.val("wd")
    ref = O.backward(x, b.off, wg, wu, wd, guv[:, 0], guv[:, 1], hk, dy, act, LIMIT)
    dh = O.rows_times(dy, np.swapaxes(wd, 1, 2), b.off)
    dh_err = sum_bound(D, O.rows_times(np.abs(dy), np.abs(np.swapaxes(wd, 1, 2)), b.off))
    eg, eu = _act_bounds(dh_err, dh, guv[:, 0], guv[:, 1], act)
    dgu = values(dgu_t)
    within("dg", dgu[:, 0], ref["dg"], eg + half * (np.abs(ref["dg"]) + eg) + 1e-38)
    within("du", dgu[:, 1], ref["du"], eu + half * (np.abs(ref["du"]) + eu) + 1e-38)
    dg, du = dgu[:, 0], dgu[:, 1]
    wgt, wut = np.swapaxes(wg, 1, 2), np.swapaxes(wu, 1, 2)
    want = O.rows_times(dg, wgt, b.off) + O.rows_times(du, wut, b.off)
    mags = O.rows_times(np.abs(dg), np.abs(wgt), b.off) + O.rows_times(np.abs(du), np.abs(wut), b.off)
    err = sum_bound(2 * F, mags)
    within("dx", values(dx), want, err + half * (np.abs(want) + err))
    most = max(counts)
    for name, a, c in (("w_gate", dg, x), ("w_up", du, x), ("w_down", dy, hk)):
        want = O.outer_sums(a, c, b.off)
        err = sum_bound(most, O.outer_sums(np.abs(a), np.abs(c), b.off))
        got = getattr(gr, name)
        assert got.dtype == (F32 if grad_f32 else dtype)
        within(name, values(got), want, err + ghalf * (np.abs(want) + err))
    # db_gate and db_up: sums of dg and du before their rounding, so against the oracle's own
    for name, a, more in (("b_gate", ref["dg"], eg), ("b_up", ref["du"], eu), ("b_down", dy, 0.0 * dy)):
        got = getattr(gr, name)
        if not bias:
            assert got is None
            continue
        want = O.column_sums(a, b.off)
        err = sum_bound(most, O.column_sums(np.abs(a) + more, b.off)) + O.column_sums(more, b.off)
        within(name, values(got), want, err + ghalf * (np.abs(want) + err))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_rows_stay_with_their_expert(api, bad):
    """Rows of one expert hold infinities or NaN: the other experts' rows and gradients, whose tiles and K
    blocks reach into those rows, are those of the clean run, bit for bit."""
    counts, D, F = [37, 21, 50, 5], 96, 112
    outs = []
    for poison in (False, True):
        b = Block(counts, D, F, BF16, True, seed=2)
        if poison:
            b.x[37:58] = bad
            b.dy[37:58] = bad
        cfg, gu, h, y = _forward(api, b, "swiglu")
        dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, b.weights(api), gu, h, b.dy)
        torch.cuda.synchronize()
        assert api.last_device_error() == 0
        outs.append((gu, h, y, dx, gr.w_gate, gr.w_up, gr.w_down, gr.b_gate, gr.b_up, gr.b_down))
    rows = torch.cat([torch.arange(37), torch.arange(58, 113)]).cuda()
    experts = torch.tensor([0, 2, 3]).cuda()
    for i, (clean, poisoned) in enumerate(zip(*outs)):
        at = rows if i < 4 else experts
        assert torch.isfinite(clean).all()
        assert torch.equal(clean[at], poisoned[at]), i


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_nan_is_not_clipped_away(api, act, dtype):
    """A NaN in a row of x reaches the whole row of gu, h and y; one in gu the row of dx, its feature's weight
    gradients and those alone."""
    D, F = 64, 48
    b = Block([9, 40], D, F, dtype, True, seed=8)
    b.x[3, 5] = float("nan")
    cfg, gu, h, y = _forward(api, b, act)
    for t in (gu, h, y):
        assert torch.isnan(t[3]).all() and torch.isfinite(torch.cat([t[:3], t[4:]])).all()
    b = Block([9, 40], D, F, dtype, True, seed=8)
    cfg, gu, h, _ = _forward(api, b, act)
    gu[3, 0, 7] = gu[20, 1, 11] = float("nan")
    gu[3, 1, 7] = gu[20, 0, 11] = 0.5      # the other factor inside its clip
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, b.weights(api), gu, h, b.dy, act=act)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    rows = torch.isnan(dx).all(1)
    assert rows.nonzero().flatten().tolist() == [3, 20] and torch.isfinite(dx[~rows]).all()
    for grad, bias in ((gr.w_gate, gr.b_gate), (gr.w_up, gr.b_up)):
        assert torch.equal(torch.isnan(grad).all(2), torch.isnan(bias))
        for e, f in ((0, 7), (1, 11)):
            bad = torch.isnan(bias[e])
            assert set(bad.nonzero().flatten().tolist()) <= {f}
    # d/dg at a NaN g, d/du at a NaN u: both; the other derivative holds the NaN factor as well
    assert torch.isnan(gr.b_gate[0, 7]) and torch.isnan(gr.b_up[0, 7])
    assert torch.isnan(gr.b_gate[1, 11])


def test_partial_requests_and_reproducible(api):
    """Some gradients only, given buffers, a second call with the same bits; nothing else is written."""
    b = Block([70, 0, 131], 96, 176, BF16, True, seed=3)
    cfg, gu, h, _ = _forward(api, b, "swiglu")
    w = b.weights(api)
    dx, full = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
    buf = api.ExpertGrads(*(torch.full_like(getattr(full, n), 7.0) for n in ("w_gate", "w_up", "w_down")))
    none, got = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, need_dx=False, grads=buf)
    assert none is None and got is buf
    for n in ("w_gate", "w_up", "w_down"):
        assert torch.equal(getattr(buf, n), getattr(full, n))
    dx2, again = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
    assert torch.equal(dx, dx2) and torch.equal(full.b_up, again.b_up) and torch.equal(full.w_up, again.w_up)


@pytest.mark.parametrize("need_dx", [True, False])
def test_workspace_content_does_not_matter(api, need_dx):
    """Calls one after another on one workspace, each time filled with other bytes (tile counter and bias sums lie
    in it), give the same bits as a call on its own."""
    b = Block([143, 0, 70, 300, 1], 200 - 200 % 16, 368, BF16, True, seed=9)
    cfg, gu, h, _ = _forward(api, b, "swiglu")
    w = b.weights(api)
    dx, want = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, need_dx=need_dx)
    ws, _ = backward_ws(cfg, b)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        for _ in range(3):
            dx2, got = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, need_dx=need_dx, ws=ws)
            assert (dx is None) == (dx2 is None) and (dx is None or torch.equal(dx, dx2))
            for n in ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"):
                assert torch.equal(getattr(got, n), getattr(want, n)), (fill, n)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0


def test_rows_of_no_expert_are_left(api):
    """expert_off ends before the last row: the rows behind it are neither read into a gradient nor written."""
    b = Block([33, 20], 64, 48, BF16, True, seed=4)
    cfg, gu, h, _ = _forward(api, b, "swiglu")
    w = b.weights(api)
    _, want = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy)
    more = 9
    nan = lambda t: torch.cat([t, torch.full((more, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")])  # noqa: E731
    ws, dgu = backward_ws(cfg, b, more)
    dgu.fill_(3.0)
    _, got = api.expert_ffn_backward(cfg, nan(b.x), b.off_gpu, w, nan(gu), nan(h), nan(b.dy), ws=ws)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert (dgu[b.R:] == 3.0).all()
    for n in ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"):
        assert torch.equal(getattr(got, n), getattr(want, n))


def test_no_rows_at_all(api):
    b = Block([0, 0], 32, 48, BF16, True)
    cfg = b.config(api)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, b.weights(api))
    assert gu.shape == (0, 2, 48) and y.shape == (0, 32)
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, b.weights(api), gu, h, b.dy)
    torch.cuda.synchronize()
    assert dx.shape == (0, 32) and all((getattr(gr, n) == 0).all() for n in ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"))


@pytest.mark.parametrize("T,k,D", [(1, 1, 16), (3, 2, 48), (37, 8, 1040), (130, 4, 2880)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_combine_backward(api, T, k, D, dtype):
    rng = np.random.default_rng(T * 10 + k)
    row = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    dy = torch.from_numpy(rng.normal(size=(T, D)).astype(np.float32)).cuda().to(dtype)
    yp = torch.from_numpy(rng.normal(size=(T * k, D)).astype(np.float32)).cuda().to(dtype)
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    cfg = api.make_config(D, 16, 8, k, dtype="bf16" if dtype == BF16 else "f32")
    dyp, dw = api.combine_backward(cfg, dy, yp, torch.from_numpy(row).cuda(), w)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    rdyp, rdw = O.combine_backward(values(dy), values(yp), row, values(w))
    # one fp32 product, then one rounding to the type
    within("dy_perm", values(dyp), rdyp, np.abs(rdyp) * (HALF[dtype] + 2.0 ** -23) + 1e-40)
    mags = O.combine_backward(np.abs(values(dy)), np.abs(values(yp)), row, values(w))[1]
    within("dw", values(dw), rdw, sum_bound(D, mags))


def test_combine_backward_bad_row_is_reported(api):
    cfg = api.make_config(32, 16, 4, 2)
    row = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32).cuda()
    dy, yp = torch.ones(2, 32, dtype=BF16).cuda(), torch.ones(4, 32, dtype=BF16).cuda()
    dyp, dw = api.combine_backward(cfg, dy, yp, row, torch.ones(2, 2).cuda())
    torch.cuda.synchronize()
    from mixture_experts_ffn_12_b200 import _lib
    assert api.last_device_error() == _lib.MOE_ERR_DEVICE_BOUNDS
    assert api.last_device_error() == 0
    assert dw[0].tolist() == [32.0, 32.0] and dw[1, 0].item() == 32.0
