"""The expert block's training pass against its definition in fp64 (torch, on the GPU), for sizes at which numpy would
take minutes.  Each stage is compared on the values that the kernels themselves handed it, as in
test_gpu_ffn_train.py, with the same bounds."""
import torch

from train_util import HALF, Block, backward_ws, offsets, sum_bound


class GpuBlock(Block):
    """A seeded expert block made on the GPU."""

    def __init__(self, counts, D, F, dtype, bias=True, seed=0, gate_std=1.5):
        self.counts, self.D, self.F, self.E, self.R, self.dtype = counts, D, F, len(counts), int(sum(counts)), dtype
        self.off, self.off_gpu = offsets(counts)
        gen = torch.Generator("cuda").manual_seed(seed)
        mk = lambda std, *s: (torch.randn(s, device="cuda", generator=gen) * std).to(dtype)  # noqa: E731
        E, R = self.E, self.R
        self.x, self.dy = mk(1.0, R, D), mk(1.0, R, D)
        self.wg, self.wu = mk(gate_std / D ** 0.5, E, F, D), mk(gate_std / D ** 0.5, E, F, D)
        self.wd = mk(1.0 / F ** 0.5, E, D, F)
        self.bg, self.bu, self.bd = (mk(0.2, E, F), mk(0.2, E, F), mk(0.2, E, D)) if bias else (None, None, None)


def within(name, got, want, bound):
    """|got - want| <= bound for every element."""
    bad = ~((got.double() - want).abs() <= bound)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; first at {at}: {got[at].item()!r} for "
                             f"{want[at].item()!r}, bound {bound[at].item():.3g}")


def _rounded(err, want, half):
    return err + half * (want.abs() + err)


def _clips(g, u, act, limit):
    if act == "silu":
        return g, u, torch.ones_like(g, dtype=torch.bool), torch.ones_like(u, dtype=torch.bool)
    return g.clamp(0, limit), u.clamp(-limit, limit), (g >= 0) & (g <= limit), u.abs() <= limit


def check_forward(b, act, limit, gu, h, y):
    """gu, h and y of ``expert_ffn_train`` on block `b`, expert by expert."""
    half, alpha = HALF[b.dtype], 1.0 if act == "silu" else 1.702
    for e in range(b.E):
        at = slice(int(b.off[e]), int(b.off[e + 1]))
        x, hk = b.x[at].double(), h[at].double()
        val, err = {}, {}
        for i, (n, w, bias) in enumerate((("g", b.wg, b.bg), ("u", b.wu, b.bu))):
            w = w[e].double()
            val[n], mags = x @ w.T, x.abs() @ w.abs().T
            if bias is not None:
                val[n], mags = val[n] + bias[e].double(), mags + bias[e].double().abs()
            err[n] = sum_bound(b.D, mags)
            # a value next to a clip bound may be rounded the other way: up to a whole step
            within(f"{n} of expert {e}", gu[at, i], val[n], _rounded(err[n], val[n], 2 * half))
        gc, uc = _clips(val["g"], val["u"], act, limit)[:2]
        want = gc * torch.sigmoid(alpha * gc) * uc
        # |f'| <= 1.13 for every alpha-scaled sigmoid, |f(a)| <= |a|; the exponential to 2^-20
        herr = 1.13 * uc.abs() * err["g"] + gc.abs() * err["u"] + (gc * uc).abs() * 2.0 ** -20 + 1.13 * err["g"] * err["u"]
        within(f"h of expert {e}", h[at], want, _rounded(herr, want, half))
        wd = b.wd[e].double()
        want, mags = hk @ wd.T, hk.abs() @ wd.abs().T
        if b.bd is not None:
            want, mags = want + b.bd[e].double(), mags + b.bd[e].double().abs()
        within(f"y of expert {e}", y[at], want, _rounded(sum_bound(b.F, mags), want, half))


def check_backward(b, act, limit, gu, h, dgu, dx, gr):
    """(dg, du) as the workspace holds them, dx and the gradients of ``expert_ffn_backward`` on block `b`."""
    half, ghalf = HALF[b.dtype], HALF[gr.w_gate.dtype]
    alpha = 1.0 if act == "silu" else 1.702
    for e in range(b.E):
        at = slice(int(b.off[e]), int(b.off[e + 1]))
        n = int(b.off[e + 1] - b.off[e])
        x, dy, hk = b.x[at].double(), b.dy[at].double(), h[at].double()
        g, u = gu[at, 0].double(), gu[at, 1].double()
        wg, wu, wd = b.wg[e].double(), b.wu[e].double(), b.wd[e].double()
        dh, dh_err = dy @ wd, sum_bound(b.D, dy.abs() @ wd.abs())
        gc, uc, gin, uin = _clips(g, u, act, limit)
        s = torch.sigmoid(alpha * gc)
        ag, au = uc * (s + alpha * gc * s * (1 - s)) * gin, gc * s * uin
        # the fp32 activation's sigmoid to 2^-20
        eg = ag.abs() * dh_err + (dh * uc).abs() * (1 + 2 * alpha * gc.abs()) * 2.0 ** -20
        eu = au.abs() * dh_err + (dh * gc).abs() * 2.0 ** -20
        dg, du = dh * ag, dh * au
        within(f"dg of expert {e}", dgu[at, 0], dg, _rounded(eg, dg, half) + 1e-38)
        within(f"du of expert {e}", dgu[at, 1], du, _rounded(eu, du, half) + 1e-38)
        # biases: sums of dg and du before their rounding
        for name, a, more in (("b_gate", dg, eg), ("b_up", du, eu), ("b_down", dy, torch.zeros_like(dy))):
            got = getattr(gr, name)
            if got is None:
                continue
            want, err = a.sum(0), sum_bound(n, (a.abs() + more).sum(0)) + more.sum(0)
            within(f"{name} of expert {e}", got[e], want, _rounded(err, want, ghalf))
        dg, du = dgu[at, 0].double(), dgu[at, 1].double()
        if dx is not None:
            want, mags = dg @ wg + du @ wu, dg.abs() @ wg.abs() + du.abs() @ wu.abs()
            within(f"dx of expert {e}", dx[at], want, _rounded(sum_bound(2 * b.F, mags), want, half))
        for name, a, c in (("w_gate", dg, x), ("w_up", du, x), ("w_down", dy, hk)):
            want, mags = a.T @ c, a.abs().T @ c.abs()
            within(f"{name} of expert {e}", getattr(gr, name)[e], want, _rounded(sum_bound(n, mags), want, ghalf))


def run_checked(api, b, act, limit, grad_f32=False):
    """One forward and one backward pass, both checked; what they returned."""
    cfg, w = b.config(api, limit), b.weights(api)
    gu, h, y = api.expert_ffn_train(cfg, b.x, b.off_gpu, w, act=act)
    ws, dgu = backward_ws(cfg, b)
    dx, gr = api.expert_ffn_backward(cfg, b.x, b.off_gpu, w, gu, h, b.dy, act=act, grad_f32=grad_f32, ws=ws)
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    check_forward(b, act, limit, gu, h, y)
    check_backward(b, act, limit, gu, h, dgu, dx, gr)
    return [gu, h, y, dx, gr.w_gate, gr.w_up, gr.w_down] + [t for t in (gr.b_gate, gr.b_up, gr.b_down) if t is not None]
