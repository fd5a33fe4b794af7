"""Helpers of the training-pass and MXFP4 tests: problems with given rows per expert, elementwise bounds."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative to the value


def values(t):
    return t.detach().double().cpu().numpy()


def to_gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def offsets(counts):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    return off, torch.from_numpy(off.astype(np.int32)).cuda()


def within(name, got, want, bound):
    """|got - want| <= bound for every element (and the same non-finite places)."""
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} off; first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r}, bound {bound[bad][0]:.3g}")


def sum_bound(n, abs_sum):
    """fp32 accumulation of n products: every addition may drop a step (2^-23, as a truncating adder does)
    of a partial sum that is at most the sum of the magnitudes."""
    return (n + 2) * 2.0 ** -23 * abs_sum


class Block:
    """A seeded expert block on the GPU, with the exact values of its tensors in fp64 on the host."""

    def __init__(self, counts, D, F, dtype, bias=True, seed=0, gate_std=1.5):
        rng = np.random.default_rng(seed)
        self.counts, self.D, self.F, self.E, self.R, self.dtype = counts, D, F, len(counts), int(sum(counts)), dtype
        self.off, self.off_gpu = offsets(counts)
        mk = lambda std, *s: to_gpu(rng.normal(0, std, s), dtype)  # noqa: E731
        E, R = self.E, self.R
        self.x, self.dy = mk(1.0, R, D), mk(1.0, R, D)
        self.wg, self.wu = mk(gate_std / D ** 0.5, E, F, D), mk(gate_std / D ** 0.5, E, F, D)
        self.wd = mk(1.0 / F ** 0.5, E, D, F)
        self.bg, self.bu, self.bd = (mk(0.2, E, F), mk(0.2, E, F), mk(0.2, E, D)) if bias else (None, None, None)

    def val(self, name):
        t = getattr(self, name)
        return None if t is None else values(t)

    def config(self, api, limit=7.0):
        return api.make_config(self.D, self.F, self.E, 1, limit, dtype="bf16" if self.dtype == torch.bfloat16 else "f32")

    def weights(self, api):
        return api.ExpertWeights(self.wg, self.wu, self.wd, self.bg, self.bu, self.bd)


def backward_ws(cfg, b, extra_rows=0):
    """(workspace of a backward call on the block's rows and extra_rows more, its (dg, du) [rows, 2, F])."""
    import ctypes
    from mixture_experts_ffn_12_b200 import _lib
    R = b.R + extra_rows
    ws = torch.empty(_lib.load().moe_expert_ffn_backward_workspace_size(ctypes.byref(cfg), R), dtype=torch.uint8, device="cuda")
    return ws, ws[:R * 2 * b.F * b.x.element_size()].view(b.dtype).view(R, 2, b.F)
