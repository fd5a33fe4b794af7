"""Oracle of the expert block's training pass and of MXFP4 quantization (numpy, fp64).

Definitions, expert by expert, on the exact values of the inputs:
  forward   g = x Wg^T + bg, u = x Wu^T + bu, h = f(g') u', y = h Wd^T + bd,
            f(a) = a / (1 + exp(-alpha a)), g' = clip(g, 0, L), u' = clip(u, -L, L)
            (SiLU: alpha = 1 and no clips)
  backward  dh = dy Wd, dg = dh u' f'(g') where the clip let g through (its ends included),
            du = dh f(g') likewise, dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x,
            dWd = dy^T h, bias gradients = column sums over the expert's rows
  combine   dy_perm[row(t, j)] = w[t, j] dy[t], dw[t, j] = dy[t] . y_perm[row(t, j)]
  MXFP4     blocks of 32 along K: X the smallest integer >= -127 with max |b| <= 6 * 2^X,
            elements to the nearest E2M1 value of b / 2^X, ties to the even code; a block
            with an infinity or NaN: scale byte 255, codes 0
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def clips(g, u, act, limit):
    if act == "silu":
        return g, u, np.ones_like(g, bool), np.ones_like(u, bool)
    return np.clip(g, 0.0, limit), np.clip(u, -limit, limit), (g >= 0) & (g <= limit), np.abs(u) <= limit


def sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def activation(g, u, act, limit=7.0, alpha=1.702):
    """(h, dh/dg, dh/du)."""
    a = 1.0 if act == "silu" else alpha
    gc, uc, gin, uin = clips(g, u, act, limit)
    s = sigmoid(a * gc)
    return gc * s * uc, np.where(gin, uc * (s + a * gc * s * (1.0 - s)), 0.0), np.where(uin, gc * s, 0.0)


def per_row(off, R):
    """Expert of each row, -1 for rows of none."""
    e = np.full(R, -1)
    for i in range(len(off) - 1):
        e[off[i]:off[i + 1]] = i
    return e


def rows_times(a, w, off):
    """a[r] W_e^T (W [E, N, K]) for every row of every expert."""
    out = np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ w[e].T
    return out


def forward(x, off, wg, wu, wd, bg, bu, bd, act, limit=7.0, alpha=1.702):
    g, u = rows_times(x, wg, off), rows_times(x, wu, off)
    e = per_row(off, x.shape[0])
    if bg is not None:
        g = g + bg[e]
    if bu is not None:
        u = u + bu[e]
    h = activation(g, u, act, limit, alpha)[0]
    y = rows_times(h, wd, off)
    return g, u, h, (y if bd is None else y + bd[e])


def outer_sums(a, b, off):
    """sum over each expert's rows of a[r]^T b[r]: [E, a columns, b columns]."""
    return np.stack([a[off[i]:off[i + 1]].T @ b[off[i]:off[i + 1]] for i in range(len(off) - 1)])


def column_sums(a, off):
    return np.stack([a[off[i]:off[i + 1]].sum(0) for i in range(len(off) - 1)])


def backward(x, off, wg, wu, wd, g, u, h, dy, act, limit=7.0, alpha=1.702):
    dh = rows_times(dy, np.swapaxes(wd, 1, 2), off)
    _, ag, au = activation(g, u, act, limit, alpha)
    dg, du = dh * ag, dh * au
    return dict(dg=dg, du=du,
                dx=rows_times(dg, np.swapaxes(wg, 1, 2), off) + rows_times(du, np.swapaxes(wu, 1, 2), off),
                w_gate=outer_sums(dg, x, off), w_up=outer_sums(du, x, off), w_down=outer_sums(dy, h, off),
                b_gate=column_sums(dg, off), b_up=column_sums(du, off), b_down=column_sums(dy, off))


def combine_backward(dy, y_perm, row_of_slot, w):
    T, k = w.shape
    out, dw = np.zeros_like(y_perm), np.zeros_like(w)
    for t in range(T):
        for j in range(k):
            out[row_of_slot[t, j]] = w[t, j] * dy[t]
            dw[t, j] = float(np.dot(dy[t], y_perm[row_of_slot[t, j]]))
    return out, dw


def quantize_mxfp4(x):
    """x [rows, K] -> (codes [rows, K] 0..15, scale bytes [rows, K/32])."""
    rows, K = x.shape
    b = x.reshape(-1, 32)
    codes, scales = np.zeros(b.shape, np.uint8), np.zeros(len(b), np.uint8)
    for i, v in enumerate(b):
        amax = np.max(np.abs(v))
        if not np.isfinite(amax):
            scales[i] = 255
            continue
        X = -127
        if amax > 0:
            X = max(-127, math.frexp(amax)[1] - 4)
            while amax > math.ldexp(6.0, X):
                X += 1
        scales[i] = X + 127
        q = np.abs(v) * math.ldexp(1.0, -X)
        d = np.abs(q[:, None] - E2M1[None])
        best = d.min(1, keepdims=True)
        near = d == best
        # of two values at the same distance, the one with the even code
        code = np.where(near.sum(1) == 1, near.argmax(1), (near & (np.arange(8) % 2 == 0)).argmax(1))
        codes[i] = code + 8 * (np.signbit(v))
    return codes.reshape(rows, K), scales.reshape(rows, K // 32)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def mxfp4_values(codes, scales):
    """codes [..., K] 0..15, scales [..., K/32] -> values."""
    v = np.where(codes >= 8, -E2M1[codes & 7], E2M1[codes & 7])
    f = np.ldexp(1.0, scales.astype(np.int64) - 127)
    f = np.where(scales == 255, np.nan, f)
    return v * np.repeat(f, 32, axis=-1)


def scale_tiles(scales):
    """[G, N, nb] scale bytes in the product's tile order, flat (127 in the padding)."""
    G, N, nb = scales.shape
    rb, kc = -(-N // 128), 2 * -(-nb // 8)
    out = np.full((G, rb, kc, 512), 127, np.uint8)
    for g in range(G):
        for n in range(N):
            for b in range(nb):
                out[g, n // 128, b // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + b % 4] = scales[g, n, b]
    return out.reshape(-1)
