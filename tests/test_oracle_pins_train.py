"""Pins of the training-pass and MXFP4 oracle (CPU): differences, hand-worked values, round trips."""
import numpy as np
import pytest

from oracle import train as T


def _problem(act, seed=0):
    rng = np.random.default_rng(seed)
    E, R, D, F = 3, 9, 5, 4
    off = np.array([0, 4, 4, 9])
    mk = lambda *s: rng.normal(0, 1, s)  # noqa: E731
    return off, mk(R, D), [mk(E, F, D), mk(E, F, D), mk(E, D, F), mk(E, F), mk(E, F), mk(E, D)], mk(R, D)


@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_backward_matches_differences(act):
    """Central differences of L = sum(y * dy) in fp64: error O(step^2) + eps / step, both below 1e-8 here."""
    off, x, p, dy = _problem(act)
    limit, step = 1.5, 1e-6                                   # a clip that some values meet
    loss = lambda x, p: float(np.sum(T.forward(x, off, *p, act, limit)[3] * dy))  # noqa: E731
    g, u, h, _ = T.forward(x, off, *p, act, limit)
    gap = min(np.min(np.abs(g)), np.min(np.abs(g - limit)), np.min(np.abs(np.abs(u) - limit)))
    assert gap > 10 * step or act == "silu"                   # no difference straddles a clip's corner
    b = T.backward(x, off, p[0], p[1], p[2], g, u, h, dy, act, limit)
    for name, arr in [("dx", x), ("w_gate", p[0]), ("w_up", p[1]), ("w_down", p[2]), ("b_gate", p[3]),
                      ("b_up", p[4]), ("b_down", p[5])]:
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + step
            hi = loss(x, p)
            arr[i] = keep - step
            lo = loss(x, p)
            arr[i] = keep
            assert abs((hi - lo) / (2 * step) - b[name][i]) < 1e-6 * (1 + abs(b[name][i])), (name, i)


def test_expert_without_rows_has_zero_gradients():
    off, x, p, dy = _problem("swiglu")
    g, u, h, _ = T.forward(x, off, *p, "swiglu")
    b = T.backward(x, off, p[0], p[1], p[2], g, u, h, dy, "swiglu")
    for n in ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down"):
        assert np.all(b[n][1] == 0)


def test_activation_at_the_clips():
    g = np.array([-1.0, 0.0, 7.0, 7.5, 3.0, 3.0])
    u = np.array([1.0, 1.0, 1.0, 1.0, -7.0, -7.5])
    h, ag, au = T.activation(g, u, "swiglu")
    assert h[0] == 0 and h[1] == 0 and h[2] == h[3] and h[4] == h[5]
    assert ag[0] == 0 and ag[1] == 0.5 and ag[2] != 0 and ag[3] == 0
    assert au[4] != 0 and au[5] == 0


def test_combine_backward_matches_differences():
    rng = np.random.default_rng(3)
    Tn, k, D = 4, 3, 5
    row = rng.permutation(Tn * k).reshape(Tn, k)
    w, yp, dy = rng.normal(size=(Tn, k)), rng.normal(size=(Tn * k, D)), rng.normal(size=(Tn, D))
    dyp, dw = T.combine_backward(dy, yp, row, w)
    # the combine is linear in each argument: its gradients are exact inner products
    for t in range(Tn):
        for j in range(k):
            assert np.isclose(dw[t, j], np.sum(dy[t] * yp[row[t, j]]))
            assert np.allclose(dyp[row[t, j]], w[t, j] * dy[t])


def test_mxfp4_worked_blocks():
    x = np.zeros((1, 160))
    x[0, 32:64] = 6.0                                          # amax exactly 6 * 2^0
    x[0, 64] = np.nextafter(np.float32(6.0), np.float32(7.0))  # just above: X = 1
    x[0, 96:104] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]   # ties
    x[0, 128] = 2.0 ** -140                                    # below the smallest scale
    c, s = T.quantize_mxfp4(x)
    assert list(s[0]) == [0, 127, 128, 127, 0]
    assert np.all(c[0, :32] == 0) and np.all(c[0, 32:64] == 7)
    assert c[0, 64] == 5                                       # 6.0000005 / 2 = 3
    assert list(c[0, 96:104]) == [0, 2, 2, 4, 4, 6, 6, 7]
    assert c[0, 128] == 0
    bad = np.ones((1, 64))
    bad[0, 3] = np.inf
    bad[0, 40] = np.nan
    c, s = T.quantize_mxfp4(bad)
    assert list(s[0]) == [255, 255] and not c.any()
    assert np.all(np.isnan(T.mxfp4_values(c, s)))


def test_mxfp4_round_trip_and_error():
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (7, 96)) * np.exp2(rng.integers(-20, 20, (7, 1)))
    c, s = T.quantize_mxfp4(x)
    v = T.mxfp4_values(c, s)
    assert np.array_equal(T.unpack(T.pack(c)), c)
    amax = np.abs(x.reshape(-1, 32)).max(1)
    X = s.reshape(-1).astype(int) - 127
    assert np.all(amax <= 6 * np.exp2(X)) and np.all(amax > 3 * np.exp2(X))
    # half of the widest gap of the grid (4 .. 6) at this scale
    assert np.all(np.abs(v - x).reshape(-1, 32) <= np.exp2(X)[:, None] * 1.0)
    c2, s2 = T.quantize_mxfp4(v)
    assert np.array_equal(T.mxfp4_values(c2, s2), v)           # values of the grid stay


def test_scale_tile_order():
    s = np.arange(2 * 130 * 3, dtype=np.int64).reshape(2, 130, 3).astype(np.uint8)
    t = T.scale_tiles(s).reshape(2, 2, 2, 32, 4, 4)
    assert t[1, 0, 0, 5, 2, 1] == s[1, 69, 1] and t[0, 1, 0, 1, 0, 2] == s[0, 129, 2]
    assert t[0, 0, 0, 0, 0, 3] == 127 and np.all(t[:, :, 1] == 127) and np.all(t[:, 1, 0, 2:] == 127)
