"""The layer's training and MXFP4 operators as measured cases.

Five operators: the MXFP4 quantizer with its inverse, the MXFP4 x MXFP4 product, the expert feed-forward
block's training forward, its backward pass, and the combine's backward pass.  ``run`` computes each in its
plain form (``own`` false: elementary torch operations in fp32, rounded once) or through this package's calls
(``own`` true).  Rows of R = T * k routed pairs are sorted by expert; ``off`` [E + 1] holds the experts' bounds.
"""
import math

import torch

own = False

LIMIT, ALPHA = 7.0, 1.702      # the clipped SwiGLU's clip and sigmoid scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    q, p, f, b, c = "quantize", "linear", "ffn", "ffn_backward", "combine_backward"
    return [
        # activations of a few decode tokens
        dict(name="quantize 8 rows", op=q, rows=8, K=2880, dtype="bf16"),
        # one projection of every expert of a GPT-OSS-20B-shaped layer (32 x 2880 rows)
        dict(name="quantize expert weights", op=q, rows=92160, K=2880, dtype="bf16"),
        # one token through one 2880 x 2880 projection
        dict(name="linear 1 token", op=p, E=1, R=1, K=2880, N=2880, empty=0),
        # a decode batch of 32 tokens, 4 experts each, ragged rows per expert
        dict(name="linear decode experts", op=p, E=32, R=128, K=2880, N=2880, empty=2),
        # the prefill batch of 4096 tokens, 4 experts each
        dict(name="linear prefill experts", op=p, E=32, R=16384, K=2880, N=2880, empty=0),
        # the tiny fp32 layer: 64 tokens, 2 of 8 experts
        dict(name="ffn tiny fp32", op=f, E=8, R=128, D=256, F=512, dtype="f32", act="swiglu", bias=True, empty=0),
        # the 20B-shaped layer's prefill batch as a training forward
        dict(name="ffn prefill", op=f, E=32, R=16384, D=2880, F=2880, dtype="bf16", act="swiglu", bias=True, empty=0),
        # the tiny fp32 layer's backward
        dict(name="ffn_backward tiny fp32", op=b, E=8, R=128, D=256, F=512, dtype="f32", act="swiglu", bias=True,
             empty=0),
        # SiLU experts without biases, ragged rows, an expert without any
        dict(name="ffn_backward ragged silu", op=b, E=8, R=1001, D=1440, F=720, dtype="bf16", act="silu", bias=False,
             empty=1),
        # the 20B-shaped layer's prefill batch, backward
        dict(name="ffn_backward prefill", op=b, E=32, R=16384, D=2880, F=2880, dtype="bf16", act="swiglu", bias=True,
             empty=0),
        # gradients of the routing weights and of the expert outputs: a small and a prefill batch
        dict(name="combine_backward 8 tokens", op=c, T=8, k=4, D=2880, dtype="bf16"),
        dict(name="combine_backward prefill", op=c, T=4096, k=4, D=2880, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "ffn", "ffn_backward", "combine_backward"])
    if op == "quantize":
        K = 32 * _log(rng, 1, 256)
        return dict(op=op, rows=min(_log(rng, 1, 100000), 250_000_000 // K), K=K, dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        E = rng.choice([1, 1, 2, 5, 8, 32])
        return dict(op=op, E=E, R=_log(rng, 1, 16384), K=32 * _log(rng, 1, 90), N=16 * _log(rng, 1, 180),
                    empty=rng.choice([0, E // 4]))
    if op == "combine_backward":
        return dict(op=op, T=_log(rng, 1, 4096), k=rng.choice([1, 2, 3, 4, 8]), D=16 * _log(rng, 1, 180),
                    dtype=rng.choice(["bf16", "f32"]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    E = rng.choice([1, 2, 5, 8, 16])
    most = 16 * 180 if dtype == "bf16" else 16 * 40      # fp32 layers are small ones
    return dict(op=op, E=E, R=_log(rng, 1, 8192 if dtype == "bf16" else 1024), D=16 * _log(rng, 1, most // 16),
                F=16 * _log(rng, 1, most // 16), dtype=dtype, act=rng.choice(["swiglu", "silu"]),
                bias=rng.choice([True, False]), empty=rng.choice([0, E // 4]))


def _rows_per_expert(case, seed):
    """Rows of each expert: every row draws an expert by uneven weights, the last `empty` experts get none."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    p = torch.rand(case["E"], generator=g) * 0.25 + 0.75
    if case["empty"]:
        p[case["E"] - case["empty"]:] = 0.0
    return torch.bincount(torch.multinomial(p, case["R"], replacement=True, generator=g), minlength=case["E"])


def _tiles(scales):
    """[G, N, K/32] scale bytes as the product's tiles: [G, N/128, K/128 (even), 32, 4, 4], 2^0 in the padding."""
    G, N, nb = scales.shape
    nt, kt = -(-N // 128), 2 * -(-nb // 8)
    full = scales.new_full((G, nt * 128, kt * 4), 127)
    full[:, :N, :nb] = scales
    return full.view(G, nt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    op, s = case["op"], dict(case)
    if op == "quantize":
        dt = DTYPES[case["dtype"]]
        x = normal(case["rows"], case["K"], std=1.0 / math.sqrt(case["K"]), dtype=dt)
        x.mul_(torch.exp2(torch.randint(-4, 4, (case["rows"], 1), generator=g, device="cuda").float()).to(dt))
        s["x"] = x
        return s
    if op == "combine_backward":
        dt, T, k, D = DTYPES[case["dtype"]], case["T"], case["k"], case["D"]
        s["dy"], s["y_perm"] = normal(T, D, dtype=dt), normal(T * k, D, dtype=dt)
        s["row_of_slot"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
        s["w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        return s
    E, R = case["E"], case["R"]
    counts = _rows_per_expert(case, seed)
    s["most"] = int(counts.max())
    s["off"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    if op == "linear":
        K, N = case["K"], case["N"]
        s["x"] = normal(R, K)
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = torch.randint(119, 128, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        s["tiles"] = _tiles(s["scales"])
        s["bias"] = normal(E, N)
        return s
    dt, D, F = DTYPES[case["dtype"]], case["D"], case["F"]
    s["x"] = normal(R, D, dtype=dt)
    s["wg"], s["wu"] = normal(E, F, D, std=D ** -0.5, dtype=dt), normal(E, F, D, std=D ** -0.5, dtype=dt)
    s["wd"] = normal(E, D, F, std=F ** -0.5, dtype=dt)
    s["bg"] = s["bu"] = s["bd"] = None
    if case["bias"]:
        s["bg"], s["bu"], s["bd"] = (normal(E, n, std=0.1, dtype=dt) for n in (F, F, D))
    if op == "ffn_backward":
        # what the forward left: pre-activations wide enough that both clips are met, and h
        s["gu"] = normal(R, 2, F, std=3.0, dtype=dt)
        s["h"] = _act(s["gu"].float(), case["act"]).to(dt)
        s["dy"] = normal(R, D, dtype=dt)
    return s


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
def _act(gu, act):
    g, u = gu[:, 0], gu[:, 1]
    if act == "silu":
        return g / (1 + torch.exp(-g)) * u
    gc, uc = g.clamp(0, LIMIT), u.clamp(-LIMIT, LIMIT)
    return gc / (1 + torch.exp(-ALPHA * gc)) * uc


def _act_grad(dh, gu, act):
    g, u = gu[:, 0], gu[:, 1]
    alpha = 1.0 if act == "silu" else ALPHA
    gc, uc = (g, u) if act == "silu" else (g.clamp(0, LIMIT), u.clamp(-LIMIT, LIMIT))
    sg = 1 / (1 + torch.exp(-alpha * gc))
    dg, du = dh * uc * (sg + alpha * gc * sg * (1 - sg)), dh * gc * sg
    if act == "silu":
        return dg, du
    return dg * ((g >= 0) & (g <= LIMIT)), du * (u.abs() <= LIMIT)


def _scale(v, n):
    """v * 2^n for whole n in [-127, 127], by two exact powers of two."""
    half = n >> 1
    power = [((k + 127) << 23).to(torch.int32).view(torch.float32) for k in (half, n - half)]
    return v * power[0] * power[1]


def _quantize(x):
    """(E2M1 values, exponents X) of fp32 rows [R, K]; ties to the even code."""
    b = x.view(x.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(2))
    X = torch.where(m > 0, torch.where(m > 0.75, e - 2, e - 3), -127).clamp(min=-127)
    v = _scale(b, -X.unsqueeze(2))
    a = v.abs()
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5).float() + (a >= 3.5) \
        + 2.0 * (a > 5)
    return torch.where(v < 0, -q, q), X


def _dequantize(q, X):
    return _scale(q, X.unsqueeze(2)).view(q.shape[0], -1)


def _decode_weights(codes, scales):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    v = torch.where(c >= 8, -grid[c & 7], grid[c & 7])
    return _scale(v.unflatten(-1, (-1, 32)), (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _spread(off, R, most):
    """Where row r sits when every expert's rows are padded to `most`: expert * most + its place there."""
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off[1:].long(), r, right=True)
    return e, e * most + r - off.long()[e]


def _pad(rows, at, E, most):
    out = rows.new_zeros(E * most, rows.shape[1])
    out[at] = rows
    return out.view(E, most, -1)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        q, X = _quantize(s["x"].float())
        return {"values": _dequantize(q, X).to(torch.bfloat16), "scales": (X + 127).to(torch.uint8)}
    if op == "combine_backward":
        dy, y, row = s["dy"].float(), s["y_perm"].float(), s["row_of_slot"].long()
        out = torch.empty_like(y)
        out[row.view(-1)] = (s["w"].unsqueeze(2) * dy.unsqueeze(1)).flatten(0, 1)
        return {"dy_perm": out.to(s["dy"].dtype), "dw": (dy.unsqueeze(1) * y[row]).sum(2)}
    E, R, most, dt = s["E"], s["R"], s["most"], s["x"].dtype
    e, at = _spread(s["off"], R, most)
    if op == "linear":
        a = _pad(_dequantize(*_quantize(s["x"].float())), at, E, most)
        y = torch.bmm(a, _decode_weights(s["codes"], s["scales"]).transpose(1, 2))
        return (y.flatten(0, 1)[at] + s["bias"].float()[e]).to(dt)
    x, wg, wu, wd = _pad(s["x"].float(), at, E, most), s["wg"].float(), s["wu"].float(), s["wd"].float()
    if op == "ffn":
        g, u = (torch.bmm(x, w.transpose(1, 2)).flatten(0, 1)[at] for w in (wg, wu))
        if s["bias"]:
            g, u = g + s["bg"].float()[e], u + s["bu"].float()[e]
        gu = torch.stack([g, u], 1)
        h = _act(gu, s["act"])
        y = torch.bmm(_pad(h, at, E, most), wd.transpose(1, 2)).flatten(0, 1)[at]
        if s["bias"]:
            y = y + s["bd"].float()[e]
        return {"gu": gu.to(dt), "h": h.to(dt), "y": y.to(dt)}
    dy = _pad(s["dy"].float(), at, E, most)
    dg, du = _act_grad(torch.bmm(dy, wd).flatten(0, 1)[at], s["gu"].float(), s["act"])
    dg, du = _pad(dg, at, E, most), _pad(du, at, E, most)
    out = {"dx": (torch.bmm(dg, wg) + torch.bmm(du, wu)).flatten(0, 1)[at],
           "dw_gate": torch.bmm(dg.transpose(1, 2), x), "dw_up": torch.bmm(du.transpose(1, 2), x),
           "dw_down": torch.bmm(dy.transpose(1, 2), _pad(s["h"].float(), at, E, most))}
    if s["bias"]:
        out |= {"db_gate": dg.sum(1), "db_up": du.sum(1), "db_down": dy.sum(1)}
    return {n: v.to(dt) for n, v in out.items()}


# --------------------------------------------------------------------------- #
# this package's calls
# --------------------------------------------------------------------------- #
def _kernels(s):
    from mixture_experts_ffn_12_b200 import api
    op = s["op"]
    if op == "quantize":
        codes, scales = api.quantize_mxfp4(s["x"])
        return {"values": api.dequantize_mxfp4(codes, scales), "scales": scales}
    if op == "linear":
        w = api.Mxfp4Weights(s["codes"], s["tiles"])
        return api.mxfp4_linear(s["x"], w, s["bias"], group_off=s["off"])
    if op == "combine_backward":
        cfg = api.make_config(s["D"], 16, max(s["k"], 1), s["k"], dtype=s["dtype"])
        dy_perm, dw = api.combine_backward(cfg, s["dy"], s["y_perm"], s["row_of_slot"], s["w"])
        return {"dy_perm": dy_perm, "dw": dw}
    cfg = api.make_config(s["D"], s["F"], s["E"], 1, LIMIT, ALPHA, dtype=s["dtype"])
    w = api.ExpertWeights(s["wg"], s["wu"], s["wd"], s["bg"], s["bu"], s["bd"])
    if op == "ffn":
        gu, h, y = api.expert_ffn_train(cfg, s["x"], s["off"], w, act=s["act"])
        return {"gu": gu, "h": h, "y": y}
    dx, grads = api.expert_ffn_backward(cfg, s["x"], s["off"], w, s["gu"], s["h"], s["dy"], act=s["act"])
    out = {"dx": dx, "dw_gate": grads.w_gate, "dw_up": grads.w_up, "dw_down": grads.w_down}
    if s["bias"]:
        out |= {"db_gate": grads.b_gate, "db_up": grads.b_up, "db_down": grads.b_down}
    return out


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    """Each input read and each output written once; the products' multiplications and additions.  Experts
    without rows need not be read, but their gradients are written."""
    op, size = case["op"], 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "quantize":
        # x read, codes and scales written, then read, and the values written
        n = case["rows"] * case["K"]
        return {"bytes": n * (size + 2 * (0.5 + 1 / 32) + 2), "flops": 2 * n}
    if op == "combine_backward":
        T, k, D = case["T"], case["k"], case["D"]
        return {"bytes": T * D * size * (1 + 2 * k) + 12 * T * k, "flops": 3 * T * k * D}
    E, R = case["E"], case["R"]
    with_rows = min(R, E - case["empty"])
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * R * (K + N) + with_rows * N * (K * (0.5 + 1 / 32) + 2), "flops": 2 * R * K * N}
    D, F = case["D"], case["F"]
    if op == "ffn":
        return {"bytes": size * (2 * R * D + 3 * R * F + 3 * with_rows * D * F), "flops": 6 * R * D * F}
    return {"bytes": size * (3 * R * D + 3 * R * F + 3 * with_rows * D * F + 3 * E * D * F),
            "flops": 12 * R * D * F}


# --------------------------------------------------------------------------- #
# the definition in 64 bits, expert by expert
# --------------------------------------------------------------------------- #
def _exact_mxfp4(x):
    """Blocks of 32 rounded to the E2M1 grid times 2^X, by distance to every grid value."""
    blocks = x.double().reshape(-1, 32)
    amax = blocks.abs().amax(1)
    X = torch.ceil(torch.log2(amax / 6)).clamp(-127, 127)
    X = torch.where(amax > 6 * torch.exp2(X), X + 1, X)                    # where the logarithm was rounded
    X = torch.where((amax <= 3 * torch.exp2(X)) & (X > -127), X - 1, X)
    X = torch.where(amax == 0, torch.full_like(X, -127), X)
    v = blocks.abs() / torch.exp2(X)[:, None]
    best, at = torch.full_like(v, math.inf), torch.zeros_like(v)
    for code, value in enumerate([0, .5, 1, 1.5, 2, 3, 4, 6]):
        d = (v - value).abs()
        take = (d < best) | ((d == best) & (code % 2 == 0))
        best, at = torch.where(take, d, best), torch.where(take, torch.full_like(at, float(value)), at)
    return (at * torch.exp2(X)[:, None] * torch.sign(blocks)).reshape(x.shape), (X + 127).reshape(x.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        parts = [_exact_mxfp4(p) for p in s["x"].split(8192)]
        return {"values": torch.cat([p[0] for p in parts]),
                "scales": torch.cat([p[1] for p in parts]).to(torch.uint8)}
    if op == "combine_backward":
        dy, y, w, k = s["dy"].double(), s["y_perm"].double(), s["w"].double(), s["k"]
        out, dw = torch.empty_like(y), torch.empty_like(w)
        for j in range(k):
            row = s["row_of_slot"][:, j].long()
            out[row] = dy * w[:, j:j + 1]
            dw[:, j] = torch.einsum("td,td->t", dy, y[row])
        return {"dy_perm": out, "dw": dw}
    off = s["off"].tolist()
    x = s["x"].double()
    names = {"linear": ["y"], "ffn": ["gu", "h", "y"]}.get(op, ["dx"])
    per_expert = ["dw_gate", "dw_up", "dw_down"] + (["db_gate", "db_up", "db_down"] if s.get("bg") is not None else [])
    rows, grads = {n: [] for n in names}, {n: [] for n in per_expert}
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=x.device).double()
    alpha = 1.0 if s.get("act") == "silu" else ALPHA

    def clip(t, lo):
        return t if s["act"] == "silu" else torch.minimum(torch.maximum(t, t.new_tensor(lo)), t.new_tensor(LIMIT))

    for e in range(s["E"]):
        xe = x[off[e]:off[e + 1]]
        if op == "linear":
            c = s["codes"][e].long()
            w = torch.empty(s["N"], s["K"], dtype=torch.float64, device=x.device)
            w[:, 0::2], w[:, 1::2] = grid[c % 16], grid[c // 16]
            w *= torch.exp2(s["scales"][e].double() - 127).repeat_interleave(32, 1)
            rows["y"].append((_exact_mxfp4(xe)[0] if len(xe) else xe) @ w.T + s["bias"][e].double())
            continue
        wg, wu, wd = s["wg"][e].double(), s["wu"][e].double(), s["wd"][e].double()
        if op == "ffn":
            g, u = xe @ wg.T, xe @ wu.T
            if s["bias"]:
                g, u = g + s["bg"][e].double(), u + s["bu"][e].double()
            h = clip(g, 0.0) * torch.sigmoid(alpha * clip(g, 0.0)) * clip(u, -LIMIT)
            y = h @ wd.T + (s["bd"][e].double() if s["bias"] else 0.0)
            for n, v in (("gu", torch.stack([g, u], 1)), ("h", h), ("y", y)):
                rows[n].append(v)
            continue
        dy, gu = s["dy"][off[e]:off[e + 1]].double(), s["gu"][off[e]:off[e + 1]].double()
        g, u, dh = gu[:, 0], gu[:, 1], dy @ wd
        sg = torch.sigmoid(alpha * clip(g, 0.0))
        du = dh * clip(g, 0.0) * sg
        dg = dh * clip(u, -LIMIT) * sg * (1 + alpha * clip(g, 0.0) * (1 - sg))
        if s["act"] != "silu":
            dg, du = dg.masked_fill((g < 0) | (g > LIMIT), 0.0), du.masked_fill((u > LIMIT) | (u < -LIMIT), 0.0)
        rows["dx"].append(dg @ wg + du @ wu)
        h = s["h"][off[e]:off[e + 1]].double()
        for n, v in (("dw_gate", dg.T @ xe), ("dw_up", du.T @ xe), ("dw_down", dy.T @ h)):
            # a bf16 layer's are held in 32 bits: all of them take 6.4 GB in 64
            grads[n].append(v.float() if s["dtype"] == "bf16" else v)
        if "db_gate" in grads:
            for n, v in (("db_gate", dg), ("db_up", du), ("db_down", dy)):
                grads[n].append(v.sum(0))
    if op == "linear":
        return torch.cat(rows["y"])
    out = {n: torch.cat(v) for n, v in rows.items()}
    if op == "ffn_backward":
        out |= {n: torch.stack(v) for n, v in grads.items()}
    return out
