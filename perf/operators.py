"""Cases, plain forms and exact values of the expert-layer operators.

Two families that a mixture-of-experts layer trained with Muon uses together:

- matrix products grouped by expert: rows of `x` are sorted by expert, expert
  e owns rows offsets[e] .. offsets[e+1]; the forward product
  y = x W_e^T, its gradient for the rows dx = dy W_e, and its gradient for
  the weights, dW_e = beta dW_e + dy_e^T x_e (beta = the momentum decay when
  the products go straight into Muon's momentum);
- the orthogonalised update of stacks of matrices (experts, attention heads,
  blocks of a fused projection): momentum, Newton-Schulz, decayed weights.

`own = False` computes them with elementary torch operations in 32 bits,
`own = True` makes the framework's calls.
"""

import math

import torch

own = False

STEPS = 5
ABC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token to each of a few experts: the latency of a single decoding step
        dict(name="y_decode_8", op="y", experts=8, tokens=8, n=1024, k=768, dtype="bf16", skew=0.0, behind=0),
        # a decoding batch over many experts: every weight is read for a handful of rows
        dict(name="y_decode_256", op="y", experts=64, tokens=256, n=2048, k=2048, dtype="bf16", skew=0.5, behind=0),
        # a ragged training batch in fp16, some experts empty, rows behind the last expert untouched
        dict(name="y_ragged_4k", op="y", experts=16, tokens=4099, n=4096, k=1024, dtype="f16", skew=1.5, behind=61),
        # a large training batch
        dict(name="y_train_32k", op="y", experts=64, tokens=32768, n=4096, k=2048, dtype="bf16", skew=0.5, behind=0),
        # the gradient for the rows, with a width that is no multiple of the tile
        dict(name="dx_8k", op="dx", experts=32, tokens=8191, n=1416, k=2048, dtype="bf16", skew=1.0, behind=0),
        # the gradient for the weights of a small layer, into the fp32 momentum
        dict(name="dw_2k", op="dw", experts=8, tokens=2048, n=768, k=768, dtype="bf16", out="f32", beta=0.95, skew=1.0, behind=0),
        # the gradient for the weights of a large layer, in the weights' type
        dict(name="dw_32k", op="dw", experts=64, tokens=32768, n=2048, k=1024, dtype="bf16", out="bf16", beta=0.0, skew=0.5, behind=0),
        # per-head update of one attention projection (heads are row blocks of one matrix)
        dict(name="step_heads", op="step", count=12, rows=64, cols=768, fused=1, weight="f32", grad="f32", compute="f16x2", nesterov=True, copy="", decay=0.0),
        # a few expert matrices of odd size, 16-bit weights
        dict(name="step_odd", op="step", count=5, rows=333, cols=200, fused=0, weight="bf16", grad="bf16", compute="f16x2", nesterov=False, copy="", decay=0.1),
        # expert stacks in bf16: the fast form
        dict(name="step_bf16_32", op="step", count=32, rows=1024, cols=2048, fused=0, weight="bf16", grad="bf16", compute="bf16", nesterov=True, copy="", decay=0.1),
        # fp32 master weights with the 16-bit copy that the products read; gate and up blocks of a fused projection
        dict(name="step_f16x2_32", op="step", count=32, rows=1024, cols=2048, fused=0, weight="f32", grad="bf16", compute="f16x2", nesterov=True, copy="bf16", decay=0.1),
        # a whole layer: forward, both gradients (the weights' into the momentum), update
        dict(name="layer_8k", op="layer", experts=16, tokens=8192, n=2048, k=1024, dtype="bf16", skew=1.0, behind=0, compute="f16x2", decay=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rows_of(rng, lo, hi):
    return 8 * _log(rng, lo / 8, hi / 8)  # 16-byte rows, as every 16-bit product needs


def draw(rng):
    op = rng.choice(["y", "y", "dx", "dx", "dw", "dw", "step", "step", "step", "layer"])
    if op == "step":
        rows, cols = _log(rng, 32, 2048), _log(rng, 32, 2048)
        count = max(1, min(_log(rng, 1, 48), int(32 * 1024 * 1024 * 2048 / (rows * cols * min(rows, cols)))))
        weight = rng.choice(["f32", "bf16"])
        return dict(op=op, count=count, rows=rows, cols=cols, fused=rng.choice([0, 1]), weight=weight, grad=rng.choice(["f32", "bf16"]),
                    compute=rng.choice(["f16x2", "bf16"]) if weight == "bf16" else "f16x2", nesterov=rng.random() < 0.5,
                    copy=rng.choice(["", "bf16"]) if weight == "f32" else "", decay=rng.choice([0.0, 0.1]))
    experts, tokens = _log(rng, 1, 64), _log(rng, 1, 32768)
    case = dict(op=op, experts=experts, tokens=tokens, n=_rows_of(rng, 64, 4096), k=_rows_of(rng, 64, 2048), dtype=rng.choice(["bf16", "f16"]),
                skew=rng.choice([0.0, 0.5, 1.0, 1.5]), behind=rng.choice([0, 0, 17]))
    if op == "dw":
        case.update(out=rng.choice(["f32", "16"]), beta=rng.choice([0.0, 0.95]))
        case["out"] = case["dtype"] if case["out"] == "16" else "f32"
        if case["out"] != "f32":
            case["beta"] = 0.0
    if op == "layer":
        case.update(experts=min(experts, 16), tokens=min(tokens, 8192), n=_rows_of(rng, 64, 2048), k=_rows_of(rng, 64, 1024), dtype="bf16",
                    behind=0, compute="f16x2", decay=rng.choice([0.0, 0.1]))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _counts(case, seed):
    """Rows per expert, from the seed: log-normal shares of the tokens, so with skew some experts get none."""
    g = torch.Generator().manual_seed(seed * 7 + 3)
    share = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g, dtype=torch.float64), 0)
    return torch.bincount(torch.multinomial(share, case["tokens"], replacement=True, generator=g), minlength=case["experts"])


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _spectrum(gen, count, rows, cols, std):
    """What a momentum or gradient looks like: a few strong directions over noise, rows of unequal size."""
    rank = max(1, min(rows, cols) // 16)
    low = torch.bmm(_normal(gen, (count, rows, rank), 1.0, torch.float32), _normal(gen, (count, rank, cols), rank ** -0.5, torch.float32))
    return (0.5 * low + _normal(gen, (count, rows, cols), 1.0, torch.float32)) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "step":
        count, rows, cols = case["count"], case["rows"], case["cols"]
        s["W"] = _normal(gen, (count, rows, cols), 0.02, DTYPES[case["weight"]])
        s["M"] = _spectrum(gen, count, rows, cols, 3e-3)
        s["G"] = _spectrum(gen, count, rows, cols, 1e-3).to(DTYPES[case["grad"]])
        if case["copy"]:
            s["copy"] = torch.empty((count, rows, cols), dtype=DTYPES[case["copy"]], device="cuda")
        if case["fused"] == 1:  # row blocks of one matrix whose rows are padded
            pad = (cols + 8 + 7) // 8 * 8
            for name in ("W", "M"):
                wide = torch.zeros((count * rows, pad), dtype=s[name].dtype, device="cuda")
                wide[:, :cols] = s[name].reshape(count * rows, cols)
                s[name] = wide.view(count, rows, pad)[:, :, :cols]
    else:
        experts, tokens, n, k = case["experts"], case["tokens"], case["n"], case["k"]
        dtype = DTYPES[case["dtype"]]
        counts = _counts(case, seed)
        s["longest"] = int(counts.max())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        total = tokens + case["behind"]
        if op in ("y", "dw", "layer"):
            s["x"] = _normal(gen, (total, k), 1.0, dtype)
        if op in ("dx", "dw", "layer"):
            s["dy"] = _normal(gen, (total, n), 1e-3, dtype)
        if op in ("y", "dx", "layer"):
            s["w"] = _normal(gen, (experts, n, k), 0.02, dtype)
        if op == "y":
            s["y"] = torch.full((total, n), 0.25, dtype=dtype, device="cuda")
        if op == "dx":
            s["dx"] = torch.full((total, k), 0.25, dtype=dtype, device="cuda")
        if op == "dw":
            s["dw"] = _normal(gen, (experts, n, k), 0.02, DTYPES[case["out"]])
        if op == "layer":
            s["y"] = torch.empty((total, n), dtype=dtype, device="cuda")
            s["dx"] = torch.empty((total, k), dtype=dtype, device="cuda")
            s["W"] = s["w"].float()
            s["M"] = _spectrum(gen, experts, n, k, 1e-2)
    if own:
        _plan(s)
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------


def _update_scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))  # update entries of root mean square about 0.2


LR = 2e-3


def _plan(s):
    """What a program keeps between steps: the prepared update and the workspaces."""
    from newton_schulz_10_b200 import muon as mu

    case = s["case"]
    if case["op"] in ("step", "layer"):
        compute = {"f16x2": mu.F16X2, "bf16": mu.BF16}[case["compute"]]
        rows, cols = s["W"].shape[1:]
        p = mu.stack_params(mu=0.95, lr=LR, weight_decay=case["decay"], scale=_update_scale(rows, cols),
                            nesterov=bool(case.get("nesterov")), ns=mu.ns_params(T=STEPS, coeffs=ABC, norm_eps=EPS, compute=compute))
        copy = s["w"] if case["op"] == "layer" else s.get("copy")
        s["step"] = mu.StackStep([mu.Stack(s["W"], s["M"], s.get("G"), copy)], p)
    if case["op"] == "dw":
        s["ws"] = mu.workspace(mu.grouped_workspace_size(case["experts"]))


def _run_own(s):
    from newton_schulz_10_b200 import muon as mu

    op = s["case"]["op"]
    if op == "y":
        return mu.grouped_matmul(s["x"], s["w"], s["offsets"], out=s["y"])
    if op == "dx":
        return mu.grouped_matmul_dx(s["dy"], s["w"], s["offsets"], out=s["dx"])
    if op == "dw":
        return mu.grouped_matmul_dw(s["dy"], s["x"], s["offsets"], out=s["dw"], beta=s["case"]["beta"], ws=s["ws"])
    if op == "step":
        s["step"]()
        return _step_outputs(s)
    mu.grouped_matmul(s["x"], s["w"], s["offsets"], out=s["y"])
    mu.grouped_matmul_dx(s["dy"], s["w"], s["offsets"], out=s["dx"])
    s["step"].accumulate(0, s["dy"], s["x"], s["offsets"])
    s["step"]()
    return _layer_outputs(s)


def _step_outputs(s):
    got = {"W": s["W"], "M": s["M"]}
    if "copy" in s:
        got["copy"] = s["copy"]
    return got


def _layer_outputs(s):
    return {"y": s["y"], "dx": s["dx"], "M": s["M"], "W": s["W"], "w": s["w"]}


# ---------------------------------------------------------------------------
# the plain forms, 32 bits throughout
# ---------------------------------------------------------------------------


def _rows(s, device_rows):
    """(index of each expert's rows, padded to the longest; which of them are its own)"""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["longest"], device=off.device)[None, :]
    mine = at < off[1:, None]
    return torch.where(mine, at, torch.full_like(at, device_rows)), mine


def _gather(x, at, mine):
    rows = x.float()[at.clamp(max=x.shape[0] - 1)]
    return torch.where(mine[:, :, None], rows, torch.zeros((), device=x.device))


def _scatter(out, at, values):
    """values to their rows of out; the padding goes to a row behind, which is dropped"""
    wide = torch.cat([out, out[:1]])
    wide[at.reshape(-1)] = values.reshape(-1, values.shape[-1]).to(out.dtype)
    out.copy_(wide[:-1])
    return out


def _plain_product(s, x, w, out):
    at, mine = _rows(s, x.shape[0])
    return _scatter(out, at, torch.bmm(_gather(x, at, mine), w))


def _plain_dw(s, out, beta):
    at, mine = _rows(s, s["x"].shape[0])
    dw = torch.bmm(_gather(s["dy"], at, mine).transpose(1, 2), _gather(s["x"], at, mine))
    out.copy_(dw + beta * out.float() if beta else dw)
    return out


def _plain_polar(X):
    a, b, c = ABC
    tall = X.shape[1] > X.shape[2]
    X = X.transpose(1, 2) if tall else X
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = torch.bmm(X, X.transpose(1, 2))
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    return X.transpose(1, 2) if tall else X


def _plain_update(W, M, nesterov_grad, copy, decay):
    X = M if nesterov_grad is None else nesterov_grad.float() + 0.95 * M
    O = _plain_polar(X)
    new = (1.0 - LR * decay) * W.float() - LR * _update_scale(*W.shape[1:]) * O
    W.copy_(new)
    if copy is not None:
        copy.copy_(new)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "y":
        return _plain_product(s, s["x"], s["w"].float().transpose(1, 2), s["y"])
    if op == "dx":
        return _plain_product(s, s["dy"], s["w"].float(), s["dx"])
    if op == "dw":
        return _plain_dw(s, s["dw"], case["beta"])
    if op == "step":
        s["M"].copy_(0.95 * s["M"] + s["G"].float())
        _plain_update(s["W"], s["M"], s["G"] if case["nesterov"] else None, s.get("copy"), case["decay"])
        return _step_outputs(s)
    _plain_product(s, s["x"], s["w"].float().transpose(1, 2), s["y"])
    _plain_product(s, s["dy"], s["w"].float(), s["dx"])
    _plain_dw(s, s["M"], 0.95)
    _plain_update(s["W"], s["M"], None, s["w"], case["decay"])
    return _layer_outputs(s)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def _size(name):
    return {"bf16": 2, "f16": 2, "f32": 4}[name]


def _step_flops(count, rows, cols):
    n, m = min(rows, cols), max(rows, cols)
    return count * STEPS * (3.0 * m * n * n + float(n) ** 3)  # symmetric products as one triangle


def work(case):
    op = case["op"]
    if op == "step":
        el = case["count"] * case["rows"] * case["cols"]
        per = 2 * 4 + _size(case["grad"]) + 2 * _size(case["weight"]) + (_size(case["copy"]) if case["copy"] else 0)
        return {"bytes": float(el * per), "flops": _step_flops(case["count"], case["rows"], case["cols"])}
    experts, tokens, n, k = case["experts"], case["tokens"], case["n"], case["k"]
    flops = 2.0 * tokens * n * k
    used = min(experts, tokens)
    rows, weights = 2.0 * tokens * (n + k), 2.0 * used * n * k
    if op in ("y", "dx"):
        return {"bytes": rows + weights, "flops": flops}
    if op == "dw":
        out = _size(case["out"]) * experts * n * k * (2 if case["beta"] else 1)
        return {"bytes": rows + out, "flops": flops}
    el = float(experts * n * k)
    return {"bytes": 3 * rows + 2 * weights + el * (2 * 4 + 2 * 4 + 2), "flops": 3 * flops + _step_flops(experts, n, k)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, expert by expert and matrix by matrix
# ---------------------------------------------------------------------------


def _exact_polar(A):
    """Newton-Schulz of one matrix, p(X) = a X + b (X X^T) X + c (X X^T)^2 X, on the side that is shorter."""
    a, b, c = ABC
    X = A / (torch.linalg.matrix_norm(A) + EPS)
    eye = torch.eye(min(A.shape), dtype=torch.float64, device=A.device)
    for _ in range(STEPS):
        if A.shape[0] <= A.shape[1]:
            G = X @ X.T
            X = (a * eye + (b * eye + c * G) @ G) @ X
        else:
            G = X.T @ X
            X = X @ (a * eye + G @ (b * eye + c * G))
    return X


def _exact_step(W, M, G, nesterov, decay):
    """(W, M) after one update, in 64 bits"""
    W, M = W.double().clone(), M.double().clone()
    step = LR * _update_scale(W.shape[1], W.shape[2])
    for i in range(W.shape[0]):
        if G is not None:
            M[i] = 0.95 * M[i] + G[i].double()
        target = 0.95 * M[i] + G[i].double() if nesterov else M[i]
        W[i] = W[i] - LR * decay * W[i] - step * _exact_polar(target)
    return W, M


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        W, M = _exact_step(s["W"], s["M"], s["G"], case["nesterov"], case["decay"])
        got = {"W": W, "M": M}
        if "copy" in s:
            got["copy"] = W
        return got
    off = s["offsets"].tolist()
    spans = [(e, slice(off[e], off[e + 1])) for e in range(case["experts"]) if off[e + 1] > off[e]]
    if op in ("y", "layer"):
        y = s["y"].double()
        for e, r in spans:
            y[r] = s["x"][r].double() @ s["w"][e].double().T
        if op == "y":
            return y
    if op in ("dx", "layer"):
        dx = s["dx"].double()
        for e, r in spans:
            dx[r] = s["dy"][r].double() @ s["w"][e].double()
        if op == "dx":
            return dx
    beta = case["beta"] if op == "dw" else 0.95
    dw = beta * (s["dw"] if op == "dw" else s["M"]).double()
    for e, r in spans:
        dw[e] += s["dy"][r].double().T @ s["x"][r].double()
    if op == "dw":
        return dw
    W, M = _exact_step(s["W"], dw, None, False, case["decay"])
    return {"y": y, "dx": dx, "M": M, "W": W, "w": W}
