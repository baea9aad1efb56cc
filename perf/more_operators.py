"""Cases of the operators around the table operators: products of the rows in
unit order with each unit's matrix, root-mean-square norm of rows with the
residual's addition, and scores over a table held in 8 bits.

`run` computes a case in plain torch operations (`own` false) or through the
package's entry points (`own` true); `exact` computes it in 64 bits.

Kinds of case:
  units        rows in unit order (unit g's are rows offsets[g] .. offsets[g + 1]
               - 1) times their unit's matrix, which holds a row per output
               column; rows of no unit give zeros
  units_grad   the same and its backward pass: gradients of the rows and of the
               units' matrices
  norm         h = x + residual, rounded to the rows' type, and h / rms(h) times
               a weight per column
  norm_grad    the same and its backward pass: the gradient of x (and of the
               residual, the same), with the one that reaches h from behind, and
               the weight's
  scores       rows quantized to 8 bits with one scale each (codes -127 .. 127,
               the largest magnitude at 127), and their products with a table in
               8 bits with one scale per row
  norm_scores  the norm of rows plus residual, its output in 8 bits with a scale
               per row, and the products with the table
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}

EPS = 1e-6


def listed():
    """The listed cases; the comment above each says what it stands for."""
    return [
        # one decoding step: 16 sequences through 2 of 64 units each
        dict(name="units_step", kind="units", m=32, groups=64, d=1024, cols=2048,
             dtype="bfloat16", spread="even", missing=0.0),
        # a prompt of 32,768 rows through 2 of 128 units each, some units liked better
        dict(name="units_prompt", kind="units", m=65536, groups=128, d=2048, cols=2048,
             dtype="bfloat16", spread="skewed", missing=0.0),
        # full precision at odd sizes, with entries dropped for want of room
        dict(name="units_odd", kind="units", m=12291, groups=100, d=250, cols=333,
             dtype="float32", spread="skewed", missing=0.05),
        # training at odd sizes, with few rows for each unit
        dict(name="units_grad_odd", kind="units_grad", m=2501, groups=60, d=257, cols=515,
             dtype="float16", spread="skewed", missing=0.1),
        # a training batch of 16,384 rows through 4 of 64 units each
        dict(name="units_grad_batch", kind="units_grad", m=65536, groups=64, d=2048, cols=1024,
             dtype="bfloat16", spread="even", missing=0.0),
        # one decoding step of 16 sequences
        dict(name="norm_step", kind="norm", n=16, d=4096, dtype="bfloat16", residual=True),
        # training at an odd width
        dict(name="norm_grad_odd", kind="norm_grad", n=1023, d=257, dtype="float16",
             residual=False),
        # a training batch, the residual's gradient with it
        dict(name="norm_grad_batch", kind="norm_grad", n=16384, d=2048, dtype="bfloat16",
             residual=True),
        # one query over the 512 x 512 map's codebook
        dict(name="scores_one", kind="scores", n=1, groups=262144, d=256, dtype="bfloat16",
             out="float32"),
        # some queries in full precision over an embedding table, odd width
        dict(name="scores_odd", kind="scores", n=37, groups=8359, d=767, dtype="float32",
             out="float32"),
        # a decoding batch against a wide output table
        dict(name="norm_scores_step", kind="norm_scores", n=16, groups=65536, d=4096,
             dtype="float16", residual=True, out="float32"),
        # a prompt through one projection
        dict(name="norm_scores_prompt", kind="norm_scores", n=8192, groups=16384, d=4096,
             dtype="bfloat16", residual=True, out="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    """Seconds at 5 TB/s and at 1,000 (float32: 125) TFLOP/s, whichever is more."""
    w = work(case)
    slow = case["kind"].startswith("units") and case["dtype"] == "float32"
    return max(w["bytes"] / 5e12, w["flops"] / (1.25e14 if slow else 1e15))


def draw(rng):
    """One more case of the listed ones' ranges."""
    top = max(_cost(c) for c in listed())
    kind = rng.choice(["units", "units_grad", "norm", "norm_grad", "scores", "norm_scores"])
    dtype = rng.choice(sorted(DTYPES))
    while True:
        case = dict(kind=kind, dtype=dtype)
        if kind.startswith("units"):
            case.update(m=_log_int(rng, 1, 65536), groups=_log_int(rng, 4, 256),
                        d=_log_int(rng, 16, 2048), cols=_log_int(rng, 16, 2048),
                        spread=rng.choice(["even", "skewed"]),
                        missing=rng.choice([0.0, 0.0, 0.05, 0.2]))
            if rng.random() < 0.5:
                case["d"] -= case["d"] % 8
                case["cols"] -= case["cols"] % 8
            if case["groups"] * case["d"] * case["cols"] > 128 * 2048 * 2048:
                continue
        else:
            case.update(n=_log_int(rng, 1, 16384), d=_log_int(rng, 16, 4096),
                        residual=kind == "norm_scores" or rng.random() < 0.5)
            if rng.random() < 0.5:
                case["d"] -= case["d"] % 8
            if kind.endswith("scores"):
                case.update(groups=_log_int(rng, 16, 262144),
                            out=rng.choice(["float32", "float32", dtype]))
                if kind == "scores":
                    case["residual"] = False
                if case["groups"] * case["d"] > 65536 * 4096 or \
                        case["n"] * case["groups"] > 8192 * 16384:
                    continue
        if _cost(case) <= top:
            return case


def work(case):
    """Bytes and operations of one pass: inputs once, outputs once."""
    kind, d, b = case["kind"], case["d"], DTYPES[case["dtype"]].itemsize
    if kind.startswith("units"):
        g, cols = case["groups"], case["cols"]
        m = case["m"] * (1.0 - case["missing"])
        hit = g * (1.0 - (1.0 - 1.0 / g) ** m)  # units that have a row, about
        total = 4 * (g + 1) + m * d * b + hit * d * cols * b + case["m"] * cols * b
        flops = 2.0 * m * d * cols
        if kind == "units_grad":
            # dY -> dX, dW (rows and matrices counted above)
            total += m * cols * b + case["m"] * d * b + g * d * cols * b
            flops *= 3.0
        return {"bytes": total, "flops": flops}
    n = case["n"]
    row = n * d * b
    if kind == "scores":
        g, o = case["groups"], DTYPES[case["out"]].itemsize
        return {"bytes": row + g * (d + 4) + n * g * o, "flops": 2.0 * n * g * d}
    total = row + d * b + (2 * row if case["residual"] else 0)  # x, weight; residual, h
    if kind == "norm_scores":
        g, o = case["groups"], DTYPES[case["out"]].itemsize
        return {"bytes": total + g * (d + 4) + n * g * o, "flops": 2.0 * n * g * d}
    total += row  # y
    flops = 5.0 * n * d
    if kind == "norm_grad":
        # dY, what reaches h, h -> dX, dweight
        total += 3 * row + (row if case["residual"] else 0) + d * b
        flops += 8.0 * n * d
    return {"bytes": total, "flops": flops}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    return g


def _normal(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _offsets(case, gen):
    """Places where the units' rows begin, int32 [groups + 1]: the rows' units
    drawn evenly or with some liked up to e^2 times better; a share of the rows
    belongs to none and lies behind."""
    m, g = case["m"], case["groups"]
    logits = torch.zeros(g, device="cuda", dtype=torch.float64)
    if case["spread"] == "skewed":
        logits = torch.linspace(2.0, 0.0, g, device="cuda", dtype=torch.float64)[
            torch.randperm(g, generator=gen, device="cuda")]
    edges = torch.cumsum(torch.softmax(logits, 0), 0)
    u = torch.rand(m, generator=gen, device="cuda", dtype=torch.float64)
    unit = torch.searchsorted(edges, u).clamp_(max=g - 1)
    gone = torch.rand(m, generator=gen, device="cuda") < case["missing"]
    count = torch.bincount(torch.where(gone, torch.full_like(unit, g), unit), minlength=g + 1)
    offsets = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(count[:g], 0)
    return offsets


def _table8(nc, d, gen):
    """A normally distributed table in 8-bit codes with one scale per row."""
    codes = torch.empty((nc, d), dtype=torch.int8, device="cuda")
    scales = torch.empty(nc, device="cuda")
    for lo in range(0, nc, 65536):
        w = torch.randn((min(nc, lo + 65536) - lo, d), generator=gen, device="cuda") * 0.05
        s = w.abs().amax(1) / 127.0
        codes[lo:lo + 65536] = torch.round(w / s[:, None]).clamp_(-127, 127).to(torch.int8)
        scales[lo:lo + 65536] = s
    return codes, scales


def prepare(case, seed):
    gen = _gen(seed)
    dt, kind, d = DTYPES[case["dtype"]], case["kind"], case["d"]
    state = dict(case=case)
    if kind.startswith("units"):
        m, g, cols = case["m"], case["groups"], case["cols"]
        state["offsets"] = _offsets(case, gen)
        live = (torch.arange(m, device="cuda") < state["offsets"][-1])[:, None]
        state["Xs"] = _normal((m, d), dt, gen) * live
        state["W"] = _normal((g, cols, d), dt, gen, 1.0 / math.sqrt(d))
        if kind == "units_grad":
            state["dYs"] = _normal((m, cols), dt, gen) * live
        return state
    n = case["n"]
    state["X"] = _normal((n, d), dt, gen)
    if kind != "scores":
        state["weight"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        state["R"] = _normal((n, d), dt, gen, 2.0) if case["residual"] else None
    if kind == "norm_grad":
        state["dY"] = _normal((n, d), dt, gen)
        state["dH"] = _normal((n, d), dt, gen) if case["residual"] else None
    if kind.endswith("scores"):
        state["codes"], state["scales"] = _table8(case["groups"], d, gen)
    return state


# -------------------------------------------------------------- plain form --

def _plain_units(state):
    """A product for each unit that has rows, as a program without the operator
    does it: it has to know the offsets on the host."""
    X, W, dY, dt = state["Xs"], state["W"], state.get("dYs"), state["Xs"].dtype
    off = state["offsets"].tolist()
    Y = X.new_zeros((X.shape[0], W.shape[1]))
    dX = torch.zeros_like(X)
    dW = torch.zeros_like(W) if dY is not None else None
    for g, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            x, w = X[lo:hi].float(), W[g].float()
            Y[lo:hi] = (x @ w.t()).to(dt)
            if dY is not None:
                dy = dY[lo:hi].float()
                dX[lo:hi] = (dy @ w).to(dt)
                dW[g] = (dy.t() @ x).to(dt)
    return dict(Y=Y, dX=dX, dW=dW) if dY is not None else Y


def _plain_sum(state):
    X, R = state["X"], state["R"]
    return X if R is None else (X.float() + R.float()).to(X.dtype)


def _plain_quantize(v):
    """Codes (in 64 bits where a value is next to a border) and the largest
    magnitude of each row."""
    top = v.abs().amax(1, keepdim=True)
    codes = torch.round(v.double() * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    return codes.float(), top


def _plain_products(codes, scales, table, table_scales):
    """Products of whole numbers, 1,024 columns at a time, within which 32-bit
    sums of them stay exact."""
    total = None
    for lo in range(0, table.shape[1], 1024):
        part = codes[:, lo:lo + 1024] @ table[:, lo:lo + 1024].float().t()
        total = part.int() if total is None else total.add_(part.int())
    return total.float() * scales * table_scales


def _plain(state):
    case = state["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind.startswith("units"):
        return _plain_units(state)
    if kind == "scores":
        codes, top = _plain_quantize(state["X"].float())
        return _plain_products(codes, top / 127.0, state["codes"],
                               state["scales"]).to(DTYPES[case["out"]])
    H = _plain_sum(state)
    h, w = H.float(), state["weight"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    if kind == "norm_scores":
        codes, top = _plain_quantize(h * w)
        return dict(H=H, y=_plain_products(codes, top * rstd / 127.0, state["codes"],
                                           state["scales"]).to(DTYPES[case["out"]]))
    xhat = h * rstd
    out = dict(Y=(xhat * w).to(dt))
    if case["residual"]:
        out["H"] = H
    if kind == "norm_grad":
        dY = state["dY"].float()
        g = dY * w
        dX = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if state["dH"] is not None:
            dX = dX + state["dH"].float()
        out.update(dX=dX.to(dt), dweight=(dY * xhat).sum(0).to(dt))
    return out


# ------------------------------------------------------------- the kernels --

def _kernels(state):
    import farthest_vector_search_amd as vs
    case = state["case"]
    kind = case["kind"]
    if kind.startswith("units"):
        X, W, offsets = state["Xs"], state["W"], state["offsets"]
        Y = vs.vs_unit_products(X, W, offsets)
        if kind == "units":
            return Y
        dX, dW = vs.vs_unit_products_backward(state["dYs"], X, W, offsets)
        return dict(Y=Y, dX=dX, dW=dW)
    if kind == "scores":
        codes, scales = vs.vs_q8_quantize(state["X"])
        return vs.vs_q8_scores(codes, scales, state["codes"], state["scales"],
                               out_dtype=DTYPES[case["out"]])
    if kind == "norm_scores":
        codes, scales, H = vs.vs_norm_rows_q8(state["X"], state["weight"], EPS,
                                              residual=state["R"])
        return dict(H=H, y=vs.vs_q8_scores(codes, scales, state["codes"], state["scales"],
                                           out_dtype=DTYPES[case["out"]]))
    Y, H, rstd = vs.vs_norm_rows(state["X"], state["weight"], EPS, residual=state["R"])
    out = dict(Y=Y)
    if case["residual"]:
        out["H"] = H
    if kind == "norm_grad":
        out["dX"], out["dweight"] = vs.vs_norm_rows_backward(state["dY"], H, state["weight"],
                                                             rstd, dH=state["dH"])
    return out


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------- exact --

def _exact_products(c, s, state):
    """Codes c (64-bit) and scales s of the rows against the table."""
    y = torch.empty((c.shape[0], state["codes"].shape[0]), dtype=torch.float64, device="cuda")
    for lo in range(0, y.shape[1], 8192):
        rows = state["codes"][lo:lo + 8192].double()
        y[:, lo:lo + 8192] = torch.matmul(rows * state["scales"][lo:lo + 8192, None].double(),
                                          (c * s).t().contiguous()).t()
    return y


def _exact_codes(v):
    """The whole number nearest to 127 v / max |v|, ties to even."""
    top = v.abs().max(1, keepdim=True).values
    c = torch.round((127.0 * v) / top.clamp(min=1e-300))
    return c, top / 127.0


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    kind, f64 = case["kind"], torch.float64
    if kind.startswith("units"):
        m, g = case["m"], case["groups"]
        X, W = s["Xs"], s["W"]
        ends = s["offsets"].long().cpu()
        unit = torch.bucketize(torch.arange(m), ends[1:].contiguous(), right=True).cuda()
        Y = torch.zeros((m, case["cols"]), dtype=f64, device="cuda")
        dX = torch.zeros((m, case["d"]), dtype=f64, device="cuda")
        dW = torch.zeros(W.shape if kind == "units_grad" else (0,), dtype=f64, device="cuda")
        for u in range(g):
            at = torch.nonzero(unit == u).flatten()
            w = W[u].double()
            Y[at] = torch.matmul(w, X[at].double().t().contiguous()).t()
            if kind == "units_grad":
                dy = s["dYs"][at].double()
                dX[at] = torch.matmul(w.t().contiguous(), dy.t().contiguous()).t()
                dW[u] = torch.matmul(X[at].double().t().contiguous(), dy).t()
        return dict(Y=Y, dX=dX, dW=dW) if kind == "units_grad" else Y
    if kind == "scores":
        return _exact_products(*_exact_codes(s["X"].double()), s)
    h = s["X"].double()
    if case["residual"]:
        h = (h + s["R"].double()).to(DTYPES[case["dtype"]]).double()  # h is held in the rows' type
    w = s["weight"].double()
    rms = torch.sqrt(h.square().sum(1, keepdim=True) / case["d"] + EPS)
    if kind == "norm_scores":
        # the codes' values are h times weight held in 32 bits
        c, step = _exact_codes((h * w).float().double())
        return dict(H=h, y=_exact_products(c, step / rms, s))
    out = dict(Y=h / rms * w)
    if case["residual"]:
        out["H"] = h
    if kind == "norm_grad":
        dY = s["dY"].double()
        # y_j = w_j h_j / rms:  dL/dh_k = w_k dY_k / rms - h_k / (d rms^3) sum_j w_j dY_j h_j
        inner = (dY * w * h).sum(1, keepdim=True)
        dX = dY * w / rms - h * inner / (case["d"] * rms ** 3)
        if case["residual"]:
            dX = dX + s["dH"].double()
        out.update(dX=dX, dweight=(dY * h / rms).sum(0))
    return out
