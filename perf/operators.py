"""What the BF16 operators beside the FP8 path are measured on.

Four operators, each with its backward pass: the expert products over ragged
row runs (`grouped_gemm_bf16*`), the dense product with bias, activation and
residual in its epilogue (`gemm_bf16_epilogue*`), layer norm (`layer_norm*`)
and the weighted return of the experts' rows to their tokens
(`moe_combine*`).  With `own` false `run` computes them in plain torch, in
32 bits, rounded once at the end; with `own` true it makes the calls a user of
moe_grouped_gemm_fp8_amd makes.

A case's "op" names the operator and direction:
  grouped_fwd    y[r] = x[r] W_e^T over expert e's run of rows
  grouped_dgrad  dx[r] = dy[r] W_e
  grouped_wgrad  dW_e = dy_e^T x_e                                  (FP32)
  dense_fwd      y = act(x W^T + bias) + residual, and z = x W^T + bias
  dense_bwd      dx, dW and dbias from dy, x, W and the saved z
  norm_fwd       y, mean, rstd
  norm_bwd       dx, dweight, dbias
  combine_fwd    out[t] = sum_j p[t, j] y[token_row[t, j]] (+ residual[t])
  combine_bwd    dy[r] = p[t, j] dout[t], dp[t, j] = dout[t] . y[r]
"""
import math

import numpy as np
import torch

own = False

#: FLOPs of the largest listed case; drawn products stay below it.
_MOST_FLOPS = 2.0 * 50021 * 4096 * 7168


def listed():
    return [
        # decode on one GPU's share of experts: a few rows for each, the
        # weights are the traffic and the call's latency counts
        dict(name="grouped fwd, 40 rows", op="grouped_fwd", rows=40, experts=8, live=7, n=1024, k=2048),
        # the first expert weight over a prefill batch: 8192 tokens, top-8,
        # a few of the rows dropped, experts of very unequal popularity
        dict(name="grouped fwd, 50021 rows", op="grouped_fwd", rows=50021, experts=32, live=32, n=4096, k=7168),
        # the second weight's input gradient in training
        dict(name="grouped dgrad, 16383 rows", op="grouped_dgrad", rows=16383, experts=32, live=30, n=7168, k=2048),
        # its weight gradient, summed over each expert's ragged run
        dict(name="grouped wgrad, 16383 rows", op="grouped_wgrad", rows=16383, experts=32, live=30, n=7168, k=2048),
        # a projection for one decode batch: 64 tokens, latency
        dict(name="dense fwd, 64x2112x7168", op="dense_fwd", m=64, n=2112, k=7168, act="silu", residual=False, save_z=False),
        # the dense half of a layer over a prefill batch, kept for training
        dict(name="dense fwd, 8191x7168x2048", op="dense_fwd", m=8191, n=7168, k=2048, act="gelu", residual=True, save_z=True),
        # its backward pass
        dict(name="dense bwd, 4096x7168x2048", op="dense_bwd", m=4096, n=7168, k=2048, act="gelu"),
        # the norm before one decode batch: latency
        dict(name="norm fwd, 64x7168", op="norm_fwd", rows=64, cols=7168, f32=False),
        # the norm over an FP32 residual stream, an odd number of rows
        dict(name="norm fwd, 16383x7168 fp32", op="norm_fwd", rows=16383, cols=7168, f32=True),
        # training: the input's gradient and both parameters' in one pass
        dict(name="norm bwd, 32768x7168", op="norm_bwd", rows=32768, cols=7168, f32=False),
        # the experts' rows of a prefill batch back to their tokens
        dict(name="combine fwd, 8192x7168", op="combine_fwd", tokens=8192, topk=8, experts=32, hidden=7168, residual=True),
        # and its gradients
        dict(name="combine bwd, 8192x7168", op="combine_bwd", tokens=8192, topk=8, experts=32, hidden=7168),
    ]


def _log(rng, low, high, of=1):
    """A multiple of `of`, spread over the logarithm of [low, high]."""
    return max(of, round(math.exp(rng.uniform(math.log(low), math.log(high))) / of) * of)


def draw(rng):
    op = rng.choice(["grouped_fwd", "grouped_fwd", "grouped_dgrad", "grouped_wgrad", "dense_fwd", "dense_fwd",
                     "dense_bwd", "norm_fwd", "norm_bwd", "combine_fwd", "combine_bwd"])
    if op.startswith("grouped"):
        experts = _log(rng, 2, 64)
        live = rng.randint(max(1, experts * 3 // 4), experts)
        n, k = _log(rng, 512, 7168, 8), _log(rng, 512, 7168, 8)
        most = _MOST_FLOPS / (2.0 * n * k)
        rows = max(live, _log(rng, 16, min(65536, most)))
        return dict(op=op, rows=rows, experts=experts, live=live, n=n, k=k)
    if op.startswith("dense"):
        n, k = _log(rng, 256, 16384, 8), _log(rng, 256, 8192, 8)
        m = _log(rng, 1 if op == "dense_fwd" else 256, 16384)
        c = dict(op=op, m=m, n=n, k=k, act=rng.choice(["none", "relu", "silu", "gelu"]))
        if op == "dense_fwd":
            c.update(residual=rng.random() < 0.5, save_z=rng.random() < 0.5)
        return c
    if op.startswith("norm"):
        cols = _log(rng, 256, 16384)
        return dict(op=op, rows=_log(rng, 1, min(65536, 2 ** 28 // cols)), cols=cols, f32=rng.random() < 0.5)
    topk = rng.randint(1, 8)
    hidden = _log(rng, 512, 7168, 8)
    tokens = _log(rng, 16, 8192)
    c = dict(op=op, tokens=tokens, topk=topk, experts=rng.choice([8, 16, 32, 64]), hidden=hidden)
    if op == "combine_fwd":
        c["residual"] = rng.random() < 0.5
    return c


def work(case):
    c, op = case, case["op"]
    if op.startswith("grouped"):
        r, n, k = c["rows"], c["n"], c["k"]
        weights = c["live"] * n * k
        per = {"grouped_fwd": 2 * (weights + r * k + r * n), "grouped_dgrad": 2 * (weights + r * n + r * k),
               "grouped_wgrad": 2 * (r * n + r * k) + 4 * c["experts"] * n * k}
        return {"bytes": per[op] + 4 * (c["experts"] + 1), "flops": 2 * r * n * k}
    if op.startswith("dense"):
        m, n, k = c["m"], c["n"], c["k"]
        if op == "dense_fwd":
            return {"bytes": 2 * (m * k + n * k) + 2 * m * n * (1 + c["residual"] + c["save_z"]) + 4 * n,
                    "flops": 2 * m * n * k}
        return {"bytes": 2 * (m * n * (1 if c["act"] == "none" else 2) + 2 * m * k + 2 * n * k) + 4 * n,
                "flops": 4 * m * n * k}
    if op.startswith("norm"):
        r, w, size = c["rows"], c["cols"], 4 if c["f32"] else 2
        if op == "norm_fwd":
            return {"bytes": 2 * size * r * w + 8 * w + 8 * r, "flops": 8 * r * w}
        return {"bytes": 3 * size * r * w + 12 * w + 8 * r, "flops": 13 * r * w}
    t, j, h = c["tokens"], c["topk"], c["hidden"]
    if op == "combine_fwd":
        return {"bytes": 2 * h * (t * j + t * (1 + c["residual"])) + 8 * t * j, "flops": 2 * t * j * h}
    padded = _capacity(t * j, c["experts"])
    return {"bytes": 2 * h * (t * j + t + t * j) + 12 * t * j + 4 * padded, "flops": 3 * t * j * h}


# ------------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def _counts(case, seed):
    """Rows of each expert: Zipf popularity over `live` experts, each with one
    row at least, in a random order among experts without any."""
    r = np.random.default_rng(seed)
    e, live, rows = case["experts"], case["live"], case["rows"]
    p = np.arange(1, live + 1) ** -0.7
    counts = np.zeros(e, dtype=np.int64)
    counts[:live] = 1 + r.multinomial(rows - live, p / p.sum())
    return r.permutation(counts)


def _capacity(rows, experts):
    return -(-(rows + 127 * experts) // 128) * 128


def _routing(case, g):
    """token_row and row_token of a layout of expert runs padded to 128 rows,
    experts in order, with one position in 64 that routes nowhere."""
    t, j, e = case["tokens"], case["topk"], case["experts"]
    keys = torch.rand(t, e, device="cuda", generator=g)
    ids = keys.topk(j, dim=1).indices.reshape(-1)
    ids[torch.rand(t * j, device="cuda", generator=g) < 1 / 64] = e
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=e + 1)
    starts = torch.cumsum((counts + 127) // 128 * 128, 0) - (counts + 127) // 128 * 128
    rank = torch.arange(t * j, device="cuda") - (torch.cumsum(counts, 0) - counts)[ids[order]]
    rows = starts[ids[order]] + rank
    token_row = torch.full((t * j,), -1, dtype=torch.int32, device="cuda")
    token_row[order] = torch.where(ids[order] < e, rows, -1).to(torch.int32)
    cap = _capacity(t * j, e)
    row_token = torch.full((cap + 1,), -1, dtype=torch.int32, device="cuda")
    at = torch.where(token_row >= 0, token_row, cap).long()
    row_token[at] = (torch.arange(t * j, device="cuda") // j).to(torch.int32)
    return token_row.reshape(t, j), row_token[:cap].contiguous(), cap


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(c)}
    if op.startswith("grouped"):
        counts = _counts(c, seed)
        ends = np.cumsum(counts)
        s["bounds"] = [(int(b - a), int(b)) for a, b in zip(counts, ends)]
        s["offsets"] = torch.tensor([0] + [int(b) for b in ends], dtype=torch.int32, device="cuda")
        e, n, k = c["experts"], c["n"], c["k"]
        if op != "grouped_wgrad":
            s["w"] = torch.empty(e, n, k, dtype=torch.bfloat16, device="cuda")
            s["w"].normal_(0, k ** -0.5, generator=g)
        if op != "grouped_dgrad":
            s["x"] = _normal(g, c["rows"], k)
        if op != "grouped_fwd":
            s["dy"] = _normal(g, c["rows"], n, scale=n ** -0.5)
    elif op.startswith("dense"):
        m, n, k = c["m"], c["n"], c["k"]
        s["x"] = _normal(g, m, k)
        s["w"] = _normal(g, n, k, scale=k ** -0.5)
        s["bias"] = _normal(g, n, scale=0.1, dtype=torch.float32)
        if op == "dense_fwd":
            s["residual"] = _normal(g, m, n) if c["residual"] else None
        else:
            s["dy"] = _normal(g, m, n, scale=n ** -0.5)
            s["z"] = (s["x"].float() @ s["w"].float().T + s["bias"]).to(torch.bfloat16)
    elif op.startswith("norm"):
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        scale = torch.exp(torch.randn(c["rows"], 1, device="cuda", generator=g))
        s["x"] = (_normal(g, c["rows"], c["cols"], dtype=torch.float32) * scale + 0.3 * scale).to(dtype)
        s["weight"] = 1 + _normal(g, c["cols"], scale=0.1, dtype=torch.float32)
        s["bias"] = _normal(g, c["cols"], scale=0.1, dtype=torch.float32)
        if op == "norm_bwd":
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + 1e-5)
            s["dy"] = _normal(g, c["rows"], c["cols"], dtype=dtype)
    else:
        s["token_row"], s["row_token"], cap = _routing(c, g)
        s["y"] = _normal(g, cap, c["hidden"])
        s["weights"] = torch.softmax(torch.randn(c["tokens"], c["topk"], device="cuda", generator=g), 1)
        if op == "combine_fwd":
            s["residual"] = _normal(g, c["tokens"], c["hidden"]) if c["residual"] else None
        else:
            s["dout"] = _normal(g, c["tokens"], c["hidden"])
    return s


# -------------------------------------------------------------------- calls
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_grouped_gemm_fp8_amd as fg8
    c, op = s["case"], s["case"]["op"]
    if op == "grouped_fwd":
        return fg8.grouped_gemm_bf16(s["x"], s["w"], s["offsets"])
    if op == "grouped_dgrad":
        return fg8.grouped_gemm_bf16_dgrad(s["dy"], s["w"], s["offsets"])
    if op == "grouped_wgrad":
        return fg8.grouped_gemm_bf16_wgrad(s["dy"], s["x"], s["offsets"])
    if op == "dense_fwd":
        return fg8.gemm_bf16_epilogue(s["x"], s["w"], s["bias"], s["residual"], activation=c["act"], save_z=c["save_z"])
    if op == "dense_bwd":
        return fg8.gemm_bf16_epilogue_backward(s["dy"], s["x"], s["w"], s["z"], activation=c["act"])
    if op == "norm_fwd":
        return fg8.layer_norm(s["x"], s["weight"], s["bias"], eps=1e-5)
    if op == "norm_bwd":
        return fg8.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    if op == "combine_fwd":
        return fg8.moe_combine(s["y"], s["token_row"], s["weights"], residual=s["residual"])
    return fg8.moe_combine_backward(s["dout"], s["y"], s["token_row"], s["row_token"], s["weights"])


def _plain(s):
    return _PLAIN[s["case"]["op"]](s)


# The experts' runs differ in length and each has a weight of its own, so the
# plain form is one product an expert: a batched one would pad every run to
# the longest, several times the work.
def _plain_grouped_fwd(s):
    out = torch.empty(s["x"].shape[0], s["w"].shape[1], dtype=torch.bfloat16, device="cuda")
    for e, (a, b) in enumerate(s["bounds"]):
        if b > a:
            out[a:b] = s["x"][a:b].float() @ s["w"][e].float().T
    return out


def _plain_grouped_dgrad(s):
    out = torch.empty(s["dy"].shape[0], s["w"].shape[2], dtype=torch.bfloat16, device="cuda")
    for e, (a, b) in enumerate(s["bounds"]):
        if b > a:
            out[a:b] = s["dy"][a:b].float() @ s["w"][e].float()
    return out


def _plain_grouped_wgrad(s):
    c = s["case"]
    out = torch.zeros(c["experts"], c["n"], c["k"], dtype=torch.float32, device="cuda")
    for e, (a, b) in enumerate(s["bounds"]):
        if b > a:
            torch.mm(s["dy"][a:b].float().T, s["x"][a:b].float(), out=out[e])
    return out


_ACT = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z / (1 + torch.exp(-z)),
        "gelu": lambda z: 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))}


def _act_slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_dense_fwd(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().T + s["bias"]
    y = _ACT[c["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if c["save_z"] else y


def _plain_dense_bwd(s):
    dz = s["dy"].float()
    if s["case"]["act"] != "none":
        dz = dz * _act_slope(s["case"]["act"], s["z"].float())
    return ((dz @ s["w"].float()).to(torch.bfloat16), (dz.T @ s["x"].float()).to(torch.bfloat16), dz.sum(0))


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-5)
    y = d * rstd * s["weight"] + s["bias"]
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * h).sum(0), dy.sum(0)


def _plain_combine_fwd(s):
    rows = s["token_row"].long()
    p = torch.where(rows >= 0, s["weights"], 0.0)
    out = (s["y"][rows.clamp(min=0)].float() * p[:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _plain_combine_bwd(s):
    rows = s["token_row"].long()
    live, dout = rows >= 0, s["dout"].float()
    dp = torch.where(live, (s["y"][rows.clamp(min=0)].float() * dout[:, None, :]).sum(2), 0.0)
    dy = torch.zeros_like(s["y"])
    t, j = live.nonzero(as_tuple=True)
    dy[rows[t, j]] = (dout[t] * s["weights"][t, j][:, None]).to(torch.bfloat16)
    return dy, dp


_PLAIN = {"grouped_fwd": _plain_grouped_fwd, "grouped_dgrad": _plain_grouped_dgrad, "grouped_wgrad": _plain_grouped_wgrad,
          "dense_fwd": _plain_dense_fwd, "dense_bwd": _plain_dense_bwd, "norm_fwd": _plain_norm_fwd,
          "norm_bwd": _plain_norm_bwd, "combine_fwd": _plain_combine_fwd, "combine_bwd": _plain_combine_bwd}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    c, op, s = case, case["op"], prepare(case, seed)
    v = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point() and n not in ("w", "y")}
    if op.startswith("grouped"):
        got = []
        for e, (a, b) in enumerate(s["bounds"]):
            if op == "grouped_fwd":
                got.append(torch.mm(v["x"][a:b], s["w"][e].double().t()))
            elif op == "grouped_dgrad":
                got.append(torch.mm(v["dy"][a:b], s["w"][e].double()))
            else:
                got.append(torch.mm(v["dy"][a:b].t(), v["x"][a:b]))
        return torch.stack(got) if op == "grouped_wgrad" else torch.cat(got)
    if op == "dense_fwd":
        z = torch.addmm(v["bias"], v["x"], s["w"].double().t())
        y = _exact_act(c["act"], z)[0]
        if c["residual"]:
            y += v["residual"]
        return (y, z) if c["save_z"] else y
    if op == "dense_bwd":
        dz = v["dy"] * _exact_act(c["act"], v["z"])[1]
        return torch.mm(dz, s["w"].double()), torch.mm(dz.t(), v["x"]), dz.sum(0)
    if op == "norm_fwd":
        var, mean = torch.var_mean(v["x"], dim=1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        return (v["x"] - mean[:, None]) * (rstd[:, None] * v["weight"]) + v["bias"], mean, rstd
    if op == "norm_bwd":
        h = (v["x"] - v["mean"][:, None]) * v["rstd"][:, None]
        g = v["dy"] * v["weight"]
        along = (g * h).sum(1, keepdim=True) / c["cols"]
        return ((g - g.sum(1, keepdim=True) / c["cols"] - h * along) * v["rstd"][:, None], (v["dy"] * h).sum(0), v["dy"].sum(0))
    at = s["token_row"].long()
    if op == "combine_fwd":
        out = v["residual"].clone() if c["residual"] else torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
        for j in range(c["topk"]):
            t = (at[:, j] >= 0).nonzero()[:, 0]
            out[t] += v["weights"][t, j][:, None] * s["y"][at[t, j]].double()
        return out
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dp = torch.zeros(c["tokens"], c["topk"], dtype=torch.float64, device="cuda")
    for j in range(c["topk"]):
        t = (at[:, j] >= 0).nonzero()[:, 0]
        dy[at[t, j]] = v["weights"][t, j][:, None] * v["dout"][t]
        dp[t, j] = (v["dout"][t] * s["y"][at[t, j]].double()).sum(1)
    return dy, dp


def _exact_act(act, z):
    """act(z) and its slope."""
    if act == "none":
        return z.clone(), torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    cdf = torch.special.ndtr(z)
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
