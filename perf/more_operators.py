"""What the gated products, the 4-bit weights and the loss are measured on.

  gated_fwd    z = x w^T, h = act(z_gate) z_up, w [2n, k] gate rows over up rows;
               with "experts" over ragged row runs, w [E, 2n, k]
  gated_bwd    dx and dw from dh, x, w and the saved z
  int4_round   weights -> 4-bit codes and group scales -> the values they stand for
  int4         y = act(x W^T + bias) + residual with W in 4 bits; "gated": as
               gated_fwd; with "experts" over row runs
  loss_fwd     loss and log-sum-exp of each row of softmax(x w^T) at its target
  loss_bwd     dx and dw from each row's dloss

With `own` false `run` computes them in plain torch, in 32 bits, rounded once
at the end; with `own` true it makes the calls a user of
moe_grouped_gemm_fp8_amd makes.
"""
import math

import numpy as np
import torch

own = False

#: FLOPs of the largest listed case; drawn ones stay below it.
_MOST_FLOPS = 2.0 * 8192 * 128000 * 7168
#: and elements of the largest quantized weight
_MOST_WEIGHTS = 32 * 4096 * 7168


def listed():
    return [
        # the shared expert's first product for one decode batch: latency
        dict(name="gated fwd 64x2048x7168", op="gated_fwd", rows=64, n=2048, k=7168, act="silu", save_z=False, experts=0, live=0),
        # the experts' first product in training: 8192 tokens, top-8, some rows
        # dropped, very unequal experts, z kept for the backward pass
        dict(name="gated fwd 50021 rows", op="gated_fwd", rows=50021, n=2048, k=7168, act="silu", save_z=True, experts=32, live=32),
        # the shared expert's backward pass
        dict(name="gated bwd 4096x2048x7168", op="gated_bwd", rows=4096, n=2048, k=7168, act="gelu", experts=0, live=0),
        # the experts', over ragged runs, two experts without a token
        dict(name="gated bwd 16383 rows", op="gated_bwd", rows=16383, n=2048, k=7168, act="silu", experts=32, live=30),
        # a projection quantized when a model is loaded
        dict(name="int4 round trip 2112x7168", op="int4_round", experts=1, n=2112, k=7168, group=128, scales="f32"),
        # every expert of one layer
        dict(name="int4 round trip 32x4096x7168", op="int4_round", experts=32, n=4096, k=7168, group=128, scales="bf16"),
        # one token through a projection: latency
        dict(name="int4 1x24576x1536", op="int4", rows=1, n=24576, k=1536, group=128, scales="bf16", act="none", gated=False,
             bias=False, residual=False, experts=0, live=0),
        # a small batch through a wide one, bias and residual in the epilogue, short groups
        dict(name="int4 13x7168x16384", op="int4", rows=13, n=7168, k=16384, group=32, scales="f32", act="none", gated=False,
             bias=True, residual=True, experts=0, live=0),
        # 64 tokens, top-8 of 32 experts, through the experts' first product
        dict(name="int4 gated 512 rows 32 experts", op="int4", rows=512, n=2048, k=7168, group=128, scales="bf16", act="silu",
             gated=True, bias=False, residual=False, experts=32, live=31),
        # scoring a short text over a vocabulary of odd size
        dict(name="loss fwd 61x32003x2048", op="loss_fwd", rows=61, vocab=32003, k=2048),
        # a training step's loss
        dict(name="loss fwd 8192x128000x7168", op="loss_fwd", rows=8192, vocab=128000, k=7168),
        # and the gradients of a smaller head
        dict(name="loss bwd 4095x100003x2048", op="loss_bwd", rows=4095, vocab=100003, k=2048),
    ]


def _log(rng, low, high, of=1):
    """A multiple of `of`, spread over the logarithm of [low, high]."""
    return max(of, round(math.exp(rng.uniform(math.log(low), math.log(high))) / of) * of)


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "int4_round", "int4", "int4", "int4", "loss_fwd",
                     "loss_bwd", "loss_bwd"])
    if op.startswith("gated"):
        experts = _log(rng, 2, 64) if rng.random() < 0.5 else 0
        live = rng.randint(max(1, experts * 3 // 4), experts) if experts else 0
        n, k = _log(rng, 256, 4096, 8), _log(rng, 256, 7168, 8)
        c = dict(op=op, rows=max(live, _log(rng, 1, 32768)), n=n, k=k, act=rng.choice(["silu", "silu", "gelu", "relu"]),
                 experts=experts, live=live)
        if op == "gated_fwd":
            c["save_z"] = rng.random() < 0.5
        return c
    if op.startswith("int4"):
        group = rng.choice([32, 64, 128])
        n, k = _log(rng, 256, 16384, 8), _log(rng, 256, 16384, group)
        c = dict(op=op, n=n, k=k, group=group, scales=rng.choice(["f32", "bf16"]))
        if op == "int4_round":
            return dict(c, experts=_log(rng, 1, min(32, max(1, _MOST_WEIGHTS // (n * k)))))
        experts = _log(rng, 2, min(32, max(2, _MOST_WEIGHTS // (2 * n * k)))) if rng.random() < 0.4 else 0
        live = rng.randint(max(1, experts * 3 // 4), experts) if experts else 0
        gated = rng.random() < 0.4
        plain = not gated and not experts
        return dict(c, rows=max(live, _log(rng, 1, 512 if experts else 64)), experts=experts, live=live, gated=gated,
                    act=rng.choice(["silu", "gelu"]) if gated else "none",
                    bias=plain and rng.random() < 0.5, residual=plain and rng.random() < 0.5)
    vocab, k = _log(rng, 1000, 131072), _log(rng, 512, 7168, 8)
    most = _MOST_FLOPS / ((2.0 if op == "loss_fwd" else 6.0) * vocab * k)
    return dict(op=op, rows=_log(rng, 1, min(8192, most)), vocab=vocab, k=k)


def work(case):
    c, op = case, case["op"]
    if op.startswith("loss"):
        m, v, k = c["rows"], c["vocab"], c["k"]
        if op == "loss_fwd":
            return {"bytes": 2 * (m * k + v * k) + 16 * m, "flops": 2 * m * v * k}
        return {"bytes": 4 * (m * k + v * k) + 16 * m, "flops": 6 * m * v * k}
    n, k, sets = c["n"], c["k"], max(c["live"], 1) if "live" in c else c["experts"]
    if op == "int4_round":
        scales = (4 if c["scales"] == "f32" else 2) * k // c["group"] * n
        return {"bytes": sets * (n * k * 5 + 2 * scales), "flops": sets * 3 * n * k}
    m = c["rows"]
    if op == "int4":
        wide = n * (1 + c["gated"])
        scales = (4 if c["scales"] == "f32" else 2) * k // c["group"] * wide
        return {"bytes": sets * (wide * k // 2 + scales) + 2 * (m * k + m * n * (1 + c["residual"])) + 4 * n * c["bias"],
                "flops": 2 * m * wide * k}
    weights = sets * 2 * n * k
    if op == "gated_fwd":
        return {"bytes": 2 * (weights + m * k + m * n * (3 if c["save_z"] else 1)), "flops": 4 * m * n * k}
    made = max(c["experts"], 1) * 2 * n * k
    return {"bytes": 2 * (weights + made + 2 * m * k + 3 * m * n), "flops": 8 * m * n * k}


# ------------------------------------------------------------------- inputs
def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0, scale, generator=g)


def _runs(case, seed, s):
    """Rows of each expert: Zipf popularity over `live` experts, each with one
    row at least, in a random order among experts without any."""
    r = np.random.default_rng(seed)
    e, live = case["experts"], case["live"]
    p = np.arange(1, live + 1) ** -0.7
    counts = np.zeros(e, dtype=np.int64)
    counts[:live] = 1 + r.multinomial(case["rows"] - live, p / p.sum())
    counts = r.permutation(counts)
    ends = np.cumsum(counts)
    s["bounds"] = [(int(b - a), int(b)) for a, b in zip(counts, ends)]
    s["offsets"] = torch.tensor([0] + [int(b) for b in ends], dtype=torch.int32, device="cuda")


def _quantized(w, group, scale_dtype):
    """(codes 0..15 as uint8 [..., n, k], scales [..., k / group, n])."""
    v = w.float().unflatten(-1, (-1, group))
    # (torch divides by a number as a product with its reciprocal; BF16 weights
    # often lie on a border between two codes, so the quotient counts)
    amax = v.abs().amax(-1).double()
    scales = torch.where(amax > 0, amax / 7, 1.0).float().to(scale_dtype)
    codes = torch.round(v / scales.float()[..., None]).clamp(-7, 7) + 8
    return codes.flatten(-2).to(torch.uint8), scales.transpose(-1, -2).contiguous()


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(c)}
    if c.get("live"):
        _runs(c, seed, s)
    lead = [c["experts"]] if c.get("experts") else []
    if op.startswith("gated"):
        m, n, k = c["rows"], c["n"], c["k"]
        s["x"] = _normal(g, m, k)
        s["w"] = _normal(g, *lead, 2 * n, k, scale=k ** -0.5)
        if op == "gated_bwd":
            s["dh"] = _normal(g, m, n, scale=n ** -0.5)
            s["z"] = torch.empty(m, 2 * n, dtype=torch.bfloat16, device="cuda")
            for e, (a, b) in enumerate(s.get("bounds", [(0, m)])):
                w = s["w"][e] if lead else s["w"]
                s["z"][a:b] = s["x"][a:b] @ w.T
        return s
    if op.startswith("int4"):
        n, k = c["n"] * (2 if c.get("gated") else 1), c["k"]
        scale_dtype = torch.float32 if c["scales"] == "f32" else torch.bfloat16
        w = _normal(g, *lead, n, k, scale=k ** -0.5)
        if op == "int4_round":
            s["w"], s["scale_dtype"] = w, scale_dtype
            return s
        codes, s["scales"] = _quantized(w, c["group"], scale_dtype)
        s["q"] = codes[..., 0::2] | codes[..., 1::2] << 4
        s["x"] = _normal(g, c["rows"], k)
        s["bias"] = _normal(g, n, scale=0.1, dtype=torch.float32) if c["bias"] else None
        s["residual"] = _normal(g, c["rows"], c["n"]) if c["residual"] else None
        return s
    m, v, k = c["rows"], c["vocab"], c["k"]
    s["x"] = _normal(g, m, k)
    s["w"] = _normal(g, v, k, scale=2 * k ** -0.5)
    # one row in 16 is padding and has no target
    s["targets"] = torch.randint(0, v, (m,), device="cuda", generator=g)
    s["targets"][torch.rand(m, device="cuda", generator=g) < 1 / 16] = -100
    if op == "loss_bwd":
        s["lse"] = torch.empty(m, device="cuda")
        for a in range(0, m, 512):
            s["lse"][a:a + 512] = torch.logsumexp(s["x"][a:a + 512].float() @ s["w"].float().T, 1)
        s["dloss"] = torch.full((m,), 1.0 / m, device="cuda") * (0.5 + torch.rand(m, device="cuda", generator=g))
    return s


# -------------------------------------------------------------------- calls
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_grouped_gemm_fp8_amd as fg8
    c, op = s["case"], s["case"]["op"]
    if op == "gated_fwd":
        if c["experts"]:
            return fg8.grouped_gemm_bf16_gated(s["x"], s["w"], s["offsets"], activation=c["act"], save_z=c["save_z"])
        return fg8.gemm_bf16_gated(s["x"], s["w"], activation=c["act"], save_z=c["save_z"])
    if op == "gated_bwd":
        if c["experts"]:
            return fg8.grouped_gemm_bf16_gated_backward(s["dh"], s["x"], s["w"], s["z"], s["offsets"], activation=c["act"],
                                                        dw_dtype=torch.bfloat16)
        return fg8.gemm_bf16_gated_backward(s["dh"], s["x"], s["w"], s["z"], activation=c["act"], dw_dtype=torch.bfloat16)
    if op == "int4_round":
        q, scales = fg8.int4_quantize(s["w"], group=c["group"], scale_dtype=s["scale_dtype"])
        return fg8.int4_dequantize(q, scales), scales
    if op == "int4":
        if c["experts"]:
            return fg8.grouped_gemm_bf16_int4(s["x"], s["q"], s["scales"], s["offsets"], activation=c["act"], gated=c["gated"])
        return fg8.gemm_bf16_int4(s["x"], s["q"], s["scales"], s["bias"], s["residual"], activation=c["act"], gated=c["gated"])
    if op == "loss_fwd":
        return fg8.linear_cross_entropy(s["x"], s["w"], s["targets"])
    return fg8.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["targets"], s["lse"], dw_dtype=torch.bfloat16)


def _plain(s):
    return _PLAIN[s["case"]["op"]](s)


_ACT = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z / (1 + torch.exp(-z)),
        "gelu": lambda z: 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))}


def _slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


# The experts' runs differ in length and each has a weight of its own, so the
# plain form is one product an expert: a batched one would pad every run to
# the longest, several times the work.
def _z(s, weight):
    wide = s["w"].shape[-2] if "w" in s else s["q"].shape[-2]
    z = torch.zeros(s["x"].shape[0], wide, dtype=torch.float32, device="cuda")
    if "bounds" not in s:
        return torch.mm(s["x"].float(), weight(...).T, out=z)
    for e, (a, b) in enumerate(s["bounds"]):
        if b > a:
            torch.mm(s["x"][a:b].float(), weight(e).T, out=z[a:b])
    return z


def _gate(act, z):
    n = z.shape[1] // 2
    return (_ACT[act](z[:, :n]) * z[:, n:]).to(torch.bfloat16)


def _plain_gated_fwd(s):
    z = _z(s, lambda e: s["w"][e].float())
    h = _gate(s["case"]["act"], z)
    return (h, z.to(torch.bfloat16)) if s["case"]["save_z"] else h


def _plain_gated_bwd(s):
    act, n = s["case"]["act"], s["case"]["n"]
    zg, zu, dh = s["z"][:, :n].float(), s["z"][:, n:].float(), s["dh"].float()
    dz = torch.cat([dh * zu * _slope(act, zg), dh * _ACT[act](zg)], 1)
    if "bounds" not in s:
        return (dz @ s["w"].float()).to(torch.bfloat16), (dz.T @ s["x"].float()).to(torch.bfloat16)
    dx, dw = torch.zeros_like(s["x"]), torch.zeros_like(s["w"])
    for e, (a, b) in enumerate(s["bounds"]):
        if b > a:
            dx[a:b] = dz[a:b] @ s["w"][e].float()
            dw[e] = dz[a:b].T @ s["x"][a:b].float()
    return dx, dw


def _plain_int4_round(s):
    codes, scales = _quantized(s["w"], s["case"]["group"], s["scale_dtype"])
    values = (codes.float() - 8).unflatten(-1, (-1, s["case"]["group"])) * scales.float().transpose(-1, -2)[..., None]
    return values.flatten(-2).to(torch.bfloat16), scales


def _values(q, scales, group):
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).float() - 8
    return (codes.unflatten(-1, (-1, group)) * scales.float().T[..., None]).flatten(-2)


def _plain_int4(s):
    c = s["case"]
    z = _z(s, lambda e: _values(s["q"][e], s["scales"][e], c["group"]))
    if c["gated"]:
        return _gate(c["act"], z)
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _ACT[c["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_loss_fwd(s):
    z = s["x"].float() @ s["w"].float().T
    most = z.amax(1)
    live, at = s["targets"] >= 0, s["targets"].clamp(min=0)
    picked = z.gather(1, at[:, None])[:, 0]
    lse = torch.exp(z - most[:, None]).sum(1).log() + most
    return torch.where(live, lse - picked, 0.0), lse


def _plain_loss_bwd(s):
    live, at = s["targets"] >= 0, s["targets"].clamp(min=0)
    dz = torch.exp(s["x"].float() @ s["w"].float().T - s["lse"][:, None])
    dz.scatter_add_(1, at[:, None], torch.full_like(s["lse"][:, None], -1.0))
    dz *= torch.where(live, s["dloss"], 0.0)[:, None]
    return (dz @ s["w"].float()).to(torch.bfloat16), (dz.T @ s["x"].float()).to(torch.bfloat16)


_PLAIN = {"gated_fwd": _plain_gated_fwd, "gated_bwd": _plain_gated_bwd, "int4_round": _plain_int4_round, "int4": _plain_int4,
          "loss_fwd": _plain_loss_fwd, "loss_bwd": _plain_loss_bwd}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    c, op, s = case, case["op"], prepare(case, seed)
    if op == "int4_round":
        # the definition rounds the scale and the quotient to 32 bits
        w = s["w"].reshape(-1, c["k"] // c["group"], c["group"])
        values, scales = torch.empty(w.shape, dtype=torch.float64, device="cuda"), []
        for a in range(0, w.shape[0], 16384):
            v = w[a:a + 16384].double()
            top = v.abs().max(2).values
            t = torch.where(top == 0, 1.0, (top / 7.0).float().double()).to(s["scale_dtype"]).double()
            scales.append(t)
            values[a:a + 16384] = (v / t[:, :, None]).float().double().round().clamp(-7, 7) * t[:, :, None]
        scales = torch.cat(scales).reshape(*s["w"].shape[:-1], -1)
        return values.reshape(s["w"].shape), scales.transpose(-1, -2).contiguous()
    x = s["x"].double()
    if op.startswith("loss"):
        z = torch.mm(x, s["w"].double().t())
        t, rows = s["targets"], torch.arange(c["rows"], device="cuda")
        live = (t >= 0).double()
        if op == "loss_fwd":
            lse = torch.logsumexp(z, 1)
            return (lse - z[rows, t.clamp(min=0)]) * live, lse
        z = z.sub_(s["lse"].double()[:, None]).exp_()
        z[rows, t.clamp(min=0)] -= 1
        z *= (live * s["dloss"].double())[:, None]
        return torch.mm(z, s["w"].double()), torch.mm(z.t(), x)
    spans = s.get("bounds", [(0, c["rows"])])
    n, made = c["n"], []
    for e, (a, b) in enumerate(spans):
        if op == "int4":
            q, scales = (s["q"][e], s["scales"][e]) if c["experts"] else (s["q"], s["scales"])
            w = torch.empty(q.shape[0], c["k"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (q % 16).double() - 8, torch.div(q, 16, rounding_mode="floor").double() - 8
            w *= scales.double().t().repeat_interleave(c["group"], 1)
        else:
            w = (s["w"][e] if c["experts"] else s["w"]).double()
        if op == "gated_bwd":
            up, gate = s["z"][a:b, n:].double(), s["z"][a:b, :n].double()
            value, slope = _exact_act(c["act"], gate)
            dz = torch.cat([s["dh"][a:b].double() * up * slope, s["dh"][a:b].double() * value], 1)
            made.append((torch.mm(dz, w), torch.mm(dz.t(), x[a:b])))
            continue
        z = torch.mm(x[a:b], w.t())
        if op == "int4" and not c["gated"]:
            if c["bias"]:
                z += s["bias"].double()
            y = _exact_act(c["act"], z)[0]
            made.append((y + s["residual"][a:b].double() if c["residual"] else y, z))
        else:
            made.append((_exact_act(c["act"], z[:, :n])[0] * z[:, n:], z))
    first = torch.cat([p[0] for p in made])
    if op == "gated_bwd":
        return first, torch.stack([p[1] for p in made]) if c["experts"] else made[0][1]
    return (first, torch.cat([p[1] for p in made])) if c.get("save_z") else first


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
