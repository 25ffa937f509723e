"""The gated feed-forward operators as cases that can be timed and compared: the plain form of each (elementary torch
operations in 32 bits, rounded once at the end), the framework's own call, and the operator's definition in 64 bits.

  fp8_gated      h = act(x Wg^T) * (x Wu^T) from block-scaled FP8 codes, with the pre-activations saved for training
  gated_bwd      the gradient of the activation and the product, quantized in both tilings that Dgrad and Wgrad take
  int8_quant     8-bit codes with one scale for each token (activations) or channel (weights)
  int8_gemm      the product of such codes, both scales and an optional bias applied
  int8_gated     h = act(g) * u with both projections in 8-bit integers

Sizes are those of one FP8 Linear layer (8192 tokens, 7168 and 18432 channels), of one expert (2048 channels), and odd
ones between a single token and those.
"""

import math

import torch

own = False

FP8_MAX = 448.0
FP8_FLOOR = 448.0 * 2.0 ** -126     # a group's smallest max-abs: its scale stays a normal number
INT8_MAX = 127.0
INT8_FLOOR = 127.0 * 2.0 ** -126
GELU_C = 2.0 * math.sqrt(2.0 / math.pi)
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through an expert of 2048 channels: latency
        {"name": "fp8 gated, one token, expert", "op": "fp8_gated", "m": 1, "k": 7168, "f": 2048, "act": "silu",
         "save": False, "out": "bf16"},
        # a ragged prefill batch of one expert
        {"name": "fp8 gated, ragged prefill", "op": "fp8_gated", "m": 1511, "k": 7168, "f": 2048, "act": "gelu_tanh",
         "save": False, "out": "bf16"},
        # a training step's forward pass, pre-activations kept
        {"name": "fp8 gated, training forward", "op": "fp8_gated", "m": 8192, "k": 7168, "f": 18432, "act": "silu",
         "save": True, "out": "bf16"},
        # a ragged micro-batch's backward pass, odd row count
        {"name": "gated backward, ragged expert", "op": "gated_bwd", "m": 777, "f": 2048, "act": "gelu_tanh",
         "dtype": "bf16"},
        # the training step's backward pass
        {"name": "gated backward, training", "op": "gated_bwd", "m": 8192, "f": 18432, "act": "silu",
         "dtype": "bf16"},
        # a decode batch's activations
        {"name": "int8 quant, decode batch", "op": "int8_quant", "rows": 16, "cols": 7168, "dtype": "bf16"},
        # weights in 32 bits, quantized once per channel when a model is loaded
        {"name": "int8 quant, weight in f32", "op": "int8_quant", "rows": 18432, "cols": 7168, "dtype": "f32"},
        # one token through the down projection
        {"name": "int8 gemm, one token", "op": "int8_gemm", "m": 1, "n": 7168, "k": 18432, "bias": False,
         "out": "bf16"},
        # sizes that are no multiple of a tile, a channel group or a 16-byte chunk, with a bias
        {"name": "int8 gemm, odd sizes", "op": "int8_gemm", "m": 333, "n": 1999, "k": 1537, "bias": True,
         "out": "f32"},
        # prefill of the down projection
        {"name": "int8 gemm, prefill", "op": "int8_gemm", "m": 8192, "n": 7168, "k": 18432, "bias": False,
         "out": "bf16"},
        # a decode batch through both projections
        {"name": "int8 gated, decode batch", "op": "int8_gated", "m": 16, "k": 7168, "f": 18432, "act": "silu",
         "out": "bf16"},
        # a ragged prefill through both projections, odd channel count
        {"name": "int8 gated, ragged prefill", "op": "int8_gated", "m": 3001, "k": 7168, "f": 2047, "act": "silu",
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp8_gated", "gated_bwd", "int8_quant", "int8_gemm", "int8_gated"])
    act = rng.choice(["silu", "gelu_tanh"])
    out = rng.choice(["bf16", "bf16", "f32"])
    if op == "fp8_gated":
        return {"op": op, "m": _log(rng, 1, 8192), "k": 128 * _log(rng, 1, 56), "f": 128 * _log(rng, 1, 144),
                "act": act, "save": rng.random() < 0.5, "out": "bf16"}
    if op == "gated_bwd":
        return {"op": op, "m": _log(rng, 1, 8192), "f": 128 * _log(rng, 1, 144), "act": act,
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "int8_quant":
        return {"op": op, "rows": _log(rng, 1, 18432), "cols": _log(rng, 16, 18432),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "int8_gemm":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 16, 18432), "k": _log(rng, 16, 7168),
                "bias": rng.random() < 0.5, "out": out}
    return {"op": op, "m": _log(rng, 1, 8192), "k": _log(rng, 16, 7168), "f": _log(rng, 16, 9216), "act": act,
            "out": out}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, sigma, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    if sigma != 1.0:
        x *= sigma
    if outliers:                                  # activations have few large entries
        hit = torch.rand(shape, generator=gen, device="cuda") < outliers
        x = torch.where(hit, x * 50.0, x)
    return x


def _rows16(rows, cols, dtype):
    """A row-major [rows][cols] tensor whose rows start at multiples of 16 bytes, as the framework asks for."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _fp8_tiles(x):
    """Codes [rows][cols] and scales [cols/128][rows] of 1x128 tiles."""
    rows, cols = x.shape
    g = x.view(rows, cols // 128, 128)
    amax = g.abs().amax(2).clamp_min(FP8_FLOOR)
    q = (g * (FP8_MAX / amax)[:, :, None]).clamp(-FP8_MAX, FP8_MAX).view(rows, cols).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), (amax / FP8_MAX).t().contiguous()


def _fp8_blocks(w):
    """Codes [rows][cols] and scales [rows/128][cols/128] of 128x128 blocks."""
    rows, cols = w.shape
    g = w.view(rows // 128, 128, cols // 128, 128)
    amax = g.abs().amax((1, 3)).clamp_min(FP8_FLOOR)
    q = (g * (FP8_MAX / amax)[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(rows, cols).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), amax / FP8_MAX


def _int8_rows(x):
    """Codes [rows][cols] (rows 16 bytes apart) and one scale for each row."""
    amax = x.abs().amax(1).clamp_min(INT8_FLOOR)
    q = _rows16(x.shape[0], x.shape[1], torch.int8)
    q.copy_((x * (INT8_MAX / amax)[:, None]).round().clamp(-INT8_MAX, INT8_MAX))
    return q, amax / INT8_MAX


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "fp8_gated":
        m, k, f = case["m"], case["k"], case["f"]
        s["a"], s["sa"] = _fp8_tiles(_normal(gen, (m, k), 1.0, 0.001).to(torch.bfloat16).float())
        s["b"], s["sb"] = _fp8_blocks(_normal(gen, (2 * f, k), 0.02))
    elif op == "gated_bwd":
        m, f, dt = case["m"], case["f"], OUT[case["dtype"]]
        s["dh"] = _normal(gen, (m, f), 1e-3).to(dt)
        s["gu"] = _normal(gen, (m, 2 * f), 1.7).to(dt)
    elif op == "int8_quant":
        x = _normal(gen, (case["rows"], case["cols"]), 1.0, 0.001)
        s["x"] = _rows16(case["rows"], case["cols"], OUT[case["dtype"]])
        s["x"].copy_(x)
    elif op == "int8_gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _int8_rows(_normal(gen, (m, k), 1.0, 0.001))
        s["b"], s["sb"] = _int8_rows(_normal(gen, (n, k), 0.02))
        s["bias"] = _normal(gen, (n,), 0.1) if case["bias"] else None
    else:
        m, k, f = case["m"], case["k"], case["f"]
        s["a"], s["sa"] = _int8_rows(_normal(gen, (m, k), 1.0, 0.001))
        s["b"], s["sb"] = _int8_rows(_normal(gen, (2 * f, k), 0.02))
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _sigma_arg(g, act):
    """Both activations are g * sigmoid(t): t(g) and its derivative."""
    if act == "silu":
        return g, 1.0
    return GELU_C * (g + 0.044715 * g * g * g), GELU_C * (1.0 + 3 * 0.044715 * g * g)


def _gate(g, u, act):
    t, _ = _sigma_arg(g, act)
    return g * (1.0 / (1.0 + torch.exp(-t))) * u


def _plain_fp8_gated(s):
    c = s["case"]
    a = s["a"].view(torch.float8_e4m3fn).float() * s["sa"].t().repeat_interleave(128, 1)
    b = s["b"].view(torch.float8_e4m3fn).float() * s["sb"].repeat_interleave(128, 0).repeat_interleave(128, 1)
    gu = a @ b.t()
    f = c["f"]
    h = _gate(gu[:, :f], gu[:, f:], c["act"]).to(OUT[c["out"]])
    return (h, gu.to(OUT[c["out"]])) if c["save"] else h


def _tiles_1x128(x):
    rows, cols = x.shape
    g = x.view(rows, cols // 128, 128)
    amax = g.abs().amax(2).clamp_min(FP8_FLOOR)
    q = (g * (FP8_MAX / amax)[:, :, None]).clamp(-FP8_MAX, FP8_MAX)
    return q.view(rows, cols).to(torch.float8_e4m3fn), (amax / FP8_MAX).t().contiguous()


def _tiles_128x1(x):
    rows, cols = x.shape
    g = x.view(rows // 128, 128, cols)
    amax = g.abs().amax(1).clamp_min(FP8_FLOOR)
    q = (g * (FP8_MAX / amax)[:, None, :]).clamp(-FP8_MAX, FP8_MAX)
    return q.view(rows, cols).to(torch.float8_e4m3fn).t().contiguous(), amax / FP8_MAX


def _plain_gated_bwd(s):
    c = s["case"]
    m, f = c["m"], c["f"]
    dh, gu = s["dh"].float(), s["gu"].float()
    g, u = gu[:, :f], gu[:, f:]
    t, dt = _sigma_arg(g, c["act"])
    e = torch.exp(-t.abs())
    r = 1.0 / (1.0 + e)
    sig, one = torch.where(t >= 0, r, e * r), torch.where(t >= 0, e * r, r)   # sigmoid(t) and 1 - sigmoid(t)
    d = torch.zeros((-(-m // 128) * 128, 2 * f), device="cuda")               # whole 128-row tiles: the rest is zero
    d[:m, :f] = dh * u * (sig + g * sig * one * dt)
    d[:m, f:] = dh * (g * sig)
    return _tiles_1x128(d) + _tiles_128x1(d)


def _plain_int8_quant(s):
    x = s["x"].float()
    amax = x.abs().amax(1).clamp_min(INT8_FLOOR)
    q = (x * (INT8_MAX / amax)[:, None]).clamp(-INT8_MAX, INT8_MAX).round().to(torch.int8)
    return q, amax / INT8_MAX


def _plain_int8_gemm(s):
    c = s["case"]
    y = (s["a"].float() @ s["b"].float().t()) * (s["sa"][:, None] * s["sb"][None, :])
    if s["bias"] is not None:
        y = y + s["bias"][None, :]
    return y.to(OUT[c["out"]])


def _plain_int8_gated(s):
    c, f = s["case"], s["case"]["f"]
    y = (s["a"].float() @ s["b"].float().t()) * (s["sa"][:, None] * s["sb"][None, :])
    return _gate(y[:, :f], y[:, f:], c["act"]).to(OUT[c["out"]])


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if not own:
        return {"fp8_gated": _plain_fp8_gated, "gated_bwd": _plain_gated_bwd, "int8_quant": _plain_int8_quant,
                "int8_gemm": _plain_int8_gemm, "int8_gated": _plain_int8_gated}[op](state)
    import precision_fp8_quant_amd as fp8q
    c = state["case"]
    if op == "int8_quant":
        return fp8q.int8_quant_rows(state["x"])
    if op == "int8_gemm":
        return fp8q.int8_gemm(state["a"], state["sa"], state["b"], state["sb"], bias=state["bias"],
                              out_dtype=OUT[c["out"]])
    act = fp8q.ACT_SILU if c["act"] == "silu" else fp8q.ACT_GELU_TANH
    if op == "int8_gated":
        return fp8q.int8_gemm_gated(state["a"], state["sa"], state["b"], state["sb"], act=act,
                                    out_dtype=OUT[c["out"]])
    if op == "fp8_gated":
        return fp8q.fp8_gemm_gated(state["a"], state["sa"], state["b"], state["sb"], act=act,
                                   out_dtype=OUT[c["out"]], save_gate_up=c["save"])
    q, sc, q_t, sc_t = fp8q.fp8_gated_backward(state["dh"], state["gu"], act=act, mode=fp8q.MAXABS)
    return q.view(torch.float8_e4m3fn), sc, q_t.view(torch.float8_e4m3fn), sc_t


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _act_slope64(g, act):
    if act == "silu":
        sg = torch.sigmoid(g)
        return sg * (1.0 + g * (1.0 - sg))
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    th = torch.tanh(z)
    return 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8_gated":
        m, k, f = case["m"], case["k"], case["f"]
        gu = torch.zeros((m, 2 * f), dtype=torch.float64, device="cuda")
        a8, b8 = s["a"].view(torch.float8_e4m3fn), s["b"].view(torch.float8_e4m3fn)
        for k0 in range(0, k, 1024):              # a slice of the groups at a time: the 64-bit operands stay small
            g0, g1 = k0 // 128, min(k, k0 + 1024) // 128
            a = a8[:, k0:k0 + 1024].double().view(m, g1 - g0, 128) * s["sa"][g0:g1].double().t()[:, :, None]
            b = (b8[:, k0:k0 + 1024].double().view(2 * f // 128, 128, g1 - g0, 128)
                 * s["sb"][:, g0:g1].double()[:, None, :, None])
            gu += a.reshape(m, -1) @ b.reshape(2 * f, -1).t()
        h = _act64(gu[:, :f], case["act"]) * gu[:, f:]
        return (h, gu) if case["save"] else h
    if op == "gated_bwd":
        m, f = case["m"], case["f"]
        dh, gu = s["dh"].double(), s["gu"].double()
        g, u = gu[:, :f], gu[:, f:]
        d = torch.zeros((-(-m // 128) * 128, 2 * f), dtype=torch.float64, device="cuda")
        d[:m, :f] = dh * u * _act_slope64(g, case["act"])
        d[:m, f:] = dh * _act64(g, case["act"])
        d = d.abs()
        rows = d.view(d.shape[0], 2 * f // 128, 128).amax(2).clamp_min(FP8_FLOOR) / FP8_MAX
        cols = d.view(d.shape[0] // 128, 128, 2 * f).amax(1).clamp_min(FP8_FLOOR) / FP8_MAX
        # a code is the step of the 32-bit value that it stands for: it has no 64-bit value of its own
        return None, rows.t().contiguous(), None, cols
    if op == "int8_quant":
        amax = s["x"].double().abs().amax(1).clamp_min(INT8_FLOOR)
        return None, amax / INT8_MAX              # whole codes are compared for equality
    y = torch.zeros((s["a"].shape[0], s["b"].shape[0]), dtype=torch.float64, device="cuda")
    for k0 in range(0, case["k"], 1024):
        y += s["a"][:, k0:k0 + 1024].double() @ s["b"][:, k0:k0 + 1024].double().t()
    y *= s["sa"].double()[:, None]
    y *= s["sb"].double()[None, :]
    if op == "int8_gemm":
        return y if s["bias"] is None else y + s["bias"].double()[None, :]
    f = case["f"]
    return _act64(y[:, :f], case["act"]) * y[:, f:]


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "fp8_gated":
        m, k, f = case["m"], case["k"], case["f"]
        es = 2 if case["out"] == "bf16" else 4
        codes = m * k + 2 * f * k
        scales = 4 * (m * k // 128 + (2 * f // 128) * (k // 128))
        return {"bytes": codes + scales + es * m * f * (3 if case["save"] else 1), "flops": 4 * m * f * k}
    if op == "gated_bwd":
        m, f = case["m"], case["f"]
        mp, es = -(-m // 128) * 128, 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 3 * es * m * f + 2 * (2 * f * mp) + 2 * 4 * (2 * f * mp // 128), "flops": 20 * m * f}
    if op == "int8_quant":
        n, es = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (es + 1) + 4 * case["rows"], "flops": 3 * n}
    es = 2 if case["out"] == "bf16" else 4
    if op == "int8_gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + 4 * (m + n) + (4 * n if case["bias"] else 0) + es * m * n,
                "flops": 2 * m * n * k}
    m, k, f = case["m"], case["k"], case["f"]
    return {"bytes": (m + 2 * f) * k + 4 * (m + 2 * f) + es * m * f, "flops": 4 * m * f * k}
