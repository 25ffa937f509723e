"""The operators in front of the projections as cases that can be timed and compared: the plain form of each (elementary
torch operations in 32 bits, rounded once at the end), the framework's own call, and the operator's definition in 64
bits.

  fp8_norm    root-mean-square norm of x (+ residual), handed on in FP8 codes with a scale for each 1x128 tile, for
              training also transposed in 128x1 tiles
  int8_norm   the same in 8-bit integers with a scale for each token
  norm_bwd    gradient of the norm: of its input (with the residual stream's own gradient added) and of its weight
  route       the k experts of each token, their weights, the tokens of each expert, and the loss that balances them
  route_bwd   gradient of the weights and of the loss with respect to the logits
  dispatch    rows of codes in the order of their experts, each expert's rows padded to whole 128-row tiles

Widths are those of one FP8 Linear layer (7168 channels, 8192 tokens), of one expert (2048), of a layer of 64 experts
that 65536 rows go to, and odd ones between a single token and those.
"""

import math

import torch

own = False

FP8_MAX = 448.0
FP8_FLOOR = 448.0 * 2.0 ** -126     # a group's smallest max-abs: its scale stays a normal number
INT8_MAX = 127.0
INT8_FLOOR = 127.0 * 2.0 ** -126
EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token in front of a projection, residual stream added: latency
        {"name": "fp8 norm, one token", "op": "fp8_norm", "m": 1, "d": 7168, "dtype": "bf16", "w": "bf16",
         "residual": True, "transposed": False, "rstd": False, "y": False},
        # a ragged prefill with the residual stream in 32 bits; y itself for a router
        {"name": "fp8 norm, ragged prefill", "op": "fp8_norm", "m": 1511, "d": 2048, "dtype": "f32", "w": "f32",
         "residual": True, "transposed": False, "rstd": False, "y": True},
        # a training step's forward pass: both tilings, and what the backward pass needs
        {"name": "fp8 norm, training", "op": "fp8_norm", "m": 8192, "d": 7168, "dtype": "bf16", "w": "bf16",
         "residual": True, "transposed": True, "rstd": True, "y": False},
        # a decode batch in front of an 8-bit integer projection
        {"name": "int8 norm, decode batch", "op": "int8_norm", "m": 16, "d": 7168, "dtype": "bf16", "w": "bf16",
         "residual": True},
        # a ragged prefill of an odd width in 32 bits
        {"name": "int8 norm, ragged prefill", "op": "int8_norm", "m": 3001, "d": 2047, "dtype": "f32", "w": "f32",
         "residual": False},
        # a ragged micro-batch's backward pass, odd width
        {"name": "norm backward, ragged", "op": "norm_bwd", "m": 777, "d": 1999, "dtype": "f32", "w": "f32",
         "dh": False},
        # the training step's backward pass
        {"name": "norm backward, training", "op": "norm_bwd", "m": 8192, "d": 7168, "dtype": "bf16", "w": "bf16",
         "dh": True},
        # a decode batch's routing: latency
        {"name": "route, decode batch", "op": "route", "t": 16, "e": 64, "k": 8, "dtype": "f32", "renorm": True,
         "padded": False},
        # a large training batch whose sequences end in padding
        {"name": "route, training", "op": "route", "t": 65536, "e": 64, "k": 8, "dtype": "bf16", "renorm": False,
         "padded": True},
        # its backward pass with more experts
        {"name": "route backward, training", "op": "route_bwd", "t": 65536, "e": 256, "k": 8, "dtype": "f32",
         "renorm": True, "padded": True},
        # a decode batch's rows to their experts
        {"name": "dispatch, decode batch", "op": "dispatch", "t": 16, "k": 8, "e": 64, "d": 7168},
        # a micro-batch's rows to the 64 experts of a layer, some of them much in demand
        {"name": "dispatch, training", "op": "dispatch", "t": 8192, "k": 8, "e": 64, "d": 7168},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp8_norm", "int8_norm", "norm_bwd", "route", "route_bwd", "dispatch"])
    dtype, w = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"])
    if op == "fp8_norm":
        return {"op": op, "m": _log(rng, 1, 8192), "d": 128 * _log(rng, 1, 56), "dtype": dtype, "w": w,
                "residual": rng.random() < 0.7, "transposed": rng.random() < 0.4, "rstd": rng.random() < 0.5,
                "y": rng.random() < 0.3}
    if op == "int8_norm":
        return {"op": op, "m": _log(rng, 1, 8192), "d": _log(rng, 16, 7168), "dtype": dtype, "w": w,
                "residual": rng.random() < 0.7}
    if op == "norm_bwd":
        return {"op": op, "m": _log(rng, 1, 8192), "d": _log(rng, 16, 7168), "dtype": dtype, "w": w,
                "dh": rng.random() < 0.7}
    if op in ("route", "route_bwd"):
        e = _log(rng, 4, 256)
        return {"op": op, "t": _log(rng, 1, 65536), "e": e, "k": rng.randint(1, min(e, 12)), "dtype": dtype,
                "renorm": rng.random() < 0.5, "padded": rng.random() < 0.5}
    e = _log(rng, 2, 256)
    return {"op": op, "t": _log(rng, 1, 8192), "k": rng.randint(1, min(e, 8)), "e": e, "d": 128 * _log(rng, 1, 56)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, sigma=1.0, outliers=0.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    if sigma != 1.0:
        x *= sigma
    if outliers:                                  # activations have few large entries
        hit = torch.rand(shape, generator=gen, device="cuda") < outliers
        x = torch.where(hit, x * 50.0, x)
    return x


def _rows16(x, dtype):
    """x as a row-major tensor of `dtype` whose rows start at multiples of 16 bytes, as the framework asks for."""
    rows, cols = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    t = torch.zeros((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]
    t.copy_(x)
    return t


def _logits(gen, t, e):
    """Logits of a router whose experts differ in how much they are in demand."""
    return _normal(gen, (t, e), 1.5) + _normal(gen, (1, e), 0.7)


def _valid(gen, t, padded):
    """Which tokens count: sequences of 512 rows that end in padding."""
    if not padded:
        return None
    n = -(-t // 512)
    length = torch.randint(300, 513, (n, 1), generator=gen, device="cuda")
    return (torch.arange(512, device="cuda")[None, :] < length).view(-1)[:t].contiguous()


def _max_rows(slots, e):
    """Rows of whole 128-row tiles that `slots` rows of `e` experts take at most."""
    return (slots + 127 * min(slots, e)) // 128 * 128


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("fp8_norm", "int8_norm", "norm_bwd"):
        m, d, dt = case["m"], case["d"], DTYPE[case["dtype"]]
        s["x"] = _rows16(_normal(gen, (m, d), 1.0, 0.001), dt)
        s["w"] = (1.0 + _normal(gen, (d,), 0.2)).to(DTYPE[case["w"]])
        if op != "norm_bwd":
            s["r"] = _rows16(_normal(gen, (m, d), 2.0), dt) if case["residual"] else None
        else:
            s["dy"] = _rows16(_normal(gen, (m, d), 1e-3), dt)
            s["dh"] = _rows16(_normal(gen, (m, d), 1e-3), dt) if case["dh"] else None
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
    elif op in ("route", "route_bwd"):
        t, e, k = case["t"], case["e"], case["k"]
        s["z"] = _rows16(_logits(gen, t, e), DTYPE[case["dtype"]])
        s["valid"] = _valid(gen, t, case["padded"])
        if op == "route_bwd":
            _, s["experts"], _, _, s["slope"] = _plain_route(s)
            s["dw"] = _normal(gen, (t, k), 1e-3)
            s["dloss"] = torch.full((1,), 0.01, device="cuda")
    else:
        t, k, e, d = case["t"], case["k"], case["e"], case["d"]
        s["experts"] = _logits(gen, t, e).topk(k, 1).indices.to(torch.int32)
        x = _normal(gen, (t, d), 1.0, 0.001)
        s["q"], s["scales"] = _tiles_1x128(x)
        s["q"] = s["q"].view(torch.uint8)
        rows = _max_rows(t * k, e)                # a program's own buffers: rows past the last tile keep what they hold
        s["a"] = torch.zeros((rows, d), dtype=torch.uint8, device="cuda")
        s["sa"] = torch.zeros((d // 128, rows), device="cuda")
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
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


def _plain_norm(s):
    """h (x, or its sum with the residual rounded to the type that it is kept in), 1 / rms and the norm of h."""
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    x = h.float()
    rstd = torch.rsqrt((x * x).mean(1) + EPS)
    return h, rstd, x * rstd[:, None] * s["w"].float()


def _plain_fp8_norm(s):
    c = s["case"]
    h, rstd, y = _plain_norm(s)
    if c["transposed"] and c["m"] % 128:          # whole 128-row tiles: the rest is zero
        full = torch.zeros((-(-c["m"] // 128) * 128, c["d"]), device="cuda")
        full[:c["m"]] = y
    else:
        full = y
    out = _tiles_1x128(full)
    if c["transposed"]:
        out += _tiles_128x1(full)
    if c["residual"]:
        out += (h,)
    if c["rstd"]:
        out += (rstd,)
    if c["y"]:
        out += (y.to(h.dtype),)
    return out


def _plain_int8_norm(s):
    h, _, y = _plain_norm(s)
    amax = y.abs().amax(1).clamp_min(INT8_FLOOR)
    q = (y * (INT8_MAX / amax)[:, None]).clamp(-INT8_MAX, INT8_MAX).round().to(torch.bfloat16)
    return (q, amax / INT8_MAX) + ((h,) if s["case"]["residual"] else ())


def _plain_norm_bwd(s):
    h, dy = s["x"].float(), s["dy"].float()
    xhat = h * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(0)


def _counted(s):
    t = s["z"].shape[0]
    return torch.ones(t, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]


def _plain_route(s):
    c = s["case"]
    e, k = c["e"], c["k"]
    z, ok = s["z"].float(), _counted(s)
    x = torch.exp(z - z.amax(1, keepdim=True))
    p = torch.where(ok[:, None], x / x.sum(1, keepdim=True), 0.0)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]    # ties: the lowest expert first
    w = p.gather(1, order)
    if c["renorm"]:
        w = torch.where(ok[:, None], w / w.sum(1, keepdim=True), 0.0)
    experts = torch.where(ok[:, None], order, -1)
    counts = (experts.reshape(-1, 1) == torch.arange(e, device="cuda")).sum(0)
    tokens = ok.sum()
    slope = counts.float() * (e / (k * tokens.float().square()))             # of the loss, by each token's p
    loss = (p.sum(0) * slope).sum()
    return w, experts.to(torch.int32), counts.to(torch.int32), loss.view(1), slope


def _plain_route_bwd(s):
    c = s["case"]
    z, ex = s["z"].float(), s["experts"].long()
    ok = ex[:, :1] >= 0
    x = torch.exp(z - z.amax(1, keepdim=True))
    p = x / x.sum(1, keepdim=True)
    chosen = ex.clamp_min(0)
    dw = s["dw"]
    if c["renorm"]:
        w = p.gather(1, chosen)
        total = w.sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True) / total) / total
    dp = (s["dloss"] * s["slope"])[None, :].expand_as(p).contiguous().scatter_add(1, chosen, dw)
    dz = p * (dp - (p * dp).sum(1, keepdim=True))
    return torch.where(ok, dz, 0.0).to(s["z"].dtype)


def _plain_dispatch(s):
    c = s["case"]
    t, k, e, d = c["t"], c["k"], c["e"], c["d"]
    rows = s["a"].shape[0]
    flat = s["experts"].reshape(-1).long()
    counts = (flat[:, None] == torch.arange(e, device="cuda")).sum(0)
    padded = (counts + 127) // 128 * 128
    start, first = padded.cumsum(0) - padded, counts.cumsum(0) - counts
    order = torch.sort(flat, stable=True).indices
    group = flat[order]
    place = start[group] + torch.arange(t * k, device="cuda") - first[group]
    row_of_slot = torch.empty(t * k, dtype=torch.int32, device="cuda")
    row_of_slot[order] = place.to(torch.int32)
    token_of_row = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    token_of_row[place] = (order // k).to(torch.int32)
    group_of_mtile = torch.full((rows // 128,), -1, dtype=torch.int32, device="cuda")
    tile = torch.arange(rows // 128, device="cuda") * 128
    used = tile < padded.sum()
    group_of_mtile[used] = torch.searchsorted(start + padded, tile[used], right=True).to(torch.int32)
    a = torch.zeros((rows, d), dtype=torch.uint8, device="cuda")
    a[place] = s["q"][order // k]
    sa = torch.where(used.repeat_interleave(128), 2.0 ** -126, 0.0).expand(d // 128, rows).contiguous()
    sa[:, place] = s["scales"][:, order // k]
    return a.view(torch.float8_e4m3fn), sa, group_of_mtile, row_of_slot.view(t, k), token_of_row


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if not own:
        return {"fp8_norm": _plain_fp8_norm, "int8_norm": _plain_int8_norm, "norm_bwd": _plain_norm_bwd,
                "route": _plain_route, "route_bwd": _plain_route_bwd, "dispatch": _plain_dispatch}[op](state)
    import precision_fp8_quant_amd as fp8q
    c = state["case"]
    if op == "fp8_norm":
        out = fp8q.fp8_rmsnorm(state["x"], state["w"], residual=state["r"], eps=EPS, transposed=c["transposed"],
                               save_rstd=c["rstd"], save_y=c["y"])
        out = (out[0].view(torch.float8_e4m3fn),) + out[1:]
        return out[:2] + (out[2].view(torch.float8_e4m3fn),) + out[3:] if c["transposed"] else out
    if op == "int8_norm":
        out = fp8q.int8_rmsnorm(state["x"], state["w"], residual=state["r"], eps=EPS)
        # the codes as the numbers that they are: BF16 holds every one of them
        return (out[0].to(torch.bfloat16),) + out[1:]
    if op == "norm_bwd":
        return fp8q.rmsnorm_backward(state["dy"], state["x"], state["w"], state["rstd"], dh=state["dh"])
    if op == "route":
        return fp8q.moe_route(state["z"], c["k"], valid=state["valid"], renormalize=c["renorm"])
    if op == "route_bwd":
        return fp8q.moe_route_backward(state["z"], state["experts"], state["slope"], dweights=state["dw"],
                                       dloss=state["dloss"], renormalize=c["renorm"])
    a, sa, group_of_mtile, row_of_slot, token_of_row = fp8q.fp8_moe_dispatch(
        state["experts"], state["q"], state["scales"], c["e"], a=state["a"], a_scales=state["sa"])
    return a.view(torch.float8_e4m3fn), sa, group_of_mtile, row_of_slot, token_of_row


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _norm64(s):
    x = s["x"].double()
    if s["r"] is not None:                        # the sum is kept, and normed, in the input's type
        x = (x + s["r"].double()).to(s["x"].dtype).double()
    rstd = (x.pow(2).sum(1) / x.shape[1] + EPS).pow(-0.5)
    return x, rstd, s["w"].double() * (rstd[:, None] * x)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fp8_norm", "int8_norm"):
        h, rstd, y = _norm64(s)
        if op == "int8_norm":
            scale = y.abs().amax(1).clamp_min(INT8_FLOOR) / INT8_MAX
            # a code is the step of the 32-bit value that it stands for: it has no 64-bit value of its own
            return (None, scale) + ((h,) if case["residual"] else ())
        m, d = y.shape
        mp = -(-m // 128) * 128 if case["transposed"] else m
        full = torch.zeros((mp, d), dtype=torch.float64, device="cuda")
        full[:m] = y
        # the numbers that the codes round
        tiles = full.view(mp, d // 128, 128)
        scale = tiles.abs().amax(2).clamp_min(FP8_FLOOR) / FP8_MAX
        out = ((tiles / scale[:, :, None]).view(mp, d), scale.t().contiguous())
        if case["transposed"]:
            cols = full.t().contiguous().view(d, mp // 128, 128)
            scale = cols.abs().amax(2).clamp_min(FP8_FLOOR) / FP8_MAX
            out += ((cols / scale[:, :, None]).view(d, mp), scale.t().contiguous())
        if case["residual"]:
            out += (h,)
        if case["rstd"]:
            out += (rstd,)
        if case["y"]:
            out += (y,)
        return out
    if op == "norm_bwd":
        h, dy, w, r = s["x"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = r * w * dy - h * (r.pow(3) * dot / h.shape[1])
        return (dx if s["dh"] is None else dx + s["dh"].double()), (dy * h * r).sum(0)
    if op == "dispatch":
        t, k, e, d = case["t"], case["k"], case["e"], case["d"]
        one_hot = torch.nn.functional.one_hot(s["experts"].reshape(-1).long(), e)
        counts = one_hot.sum(0)
        tiles = -(-counts // 128)
        rank = ((one_hot.cumsum(0) - one_hot) * one_hot).sum(1)            # earlier rows of the same expert
        place = (one_hot * (128 * (tiles.cumsum(0) - tiles))).sum(1) + rank
        a = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
        sa = torch.zeros(s["sa"].shape, dtype=torch.float64, device="cuda")
        sa[:, :128 * int(tiles.sum())] = 2.0 ** -126
        a.view(-1, d).index_copy_(0, place, s["q"].view(torch.float8_e4m3fn).double().repeat_interleave(k, 0))
        sa.index_copy_(1, place, s["scales"].double().repeat_interleave(k, 1))
        return a, sa, None, None, None
    k, e = case["k"], case["e"]
    z = s["z"].double()
    p = torch.softmax(z, 1)
    if op == "route":
        ok = _counted(s).double()[:, None]
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
        chosen = p.gather(1, order)
        w = chosen / chosen.sum(1, keepdim=True) if case["renorm"] else chosen
        share = torch.zeros(e, dtype=torch.float64, device="cuda")
        share.scatter_add_(0, order.reshape(-1), ok.expand(-1, k).reshape(-1))
        n = ok.sum()
        share /= k * n                            # f_e, of the choices
        mean = (p * ok).sum(0) / n                # P_e, of the probability
        return w * ok, None, None, (e * (share * mean).sum()).view(1), e * share / n
    ok = s["experts"][:, :1] >= 0
    z.requires_grad_(True)
    with torch.enable_grad():
        p = torch.softmax(z, 1)
        w = p.gather(1, s["experts"].long().clamp_min(0))
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        total = (w * s["dw"].double()).sum() + s["dloss"].double()[0] * (p * s["slope"].double()).sum()
        dz, = torch.autograd.grad(total, z)
    return torch.where(ok, dz, 0.0)


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("fp8_norm", "int8_norm", "norm_bwd"):
        m, d = case["m"], case["d"]
        n, es = m * d, size[case["dtype"]]
        weight = size[case["w"]] * d
        if op == "norm_bwd":
            return {"bytes": n * es * (4 if case["dh"] else 3) + weight + 4 * m + 4 * d, "flops": 9 * n}
        stream = n * es * (3 if case["residual"] else 1) + weight
        if op == "int8_norm":
            return {"bytes": stream + n + 4 * m, "flops": 7 * n}
        mp = -(-m // 128) * 128 if case["transposed"] else m
        tilings = 2 if case["transposed"] else 1
        return {"bytes": stream + tilings * (mp * d + 4 * mp * d // 128) + (4 * m if case["rstd"] else 0)
                + (n * es if case["y"] else 0), "flops": (5 + 2 * tilings) * n}
    if op in ("route", "route_bwd"):
        t, e, k, es = case["t"], case["e"], case["k"], size[case["dtype"]]
        mask = t if case["padded"] else 0
        if op == "route":
            return {"bytes": t * e * es + mask + 8 * t * k + 8 * e + 4, "flops": 6 * t * e}
        return {"bytes": 2 * t * e * es + 8 * t * k + 4 * e + 4, "flops": 10 * t * e}
    t, k, e, d = case["t"], case["k"], case["e"], case["d"]
    row = d + 4 * (d // 128)
    return {"bytes": (t + t * k) * row + 8 * t * k + 4 * t * k, "flops": 0}
