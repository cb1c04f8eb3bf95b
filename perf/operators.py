"""Measured cases of the 8-bit linear layer and of the expert-grouped NF4 linear layer.

Each case is one call of one operator:

  quantize      rows of a 16- or 32-bit matrix to 8-bit integers, one float32
                scale a row (a weight by output channel, activations by token)
  int8_linear   Y = X W^T with W in 8 bits and a scale a channel, X in 16 bits
                and quantised by token within the call
  int8_matmul   the same product with the tokens' codes and scales given
  grouped_fwd   Y = X_e dequant(W_e)^T + s (X_e A_e^T) B_e^T over the rows X_e
                of each expert e (rows sorted by expert), frozen NF4 experts
                with a LoRA adapter each
  grouped_bwd   dX, dA and dB of grouped_fwd (no gradient for the frozen W)

run() computes them in plain torch in 32 bits, or, with `own`, by the calls a
user makes of the package.  The sizes are those of the linears of a 7B block
(4096, 11008) and of a 65B block (8192, 22016), a 1024 x 1024 linear, and
generic mixtures of a few wide or many narrow experts.
"""
import math
from statistics import NormalDist

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 64       # weights per NF4 block constant
GROUP = 256      # block constants per second-level scale


def nf4_levels():
    """The 16 NF4 levels in 64 bits: normal quantiles at 8 even probabilities
    above one half and 7 below, an exact 0, divided by the largest."""
    top, inv = 0.9677083, NormalDist().inv_cdf
    up = [inv(top + (0.5 - top) * i / 8) for i in range(8)]
    down = [-inv(top + (0.5 - top) * i / 7) for i in range(7)]
    return sorted(v / up[0] for v in up + down + [0.0])


LEVELS = np.array(nf4_levels(), dtype=np.float32)
MIDS = (LEVELS.astype(np.float64)[1:] + LEVELS.astype(np.float64)[:-1]) / 2
# the largest float32 not above each exact midpoint: r lies above the midpoint
# where r > threshold, so ties stay with the lower level
THRESHOLDS = MIDS.astype(np.float32)
THRESHOLDS = np.where(THRESHOLDS.astype(np.float64) > MIDS,
                      np.nextafter(THRESHOLDS, np.float32(-2)), THRESHOLDS)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the activations of a 7B block's prompt, and a block's weight at load time
        {"name": "quantize_tokens", "op": "quantize", "rows": 4001, "cols": 4096, "dtype": "bf16"},
        {"name": "quantize_weight", "op": "quantize", "rows": 11008, "cols": 4096,
         "dtype": "fp32"},
        # one generated token of one user; a batch of users on a 65B linear; a
        # short prompt; a long one
        {"name": "int8_one_token", "op": "int8_linear", "tokens": 1, "rows": 4096, "cols": 4096,
         "dtype": "bf16"},
        {"name": "int8_16_tokens", "op": "int8_linear", "tokens": 16, "rows": 22016,
         "cols": 8192, "dtype": "bf16"},
        {"name": "int8_211_tokens", "op": "int8_linear", "tokens": 211, "rows": 4096,
         "cols": 11008, "dtype": "fp16"},
        {"name": "int8_8192_tokens", "op": "int8_linear", "tokens": 8192, "rows": 11008,
         "cols": 4096, "dtype": "bf16"},
        # codes shared by several linears (the gate and up projections)
        {"name": "int8_codes_1000", "op": "int8_matmul", "tokens": 1000, "rows": 11008,
         "cols": 4096, "dtype": "bf16"},
        # generation: one token routed to two wide experts, a batch to many
        # narrow ones; training steps: few wide experts, many narrow ones
        {"name": "experts_one_token", "op": "grouped_fwd", "tokens": 2, "experts": 8,
         "rows": 11008, "cols": 4096, "rank": 16, "dtype": "bf16", "skew": 0.0},
        {"name": "experts_batch", "op": "grouped_fwd", "tokens": 250, "experts": 64,
         "rows": 1024, "cols": 2048, "rank": 16, "dtype": "fp16", "skew": 0.5},
        {"name": "experts_train", "op": "grouped_fwd", "tokens": 8192, "experts": 8,
         "rows": 11008, "cols": 4096, "rank": 64, "dtype": "bf16", "skew": 0.5},
        {"name": "experts_narrow_bwd", "op": "grouped_bwd", "tokens": 8191, "experts": 64,
         "rows": 1024, "cols": 2048, "rank": 16, "dtype": "fp16", "skew": 0.5},
        {"name": "experts_train_bwd", "op": "grouped_bwd", "tokens": 8192, "experts": 8,
         "rows": 11008, "cols": 4096, "rank": 64, "dtype": "bf16", "skew": 0.5},
    ]


MOST_FLOPS = 2.0 * 8192 * 11008 * 4096


def spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "int8_linear", "int8_linear", "int8_matmul", "grouped_fwd",
                     "grouped_fwd", "grouped_bwd"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "quantize":
        cols = 16 * spread(rng, 16, 1376)
        rows = min(spread(rng, 1, 16384), 11008 * 4096 // cols)
        return {"op": op, "rows": rows, "cols": cols,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op in ("int8_linear", "int8_matmul"):
        rows, cols = spread(rng, 256, 22016), 16 * spread(rng, 16, 1376)
        if rng.random() < 0.7:
            rows = -(-rows // 16) * 16
        tokens = min(spread(rng, 1, 8192), int(MOST_FLOPS / (2.0 * rows * cols)))
        return {"op": op, "tokens": max(1, tokens), "rows": rows, "cols": cols, "dtype": dtype}
    experts = rng.choice([2, 4, 8, 16, 32, 64, 5, 60])
    area = 8 * 11008 * 4096 // experts
    cols = 64 * spread(rng, 8, 172)
    rows = min(16 * spread(rng, 32, 688), area // cols // 16 * 16)
    low = 1 if op == "grouped_fwd" else 16
    tokens = min(spread(rng, low, 8192), int(MOST_FLOPS / (2.0 * rows * cols)))
    return {"op": op, "tokens": max(1, tokens), "experts": experts, "rows": rows, "cols": cols,
            "rank": rng.choice([16, 32, 64]), "dtype": dtype, "skew": rng.choice([0.0, 0.5, 1.0])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def activations(shape, dtype, gen):
    """Unit normal with a few wide channels, as activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    wide = torch.rand(shape[-1], generator=gen, device="cuda") < 0.004
    return torch.where(wide, 8 * x, x).to(dtype)


def pack_nf4(experts, rows, cols, gen):
    """A stacked normal weight [experts * rows, cols] in the packed format:
    4-bit codes, 8-bit codes of the block constants, group scales, offset."""
    levels = torch.from_numpy(THRESHOLDS.copy()).cuda()
    codes = torch.empty(experts, rows * cols // 2, dtype=torch.uint8, device="cuda")
    const = torch.empty(experts, rows * cols // BLOCK, device="cuda")
    for e in range(experts):
        w = torch.randn(rows * cols // BLOCK, BLOCK, generator=gen, device="cuda") * 0.02
        const[e] = w.abs().amax(1)
        c = torch.bucketize(w / const[e][:, None], levels, out_int32=True).to(torch.uint8)
        c = c.view(-1, 2)
        codes[e] = c[:, 0] | (c[:, 1] << 4)
    const = const.view(-1)
    offset = const.double().mean().float().view(1)
    d = const - offset
    groups = -(-d.numel() // GROUP)
    padded = torch.zeros(groups * GROUP, device="cuda")
    padded[:d.numel()] = d
    scale = padded.view(groups, GROUP).abs().amax(1)
    code8 = (padded.view(groups, GROUP) / scale[:, None] * 256).to(torch.float8_e4m3fn)
    code8 = code8.view(torch.uint8).view(-1)[:d.numel()].clone()
    return {"codes": codes.view(-1), "absmax_code": code8, "absmax_scale": scale,
            "absmax_offset": offset}


def route(case, gen):
    """Row offsets of each expert's rows, and which experts have any."""
    rng = np.random.default_rng(int(torch.randint(1 << 31, (1,), generator=gen,
                                                  device="cuda").item()))
    p = np.exp(case["skew"] * rng.standard_normal(case["experts"]))
    count = rng.multinomial(case["tokens"], p / p.sum())
    offsets = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    return torch.from_numpy(offsets).cuda(), count


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"op": case["op"], "dtype": dt}
    if case["op"] == "quantize":
        if case["dtype"] == "fp32":
            s["X"] = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda") * 0.02
        else:
            s["X"] = activations((case["rows"], case["cols"]), dt, gen)
        return s
    rows, cols, tokens = case["rows"], case["cols"], case["tokens"]
    if case["op"] in ("int8_linear", "int8_matmul"):
        w = torch.randn(rows, cols, generator=gen, device="cuda") * 0.02
        s["W"], s["w_scale"] = quantize_plain(w)
        x = activations((tokens, cols), dt, gen)
        if case["op"] == "int8_linear":
            s["X"] = x
        else:
            s["X"], s["x_scale"] = quantize_plain(x)
        if own:
            import bit_nf4_quantized_06_amd as q
            s["weight"] = q.Int8Weight(s["W"], s["w_scale"])
        return s
    e, r = case["experts"], case["rank"]
    s.update(pack_nf4(e, rows, cols, gen), experts=e, rows=rows, cols=cols)
    s["offsets"], count = route(case, gen)
    s["active"] = torch.from_numpy(np.flatnonzero(count)).cuda()
    s["longest"] = int(count.max())
    s["alpha"] = 16.0
    s["X"] = activations((tokens, cols), dt, gen)
    s["A"] = (torch.randn(e, r, cols, generator=gen, device="cuda") / math.sqrt(r)).to(dt)
    s["B"] = (torch.randn(e, rows, r, generator=gen, device="cuda") * 0.01).to(dt)
    if case["op"] == "grouped_bwd":
        s["dY"] = torch.randn(tokens, rows, generator=gen, device="cuda").to(dt)
        # what the forward kept: the rows times their expert's A, in 16 bits
        s["U"] = from_groups(s, torch.bmm(to_groups(s, s["X"]),
                                          s["A"][s["active"]].float().mT.contiguous())).to(dt)
    if own:
        import bit_nf4_quantized_06_amd as q
        s["weight"] = q.NF4Weight(e * rows, cols, s["codes"], s["absmax_code"],
                                  s["absmax_scale"], s["absmax_offset"],
                                  compute_dtype=case["dtype"])
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def quantize_plain(x):
    """Nearest whole number to x / scale, ties to even, scale = max |row| / 127
    in float32.  The quotients are taken in 64 bits: next to a border between
    two codes 32 would round to the other side."""
    scale = (x.abs().amax(1, keepdim=True).double() / 127).float()
    code = torch.round(x.double() / scale.double().clamp_min(1e-300)).clamp(-127, 127)
    return code.to(torch.int8), scale[:, 0]


def int8_product_plain(codes, x_scale, w, w_scale, dtype):
    y = codes.float() @ w.float().T
    return (y * (x_scale[:, None] * w_scale)).to(dtype)


def row_index(s):
    """[active experts, longest] row of each expert's j-th token, and whether
    it has one."""
    first = s["offsets"][s["active"]].long()[:, None]
    last = s["offsets"][s["active"] + 1].long()[:, None]
    at = first + torch.arange(s["longest"], device="cuda")
    return at.clamp_max(max(0, s["X"].shape[0] - 1)), at < last


def to_groups(s, x):
    """Rows [T, n] as [active experts, longest, n] in 32 bits, zero-padded."""
    at, has = row_index(s)
    return torch.where(has[..., None], x[at].float(), 0.0)


def from_groups(s, y):
    at, has = row_index(s)
    return y[has]


def weight_plain(s):
    """The active experts' weights as their 16-bit values, in 32 bits."""
    e, k, on = s["experts"], s["rows"] * s["cols"], s["active"]
    code8 = s["absmax_code"].view(e, -1)[on]
    block = torch.arange(e * k // BLOCK, device="cuda").view(e, -1)[on]
    const = code8.view(torch.float8_e4m3fn).float() * 2.0 ** -8 * s["absmax_scale"][block // GROUP]
    const = const + s["absmax_offset"]
    byte = s["codes"].view(e, -1)[on]
    code = torch.stack((byte & 15, byte >> 4), -1).view(len(on), -1, BLOCK)
    levels = torch.from_numpy(LEVELS.copy()).cuda()
    w = (levels[code.int()] * const[..., None]).to(s["dtype"])
    return w.view(len(on), s["rows"], s["cols"]).float()


def run_plain(s):
    if s["op"] == "quantize":
        return quantize_plain(s["X"])
    if s["op"] == "int8_linear":
        codes, x_scale = quantize_plain(s["X"])
        return int8_product_plain(codes, x_scale, s["W"], s["w_scale"], s["dtype"])
    if s["op"] == "int8_matmul":
        return int8_product_plain(s["X"], s["x_scale"], s["W"], s["w_scale"], s["dtype"])
    scale = s["alpha"] / s["A"].shape[1]
    w, x = weight_plain(s), to_groups(s, s["X"])
    a, b = s["A"][s["active"]].float(), s["B"][s["active"]].float()
    if s["op"] == "grouped_fwd":
        u = torch.bmm(x, a.mT.contiguous())
        y = torch.bmm(x, w.mT.contiguous()) + scale * torch.bmm(u, b.mT.contiguous())
        return from_groups(s, y).to(s["dtype"]), from_groups(s, u).to(s["dtype"])
    dy, u = to_groups(s, s["dY"]), to_groups(s, s["U"])
    g = torch.bmm(dy, b)
    dx = torch.bmm(dy, w) + scale * torch.bmm(g, a)
    da = torch.zeros(s["A"].shape, device="cuda")
    db = torch.zeros(s["B"].shape, device="cuda")
    da[s["active"]] = scale * torch.bmm(g.mT.contiguous(), x)
    db[s["active"]] = scale * torch.bmm(dy.mT.contiguous(), u)
    return from_groups(s, dx).to(s["dtype"]), da, db


def run_own(s):
    import bit_nf4_quantized_06_amd as q
    if s["op"] == "quantize":
        return q.qlora_int8_quantize(s["X"])
    if s["op"] == "int8_linear":
        return q.qlora_int8_linear_fwd(s["weight"], s["X"])
    if s["op"] == "int8_matmul":
        return q.qlora_int8_matmul(s["weight"], s["X"], s["x_scale"], dtype=s["dtype"])
    if s["op"] == "grouped_fwd":
        return q.qlora_grouped_linear_fwd(s["weight"], s["X"], s["offsets"], s["A"], s["B"],
                                          s["alpha"])
    return q.qlora_grouped_linear_bwd(s["weight"], s["X"], s["dY"], s["offsets"], s["A"], s["B"],
                                      s["alpha"], s["U"])


def run(state):
    return run_own(state) if own else run_plain(state)


# --------------------------------------------------------------------------
# the work that a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size + 1) + 4 * case["rows"], "flops": 3 * n}
    t, n, k = case["tokens"], case["rows"], case["cols"]
    if case["op"] in ("int8_linear", "int8_matmul"):
        x = 2 * t * k if case["op"] == "int8_linear" else t * k + 4 * t
        return {"bytes": n * k + 4 * n + x + 2 * t * n, "flops": 2 * t * n * k}
    e, r = case["experts"], case["rank"]
    used = e * (1 - (1 - 1 / e) ** t)     # experts that t even choices touch
    frozen = used * (n * k * (0.5 + 1 / BLOCK + 4 / (BLOCK * GROUP)) + 2 * r * (n + k))
    if case["op"] == "grouped_fwd":
        return {"bytes": frozen + 2 * t * (k + n + r), "flops": 2 * t * (n * k + r * (n + k))}
    return {"bytes": frozen + 2 * t * (2 * k + n + r) + 4 * e * r * (n + k),
            "flops": 2 * t * (n * k + 2 * r * (n + k))}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact_codes(x):
    """Whole numbers nearest to x over the row's float32 scale, by the
    remainder of the division; ties to even."""
    x = x.double()
    scale = (x.abs().max(dim=1).values / 127).to(torch.float32).double()
    some = scale > 0
    q = x / torch.where(some, scale, torch.ones_like(scale))[:, None]
    low = torch.floor(q)
    rest = q - low
    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))
    code = torch.clamp(low + up, -127, 127)
    return torch.where(some[:, None], code, torch.zeros_like(code)), scale


def exact_weight(s, e):
    """Expert e's weight [rows, cols] in 64 bits: level times block constant,
    each rounded where the format says so."""
    n = s["rows"] * s["cols"]
    byte = s["codes"][e * n // 2:(e + 1) * n // 2].to(torch.int64)
    code = torch.empty(n, dtype=torch.int64, device="cuda")
    code[0::2], code[1::2] = byte % 16, byte // 16
    nb = n // BLOCK
    c8 = s["absmax_code"][e * nb:(e + 1) * nb].to(torch.int64)
    power, part = c8 // 8 % 16, (c8 % 8).double()
    value = torch.where(power == 0, part * 2.0 ** -9,
                        (8 + part) * torch.exp2(power.double() - 10))
    value = torch.where(c8 >= 128, -value, value) / 256
    group = torch.arange(e * nb, (e + 1) * nb, device="cuda") // GROUP
    const = (value * s["absmax_scale"].double()[group]).float().double()
    const = (const + s["absmax_offset"].double()).float().double()
    level = torch.tensor([float(np.float32(v)) for v in nf4_levels()], dtype=torch.float64,
                         device="cuda")
    w = (level[code] * const.repeat_interleave(BLOCK)).float().to(s["dtype"])
    return w.double().view(s["rows"], s["cols"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        codes, scale = exact_codes(s["X"])
        return None, scale
    if case["op"] in ("int8_linear", "int8_matmul"):
        if case["op"] == "int8_linear":
            codes, x_scale = exact_codes(s["X"])
        else:
            codes, x_scale = s["X"].double(), s["x_scale"].double()
        w = s["W"].double() * s["w_scale"].double()[:, None]
        return torch.matmul(codes * x_scale[:, None], w.t())
    scale = s["alpha"] / case["rank"]
    x = s["X"].double()
    at = s["offsets"].tolist()
    if case["op"] == "grouped_fwd":
        y = torch.zeros(case["tokens"], case["rows"], dtype=torch.float64, device="cuda")
        u = torch.zeros(case["tokens"], case["rank"], dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(zip(at, at[1:])):
            if j > i:
                u[i:j] = x[i:j] @ s["A"][e].double().t()
                y[i:j] = x[i:j] @ exact_weight(s, e).t() + scale * u[i:j] @ s["B"][e].double().t()
        return y, u
    dy, u = s["dY"].double(), s["U"].double()
    dx = torch.zeros_like(x)
    da = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for e, (i, j) in enumerate(zip(at, at[1:])):
        if j > i:
            g = scale * dy[i:j] @ s["B"][e].double()
            dx[i:j] = dy[i:j] @ exact_weight(s, e) + g @ s["A"][e].double()
            da[e] = g.t() @ x[i:j]
            db[e] = scale * dy[i:j].t() @ u[i:j]
    return dx, da, db
