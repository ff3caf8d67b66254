"""Measured cases of the dense MXFP4 operators and of the router's training operators.

Each case is one pass through one operator:

  quant     MXFP4 quantisation of a matrix along rows and along columns, and the values the codes stand for;
  linear    y = Q(x) Wq^T: activations quantised on the way, weights held as MXFP4 codes;
  backward  the linear layer's gradients: dx = Q(dy) W, dw = Q(dy)^T x, all operands MXFP4 along the summed axis;
  balance   the router's balance loss, z loss and per-expert counts over ragged sequences;
  router    the gradient to the router's logits, of both losses and of the routing weights.

``run`` computes them in elementary torch operations, or, where ``own`` is set, through the library's entry points.
``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
GROUP = 32      # elements that share one scale
ALIGN = 128     # columns of codes are padded to this
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _up(n):
    return -(-n // ALIGN) * ALIGN


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # weights brought to MXFP4 for both passes of training: fp32 master weights of a shared expert's gate/up projection
        {"name": "quant_weight_2048x4096", "op": "quant", "rows": 2048, "cols": 4096, "dtype": "fp32"},
        # a ragged batch of activations, padded hidden size
        {"name": "quant_act_333x4000", "op": "quant", "rows": 333, "cols": 4000, "dtype": "bf16"},
        # a single token through a shared expert's gate/up projection (H = 4096, 2I = 2048)
        {"name": "linear_decode_1", "op": "linear", "m": 1, "n": 2048, "k": 4096},
        # a small odd decode batch through its down projection, with the padded sizes H = 4000, I = 1000
        {"name": "linear_decode_13", "op": "linear", "m": 13, "n": 4000, "k": 1000},
        # a decode batch through the gate/up projection
        {"name": "linear_decode_64", "op": "linear", "m": 64, "n": 2048, "k": 4096},
        # a long prompt through the gate/up projection
        {"name": "linear_prefill_4096", "op": "linear", "m": 4096, "n": 2048, "k": 4096},
        # the longest prefill through a wide projection
        {"name": "linear_prefill_16384", "op": "linear", "m": 16384, "n": 8192, "k": 4096},
        # a training step of the gate/up projection on a ragged batch
        {"name": "backward_4001", "op": "backward", "m": 4001, "n": 2048, "k": 4096},
        # router of 288 experts, top-8: one decode batch's statistics
        {"name": "balance_64", "op": "balance", "tokens": 64, "experts": 288, "top_k": 8, "seqs": 1},
        # a training batch of 16 ragged sequences, one of them empty
        {"name": "balance_16384", "op": "balance", "tokens": 16384, "experts": 288, "top_k": 8, "seqs": 16},
        {"name": "router_64", "op": "router", "tokens": 64, "experts": 288, "top_k": 8, "seqs": 1},
        {"name": "router_16384", "op": "router", "tokens": 16384, "experts": 288, "top_k": 8, "seqs": 16},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "backward", "balance", "router"])
    if op == "quant":
        rows = _log_uniform(rng, 1, 8192)
        return {"op": op, "rows": rows, "cols": _log_uniform(rng, 32, min(8192, 2048 * 4096 // rows)),
                "dtype": rng.choice(["bf16", "fp32"])}
    if op in ("linear", "backward"):
        m = _log_uniform(rng, 1 if op == "linear" else 33, 16384 if op == "linear" else 4096)
        return {"op": op, "m": m, "n": _log_uniform(rng, 16, 8192 if op == "linear" else 2048),
                "k": _log_uniform(rng, 33, 4096)}
    tokens = _log_uniform(rng, 1, 16384)
    experts = _log_uniform(rng, 8, 288)
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(8, experts)),
            "seqs": _log_uniform(rng, 1, 16)}


# ---- MXFP4 in elementary operations (fp32; every step of the format is exact there) -----

def _scale_bytes(groups):
    """E8M0 byte of each group of 32 along the last axis: 2^(floor(log2 amax) - 2), biased by 127."""
    amax = groups.abs().amax(-1)
    exponent = torch.frexp(amax)[1] - 1
    return torch.where(amax > 0, (exponent - 2 + 127).clamp(0, 254), torch.zeros_like(exponent))


def _grid(a):
    """|values| up to 6 rounded to the E2M1 grid, ties to the even code."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _pad(v):
    return torch.nn.functional.pad(v, (0, _up(v.shape[1]) - v.shape[1]))


def _quantised(v):
    """fp32 [R, C] -> (the E2M1 values [R, Cp/32, 32] with their signs, the scale bytes [R, Cp/32])."""
    groups = _pad(v).reshape(v.shape[0], -1, GROUP)
    b = _scale_bytes(groups)
    scaled = torch.ldexp(groups, (127 - b).unsqueeze(-1))
    return torch.copysign(_grid(scaled.abs().clamp(max=6.0)), scaled), b


def _values(v):
    """What fp32 [R, C] becomes through MXFP4, fp32 [R, C]."""
    q, b = _quantised(v)
    return torch.ldexp(q, (b - 127).unsqueeze(-1)).reshape(v.shape[0], -1)[:, :v.shape[1]]


def _packed(v):
    """fp32 [R, C] -> codes uint8 [R, Cp/2] (low nibble first), scales uint8 [R, Cp/32]."""
    q, b = _quantised(v)
    a = q.abs()
    code = sum((a >= x).to(torch.uint8) for x in E2M1[1:])
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).reshape(v.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), b.to(torch.uint8)


def _unpacked(codes, scales, cols, dtype=torch.float32):
    """The values [R, cols] of packed codes and scales."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).reshape(codes.shape[0], -1, GROUP)
    return torch.ldexp(v, (scales.to(torch.int32) - 127).unsqueeze(-1)).reshape(codes.shape[0], -1)[:, :cols]


# ---- inputs ---------------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """N(0, 1) with one value in a hundred 30 times as large."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    return torch.where(torch.rand(rows, cols, generator=g, device=DEVICE) < 0.01, x * 30, x).to(dtype)


def _router_inputs(case, g):
    tokens, experts, k, seqs = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    logits = torch.randn(tokens, experts, generator=g, device=DEVICE) * 1.5
    logits += torch.linspace(1.0, -1.0, experts, device=DEVICE)         # some experts are more popular
    # one expert in sixteen is switched off for some tokens, where enough others are left
    off = torch.rand(tokens, experts, generator=g, device=DEVICE) < 1 / 64
    if experts >= 2 * k + 8:
        off[:, :2 * k] = False
        logits = logits.masked_fill(off, float("-inf"))
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, 1)
    cuts = torch.sort(torch.randint(0, tokens + 1, (max(seqs - 1, 0),), generator=g, device=DEVICE)).values
    if seqs >= 4:
        cuts[1] = cuts[0]                                               # an empty sequence
    ends = torch.tensor([0, tokens - tokens // 100], device=DEVICE)     # some rows lie behind the last sequence
    offsets = torch.cat([ends[:1], torch.minimum(cuts, ends[1]), ends[1:]]).to(torch.int32)
    mask = (torch.rand(tokens, generator=g, device=DEVICE) > 0.05).to(torch.uint8)
    return {"logits": logits, "ids": ids.to(torch.int32), "weights": weights, "offsets": offsets, "mask": mask}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    state = {"case": case}
    op = case["op"]
    if op == "quant":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        state["x"] = _activations(g, case["rows"], case["cols"], dtype)
    elif op == "linear":
        state["x"] = _activations(g, case["m"], case["k"], torch.bfloat16)
        state["w"] = _packed(torch.randn(case["n"], case["k"], generator=g, device=DEVICE) * 0.02)
    elif op == "backward":
        state["dy"] = (torch.randn(case["m"], case["n"], generator=g, device=DEVICE) * 1e-3).to(torch.bfloat16)
        w = torch.randn(case["n"], case["k"], generator=g, device=DEVICE) * 0.02
        x = _activations(g, case["m"], case["k"], torch.float32)
        state["w_cols"] = _packed(w.t().contiguous())      # [k, n]: along n
        state["x_cols"] = _packed(x.t().contiguous())      # [k, m]: along m
    else:
        state.update(_router_inputs(case, g))
        if op == "router":
            state["d_weights"] = torch.randn(case["tokens"], case["top_k"], generator=g, device=DEVICE)
            state["d_loss"] = torch.tensor([1e-2, 1e-3], device=DEVICE) * case["tokens"]
            _, state["counts"], state["seq_tokens"], state["lse"] = _balance(state, torch.float32)
    return state


# ---- the plain forms of the router's operators ---------------------------------

def _members(state, dtype):
    """-> valid tokens (bool [T]) and their sequences as a 0/1 matrix [S, T]."""
    logits, offsets = state["logits"], state["offsets"].long()
    t = torch.arange(logits.shape[0], device=logits.device)
    valid = (state["mask"] != 0) & (logits != float("-inf")).any(1)
    member = (t >= offsets[:-1, None]) & (t < offsets[1:, None]) & valid
    return member.any(0), member.to(dtype)


def _balance(state, dtype):
    logits, ids = state["logits"].to(dtype), state["ids"].long()
    tokens, experts = logits.shape
    k = ids.shape[1]
    valid, member = _members(state, dtype)
    high = logits.amax(1, keepdim=True)
    high = torch.where(high == float("-inf"), torch.zeros_like(high), high)
    ex = torch.exp(logits - high)
    total = ex.sum(1, keepdim=True)
    lse = torch.where(valid, (torch.log(total) + high)[:, 0], torch.zeros_like(total[:, 0]))
    p = ex / total
    p = torch.where(valid[:, None], p, torch.zeros_like(p))
    chosen = torch.zeros_like(logits).scatter_add_(1, ids, torch.ones_like(ids, dtype=dtype))
    counts = member @ chosen
    n = member.sum(1)
    f = counts * (experts / k) / n.clamp(min=1)[:, None]
    mean_p = (member @ p) / n.clamp(min=1)[:, None]
    filled = (n > 0).sum()
    balance = (f * mean_p).sum() / filled.clamp(min=1)
    z = (lse * lse).sum() / n.sum().clamp(min=1)
    seq_tokens = torch.cat([n, n.sum()[None], filled[None].to(dtype)]).to(torch.int32)
    return torch.stack([balance, z]), counts.to(torch.int32), seq_tokens, lse


def _router_gradient(state, dtype):
    logits, ids = state["logits"].to(dtype), state["ids"].long()
    experts, k = logits.shape[1], ids.shape[1]
    valid, member = _members(state, dtype)
    n, filled = state["seq_tokens"][:-2].to(dtype), state["seq_tokens"][-1].to(dtype).clamp(min=1)
    total = state["seq_tokens"][-2].to(dtype).clamp(min=1)
    d_loss = state["d_loss"].to(dtype)
    lse = state["lse"].to(dtype)[:, None]
    p = torch.where(valid[:, None], torch.exp(logits - lse), torch.zeros_like(logits))
    per_seq = state["counts"].to(dtype) * (d_loss[0] * experts / (k * filled)) / (n * n).clamp(min=1)[:, None]
    a = member.t() @ per_seq
    d = p * (a - (p * a).sum(1, keepdim=True)) + d_loss[1] * 2 / total * lse * p
    w, dw = state["weights"].to(dtype), state["d_weights"].to(dtype)
    through = w * (dw - (w * dw).sum(1, keepdim=True))
    d = d.scatter_add(1, ids, torch.where(valid[:, None], through, torch.zeros_like(through)))
    return d


# ---- one pass -----------------------------------------------------------------------

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        return _run_own(state)
    if op == "quant":
        x = state["x"].float()
        return {"along_rows": _values(x).to(torch.bfloat16), "along_cols": _values(x.t().contiguous()).to(torch.bfloat16)}
    if op == "linear":
        y = _values(state["x"].float()) @ _unpacked(*state["w"], case["k"]).t()
        return {"y": y.to(torch.bfloat16)}
    if op == "backward":
        dy = state["dy"].float()
        dx = _values(dy) @ _unpacked(*state["w_cols"], case["n"]).t()
        dw = _values(dy.t().contiguous()) @ _unpacked(*state["x_cols"], case["m"]).t()
        return {"dx": dx.to(torch.bfloat16), "dw": dw}
    if op == "balance":
        loss, counts, seq_tokens, lse = _balance(state, torch.float32)
        return {"loss": loss, "counts": counts, "seq_tokens": seq_tokens, "lse": lse}
    return {"d_logits": _router_gradient(state, torch.float32)}


def _run_own(state):
    import mxfp4_quantized_weights_amd as moe
    case, op = state["case"], state["case"]["op"]
    if op == "quant":
        q_row, s_row, q_col, s_col = moe.moe_mxfp4_quant(state["x"], rows=True, cols=True)
        return {"along_rows": moe.moe_mxfp4_dequant(q_row, s_row, case["cols"], torch.bfloat16),
                "along_cols": moe.moe_mxfp4_dequant(q_col, s_col, case["rows"], torch.bfloat16)}
    if op == "linear":
        return {"y": moe.moe_mxfp4_linear(state["x"], *state["w"])}
    if op == "backward":
        dx, dw = moe.moe_mxfp4_linear_bwd(state["dy"], state["x_cols"], state["w_cols"])
        return {"dx": dx, "dw": dw}
    if op == "balance":
        loss, counts, seq_tokens, lse = moe.moe_balance_loss(state["logits"], state["ids"], token_mask=state["mask"],
                                                             seq_offsets=state["offsets"])
        return {"loss": loss, "counts": counts, "seq_tokens": seq_tokens, "lse": lse}
    return {"d_logits": moe.moe_router_bwd(state["logits"], state["ids"], state["weights"], state["d_weights"],
                                           state["lse"], state["counts"], state["seq_tokens"], state["d_loss"],
                                           token_mask=state["mask"], seq_offsets=state["offsets"])}


# ---- what a pass cannot do without ----------------------------------------------------

def _mx_bytes(rows, cols):
    return rows * _up(cols) * (1 / 2 + 1 / 32)


def work(case):
    op = case["op"]
    if op == "quant":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * ((2 if case["dtype"] == "bf16" else 4) + 2 + 2), "flops": 8.0 * r * c}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * 2 + _mx_bytes(n, k) + m * n * 2, "flops": 2.0 * m * n * k}
    if op == "backward":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * n * 2 + _mx_bytes(k, n) + _mx_bytes(k, m) + m * k * 2 + n * k * 4, "flops": 4.0 * m * n * k}
    t, e, k, s = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    if op == "balance":
        return {"bytes": t * (4 * e + 4 * k + 1 + 4) + s * (4 * e + 8), "flops": 5.0 * t * e}
    return {"bytes": t * (8 * e + 12 * k + 1 + 4) + s * (4 * e + 8), "flops": 8.0 * t * e}


# ---- from the definitions, in 64 bits ---------------------------------------------------

def _exact_values(v):
    """MXFP4 of [R, C] by search: the scale is 2^(e - 2), 2^e the largest power of two not above the group's largest
    magnitude; each value goes to the nearest grid point, of two equally near ones to that of even code."""
    v = v.double()
    rows, cols = v.shape
    full = torch.zeros(rows, _up(cols), dtype=torch.float64, device=v.device)
    full[:, :cols] = v
    groups = full.view(rows, -1, GROUP)
    amax = groups.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    scale = torch.exp2((e - 2).clamp(-127, 127))
    a = groups.abs() / scale
    code = torch.zeros_like(a, dtype=torch.int64)
    for upper in range(1, 8):
        middle = (E2M1[upper - 1] + E2M1[upper]) / 2
        code += (a >= middle) if upper % 2 == 0 else (a > middle)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    out = torch.sign(groups) * grid[code] * scale
    return torch.where(amax > 0, out, torch.zeros_like(out)).view(rows, -1)[:, :cols]


def _exact_unpacked(codes, scales, cols):
    """Values of packed codes: sign, two exponent bits and one mantissa bit of each nibble, times 2^(byte - 127)."""
    nibble = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).to(torch.float64)
    sign = 1 - 2 * torch.floor(nibble / 8)
    field = nibble % 8
    exponent, mantissa = torch.floor(field / 2), field % 2
    magnitude = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(exponent - 1))
    scale = torch.exp2(scales.to(torch.float64) - 127).repeat_interleave(GROUP, 1)
    return (sign * magnitude * scale)[:, :cols]


def _exact_router(state, gradient):
    """Sequence by sequence, from the probabilities themselves."""
    logits = state["logits"].double()
    tokens, experts = logits.shape
    ids = state["ids"].long()
    k = ids.shape[1]
    edges = state["offsets"].tolist()
    seqs = len(edges) - 1
    usable = (state["mask"] != 0) & ~torch.isinf(logits).all(1)
    lse_all = torch.logsumexp(logits, 1)
    prob = torch.softmax(logits, 1)
    lse = torch.zeros(tokens, dtype=torch.float64, device=logits.device)
    counts = torch.zeros(seqs, experts, dtype=torch.int32, device=logits.device)
    sizes, parts, chosen_rows = [], [], []
    for s in range(seqs):
        rows = torch.arange(edges[s], edges[s + 1], device=logits.device)
        rows = rows[usable[rows]]
        chosen_rows.append(rows)
        sizes.append(len(rows))
        lse[rows] = lse_all[rows]
        if not len(rows):
            continue
        count = torch.bincount(ids[rows].reshape(-1), minlength=experts)
        counts[s] = count.to(torch.int32)
        share = count.double() / (k * len(rows))
        parts.append(experts * (share * prob[rows].mean(0)).sum())
    filled, total = len(parts), sum(sizes)
    if not gradient:
        zero = torch.zeros((), dtype=torch.float64, device=logits.device)
        loss = torch.stack([torch.stack(parts).mean() if parts else zero, lse.square().sum() / max(total, 1)])
        seq_tokens = torch.tensor(sizes + [total, filled], dtype=torch.int32, device=logits.device)
        return {"loss": loss, "counts": counts, "seq_tokens": seq_tokens, "lse": lse}
    g_balance, g_z = state["d_loss"].double()
    d = torch.zeros_like(logits)
    for s, rows in enumerate(chosen_rows):
        if not len(rows):
            continue
        p = prob[rows]
        slope = g_balance / filled * experts * counts[s].double() / (k * len(rows)) / len(rows)
        row = p * slope - p * (p @ slope)[:, None] + g_z / total * 2 * lse[rows, None] * p
        w, dw = state["weights"][rows].double(), state["d_weights"][rows].double()
        row.scatter_add_(1, ids[rows], w * dw - w * (w * dw).sum(1, keepdim=True))
        d[rows] = row
    return {"d_logits": d}


def exact(case, seed):
    state, op = prepare(case, seed), case["op"]
    if op == "quant":
        return {"along_rows": _exact_values(state["x"]), "along_cols": _exact_values(state["x"].t())}
    if op == "linear":
        return {"y": _exact_values(state["x"]) @ _exact_unpacked(*state["w"], case["k"]).t()}
    if op == "backward":
        return {"dx": _exact_values(state["dy"]) @ _exact_unpacked(*state["w_cols"], case["n"]).t(),
                "dw": _exact_values(state["dy"].t()) @ _exact_unpacked(*state["x_cols"], case["m"]).t()}
    return _exact_router(state, op == "router")
