"""Plain 64-bit forms of the dense MXFP4 operators and of the router's
training operators, written from their definitions, for the tests."""
import math

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def up128(n):
    return -(-n // 128) * 128


def quantise(v):
    """[R, C] -> (codes uint8 [R, Cp] one per byte, scale bytes int64 [R, Cp/32])."""
    v = v.detach().cpu().double()
    R, C = v.shape
    full = torch.zeros(R, up128(C), dtype=torch.float64)
    full[:, :C] = v
    g = full.view(R, up128(C) // 32, 32)
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], torch.zeros_like(g), g)
    amax = g.abs().amax(-1)
    # floor(log2): an fp32 value is m 2^e with 0.5 <= m < 1 exactly in 64 bits
    b = (torch.frexp(amax)[1].long() - 1 - 2 + 127).clamp(0, 254)
    b = torch.where(amax > 0, b, torch.zeros_like(b))
    a = (g.abs() / torch.exp2(b.double() - 127)[..., None]).clamp(max=6.0)
    code = torch.zeros_like(a, dtype=torch.long)
    for i in range(1, 8):
        mid = (GRID[i - 1] + GRID[i]) / 2
        code += ((a >= mid) if i % 2 == 0 else (a > mid)).long()
    code |= torch.signbit(g).long() << 3
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    b = torch.where(bad, torch.full_like(b, 255), b)
    return code.view(R, -1).to(torch.uint8), b


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(q):
    return torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def values(code, b):
    """Codes (one per byte) and scale bytes -> float64 values [R, Cp]."""
    table = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64)
    scale = torch.where(b == 255, torch.full(b.shape, math.nan, dtype=torch.float64), torch.exp2(b.double() - 127))
    return table[code.long()] * scale.repeat_interleave(32, 1)


def quantised_values(v):
    return values(*quantise(v))[:, :v.shape[1]]


def product(a, b):
    """-> (a b^T, |a| |b|^T) in 64 bits, on the GPU where there is one."""
    if torch.cuda.is_available():
        a, b = a.cuda(), b.cuda()
    return (a @ b.t().contiguous()).cpu(), (a.abs() @ b.abs().t().contiguous()).cpu()


def product_bound(ref, mass, K, dtype):
    """Largest error of a product's elements: K additions in fp32, each off by
    at most 2^-23 of a partial sum that `mass` bounds (2^-24 rounding, twice
    that where the matrix core truncates), then one rounding to the output
    type, off by half a step."""
    acc = (K + 2) * 2.0 ** -23 * mass
    return acc + torch.finfo(dtype).eps / 2 * (ref.abs() + acc) + 1e-38


def balance(logits, ids, mask=None, offsets=None):
    """-> (loss [2], counts [S, E], seq_tokens, lse, valid) as moe_balance_loss defines them."""
    lg = logits.detach().cpu().double()
    T, E = lg.shape
    k = ids.shape[1]
    ids = ids.cpu().long()
    edges = offsets.tolist() if offsets is not None else [0, T]
    ok = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu() != 0
    ok &= ~(lg == -math.inf).all(1)
    counts = torch.zeros(len(edges) - 1, E, dtype=torch.int64)
    lse = torch.zeros(T, dtype=torch.float64)
    valid = torch.zeros(T, dtype=torch.bool)
    n, parts, zs = [], [], []
    for s, (lo, hi) in enumerate(zip(edges, edges[1:])):
        rows = [t for t in range(lo, hi) if ok[t]]
        n.append(len(rows))
        if not rows:
            continue
        valid[rows] = True
        l = lg[rows]
        lse[rows] = torch.logsumexp(l, 1)
        P = torch.softmax(l, 1).sum(0) / len(rows)
        picked = ids[rows].reshape(-1)
        counts[s] = torch.bincount(picked[(picked >= 0) & (picked < E)], minlength=E)
        parts.append((counts[s].double() * E / (k * len(rows)) * P).sum().item())
        zs.append((lse[rows] ** 2).sum().item())
    N = sum(n)
    loss = torch.tensor([sum(parts) / len(parts) if parts else 0.0, sum(zs) / N if N else 0.0], dtype=torch.float64)
    return loss, counts, torch.tensor(n + [N, len(parts)]), lse, valid


def router_gradient(logits, ids, weights, d_weights, d_loss, mask=None, offsets=None):
    lg = logits.detach().cpu().double()
    T, E = lg.shape
    k = ids.shape[1]
    ids = ids.cpu().long()
    _, counts, seq_tokens, lse, valid = balance(logits, ids, mask, offsets)
    edges = offsets.tolist() if offsets is not None else [0, T]
    N, filled = int(seq_tokens[-2]), int(seq_tokens[-1])
    d = torch.zeros(T, E, dtype=torch.float64)
    for s, (lo, hi) in enumerate(zip(edges, edges[1:])):
        for t in range(lo, hi):
            if not valid[t]:
                continue
            if d_loss is not None:
                g = d_loss.cpu().double()
                p = torch.softmax(lg[t], 0)
                a = g[0] * E * counts[s].double() / (filled * k * float(seq_tokens[s]) ** 2)
                d[t] += p * (a - (p * a).sum()) + g[1] * 2 / N * lse[t] * p
            if d_weights is not None:
                live = [j for j in range(k) if 0 <= ids[t, j] < E]
                w, dw = weights[t].cpu().double(), d_weights[t].cpu().double()
                mean = sum(float(w[j] * dw[j]) for j in live)
                for j in live:
                    d[t, ids[t, j]] += w[j] * (dw[j] - mean)
    return d
