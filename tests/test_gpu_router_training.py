"""A training step of the trainable dense parts of an MoE layer around frozen
quantised experts: router logits by a dense MXFP4 product, routing, the experts'
outputs per pair, balance and z loss, the gradient to the logits, and the router
layer's own gradients.  Each stage against a plain 64-bit form on the stage's own
inputs, and the loss against differences in the logits."""
import pytest
import torch

import mx_reference as R
import workloads as W
from parity_util import gpu_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_quantized_weights_amd as mod
    return mod


def _pair_outputs(M, wl, x, ids, ew):
    """y [T * k, H]: the expert's output for each (token, slot) pair, unweighted:
    the layer's stages with every pair a token of its own."""
    T, k = ids.shape
    cfg = M.make_cfg(wl.E, 1, wl.mode, wl.H, wl.I, block_m=16, swiglu_limit=wl.swiglu_limit)
    xq, xs = M.moe_quant_act(x.repeat_interleave(k, 0), cfg.pad.hidden_padded, wl.mode)
    sorted_ids, block_expert, _, npp = M.moe_permute_align(ids.reshape(-1, 1).contiguous(), wl.E, cfg.block_m)
    w13, s13, w2, s2 = ew.tiled()
    aq, as_ = M.moe_grouped_gemm1_swiglu(cfg, T * k, xq, xs, sorted_ids, block_expert, npp, w13, s13)
    ones = torch.ones(T * k, 1, device="cuda")
    return M.moe_grouped_gemm2_combine(cfg, T * k, aq, as_, sorted_ids, block_expert, npp, w2, s2, ones)


@pytest.mark.parametrize("T", [5, 150])
def test_training_step(M, T):
    wl = W.WORKLOADS["tiny_fp8"].with_(mode="mxfp4", T=T, E=24, top_k=4)
    E, k, H = wl.E, wl.top_k, wl.H
    cfg = M.make_cfg(E, k, wl.mode, H, wl.I, block_m=16, swiglu_limit=wl.swiglu_limit)
    ew = gpu_weights(M, cfg, wl, source="cuda")
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn(E, H, generator=g) * 0.1).cuda()
    mask = torch.ones(T, dtype=torch.uint8)
    mask[T // 2] = 0
    off = torch.tensor([0, T // 3, T - 1])              # the last row lies behind the last sequence
    mask_d, off_d = mask.cuda(), off.to(torch.int32).cuda()
    coef, goal = (0.3, 0.02), torch.randn(T, H, generator=g, dtype=torch.float64)
    goal[T // 2] = goal[T - 1] = 0                     # padding takes no part in the loss

    # forward
    xq, xs, xc, xcs = M.moe_mxfp4_quant(x, rows=True, cols=True)
    wq, ws, wc, wcs = M.moe_mxfp4_quant(wr, rows=True, cols=True)
    logits = M.moe_mxfp4_matmul(xq, xs, wq, ws, out_dtype=torch.float32)
    assert torch.equal(M.moe_mxfp4_linear(x, wq, ws, out_dtype=torch.float32).argmax(1), logits.argmax(1))
    ref, mass = R.product(R.quantised_values(x), R.quantised_values(wr))
    assert ((logits.cpu().double() - ref).abs() <= R.product_bound(ref, mass, H, torch.float32)).all()
    ids, weights = M.moe_route_topk(logits, k)
    y = _pair_outputs(M, wl, x, ids, ew).double().cpu().view(T, k, H)
    out = M.moe_forward(cfg, x, logits, *ew.tiled()).double().cpu()
    # the layer's own combine of the same pair outputs: each rounded to bf16 here (2^-8 of it), its block floating
    # point rows and the bf16 result there
    mix = (weights.cpu().double()[..., None] * y).sum(1)
    size = (weights.cpu().double()[..., None] * y.abs()).sum(1).amax(1, keepdim=True)
    assert ((out - mix).abs() <= 3 * 2.0 ** -8 * size).all()
    loss, counts, seq_tokens, lse = M.moe_balance_loss(logits, ids, mask_d, off_d)

    # backward
    d_weights = (y * goal[:, None]).sum(2).float().cuda()
    d_loss = torch.tensor(coef, device="cuda")
    d_logits = M.moe_router_bwd(logits, ids, weights, d_weights, lse, counts, seq_tokens, d_loss, mask_d, off_d)
    dx, dwr = M.moe_mxfp4_linear_bwd(d_logits, (xc, xcs), (wc, wcs), dx_dtype=torch.float32)

    want = R.router_gradient(logits, ids, weights, d_weights, d_loss, mask, off)
    scale = want.abs().max()
    assert ((d_logits.cpu().double() - want).abs() <= 1e-4 * scale).all()   # (E + 400 + 4 L) 2^-24 with E = 24, L < 100

    def total(l):
        rl = R.balance(l, ids, mask, off)[0]
        w = torch.softmax(l.gather(1, ids.cpu().long()), 1)
        return coef[0] * rl[0] + coef[1] * rl[1] + ((w[..., None] * y).sum(1) * goal).sum()

    l0 = logits.cpu().double()
    for t, e in ((0, int(ids[0, 0])), (1, int(ids[1, 3])), (T // 3, 5), (T - 2, 7)):
        if not mask[t]:
            continue
        h = 1e-5
        up, dn = l0.clone(), l0.clone()
        up[t, e] += h
        dn[t, e] -= h
        diff = (total(up) - total(dn)).item() / (2 * h)
        # h^2 of third derivatives and 2^-52 / h of the loss's size, beside the gradient's own error
        bound = 1e-4 * scale + h * h * 100 * scale + 2.0 ** -50 * (y.abs() * goal.abs()[:, None]).sum() / h
        assert abs(diff - d_logits[t, e].item()) <= bound

    for got, (ref, mass), n in (
            (dx, R.product(R.quantised_values(d_logits), R.quantised_values(wr.t())), E),
            (dwr, R.product(R.quantised_values(d_logits.t()), R.quantised_values(x.t())), T)):
        assert ((got.cpu().double() - ref).abs() <= R.product_bound(ref, mass, n, torch.float32)).all()
    again = M.moe_mxfp4_linear_bwd(d_logits, (xc, xcs), dw=dwr.clone(), accumulate=True)[1]
    assert torch.allclose(again, 2 * dwr, rtol=2.0 ** -22, atol=0)
