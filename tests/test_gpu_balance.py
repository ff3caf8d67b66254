"""GPU tests of the router's training operators against plain 64-bit forms
and differences.

Tolerances.  With u = 2^-24 and L = max |lse| + max |l - lse| of the finite
logits: the row sum of E exponentials (each a few ulp) is off by (E + 8) u
relative, lse by that plus 2 u |lse| absolute, p by
(E + 8 + 4 L) u relative; call it d.  A loss or a gradient is a sum of at most
E terms, each a product of a few such factors, averaged over tokens; sums of n
terms in fp32 add n u of the terms' total magnitude.  The chunk sums are at
most 64 + 16 + 256 additions deep."""
import math

import pytest
import torch

import mx_reference as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def M():
    import mxfp4_quantized_weights_amd as mod
    return mod


def _rel(logits):
    lg = logits.cpu().double()
    lse = torch.logsumexp(lg, 1)
    ok = torch.isfinite(lse)
    if not ok.any():
        return 400 * U
    d = (lg[ok] - lse[ok, None])
    L = lse[ok].abs().max().item() + d[torch.isfinite(d)].abs().clamp(max=110).max().item()
    return (lg.shape[1] + 400 + 4 * L) * U


def _inputs(T, E, k, seed, off=0.0):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(T, E, generator=g) * 2
    if off:
        drop = torch.rand(T, E, generator=g) < off
        drop[:, :k] = False
        lg[drop] = -math.inf
    return lg.cuda()


def _check(M, lg, k, mask=None, offsets=None, ids=None, seed=0):
    T, E = lg.shape
    routed, w = M.moe_route_topk(lg.nan_to_num(0.0, neginf=-math.inf), k)
    ids = routed if ids is None else ids
    mask_d = mask.cuda() if mask is not None else None
    off_d = torch.tensor(offsets, dtype=torch.int32, device="cuda") if offsets is not None else None
    off_c = torch.tensor(offsets) if offsets is not None else None
    loss, counts, seq_tokens, lse = M.moe_balance_loss(lg, ids, mask_d, off_d)
    rl, rc, rs, rlse, valid = R.balance(lg, ids, mask, off_c)
    rel = _rel(lg)
    assert torch.equal(counts.cpu().long(), rc) and torch.equal(seq_tokens.cpu().long(), rs)
    assert ((lse.cpu().double() - rlse).abs() <= rel * (1 + rlse.abs())).all()
    assert ((loss.cpu().double() - rl).abs() <= 4 * rel * (rl.abs() + (rl[1] > 0) * 1.0)).all(), (loss, rl)
    again = M.moe_balance_loss(lg, ids, mask_d, off_d)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, seq_tokens, lse)))

    g = torch.Generator().manual_seed(seed)
    dw = torch.randn(T, k, generator=g).cuda()
    d_loss = torch.tensor([0.7 * T, -0.3 * T], device="cuda")
    both = M.moe_router_bwd(lg, ids, w, dw, lse, counts, seq_tokens, d_loss, mask_d, off_d)
    only_w = M.moe_router_bwd(lg, ids, w, dw, token_mask=mask_d, seq_offsets=off_d)
    only_l = M.moe_router_bwd(lg, ids, lse=lse, counts=counts, seq_tokens=seq_tokens, d_loss=d_loss, token_mask=mask_d,
                              seq_offsets=off_d)
    n_min = max(1, min([int(x) for x in rs[:-2] if x > 0] or [1]))
    # magnitudes of the terms: a_e <= |g_b| E / (S' n_s) (counts <= k n_s), z term |g_z| 2 |lse| / N, w dw
    top = (0.7 * T * E / (max(1, int(rs[-1])) * n_min) * (rc.double().max().item() / (k * n_min) if rc.numel() else 0)
           + 0.6 * T * rlse.abs().max().item() / max(1, int(rs[-2])) if T else 0.0)
    for got, dwx, dlx in ((both, dw, d_loss), (only_w, dw, None), (only_l, None, d_loss)):
        ref = R.router_gradient(lg, ids, w, dwx, dlx, mask, off_c)
        size = (top if dlx is not None else 0.0) + (2 * dw.abs().max().item() if dwx is not None and T else 0.0)
        assert ((got.cpu().double() - ref).abs() <= 4 * rel * size).all(), ((got.cpu().double() - ref).abs().max(), size)
        assert (got.cpu()[~valid] == 0).all()
    return loss, counts


@pytest.mark.parametrize("T", [1, 2, 5, 63, 64, 65, 130, 700])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (63, 3), (64, 8), (65, 1), (288, 8), (300, 16), (513, 4), (1024, 16)])
def test_one_sequence(M, T, E, k):
    _check(M, _inputs(T, E, k, T + E), k)


def test_even_counts_give_one(M):
    E, k = 16, 4
    lg = torch.zeros(8, E, device="cuda")
    ids = (torch.arange(8 * k).reshape(8, k) % E).to(torch.int32).cuda()
    loss, counts, _, _ = M.moe_balance_loss(lg, ids)
    assert (counts == 2).all()
    assert abs(loss[0].item() - 1.0) <= 40 * U and abs(loss[1].item() - math.log(E) ** 2) <= 40 * U * 8


@pytest.mark.parametrize("offsets", [[0, 300], [0, 0, 300], [0, 300, 300], [5, 64, 64, 65, 128, 200, 290], [0, 1, 2, 3, 300],
                                     [300, 300], [0, 0], [64, 128], list(range(0, 301))])
@pytest.mark.parametrize("masked", [False, True])
def test_sequences_and_masks(M, offsets, masked):
    lg = _inputs(300, 40, 4, 1, off=0.2)
    mask = None
    if masked:
        mask = (torch.rand(300, generator=torch.Generator().manual_seed(2)) > 0.3).to(torch.uint8)
        mask[64:128] = 0                        # a whole sequence and a whole chunk
        lg[mask.cuda() == 0] = math.nan         # what is left out is not used
    _check(M, lg, 4, mask, offsets)


def test_rows_with_nothing_left(M):
    lg = _inputs(100, 24, 2, 3)
    lg[10] = -math.inf
    lg[99] = -math.inf
    lg[20, 3:] = -math.inf
    lg[30] = torch.finfo(torch.float32).min     # uniform, not excluded
    lg[31, 1:] = torch.finfo(torch.float32).min
    ids, w = M.moe_route_topk(lg, 2)
    loss, counts, seq_tokens, lse = M.moe_balance_loss(lg, ids)
    rl, rc, rs, rlse, _ = R.balance(lg, ids)
    assert torch.equal(counts.cpu().long(), rc) and torch.equal(seq_tokens.cpu().long(), rs)
    assert seq_tokens[0] == 98 and lse[10] == 0 and math.isinf(loss[1].item())   # lse^2 of the lowest row passes fp32
    assert abs(loss[0].item() - rl[0].item()) <= 4 * _rel(lg[:10]) * rl[0].item()
    d = M.moe_router_bwd(lg, ids, lse=lse, counts=counts, seq_tokens=seq_tokens, d_loss=torch.tensor([1.0, 0.0], device="cuda"))
    assert torch.isfinite(d).all() and (d[10] == 0).all() and (d[20, 3:] == 0).all()
    ref = R.router_gradient(lg, ids, None, None, torch.tensor([1.0, 0.0]))
    # terms up to E counts / n^2 in size (counts <= 98); the row sums' and exponentials' error as above
    assert ((d.cpu().double() - ref).abs() <= 4 * _rel(lg[:10]) * 24 * 98 / 98 ** 2).all()
    everything = torch.full((5, 24), -math.inf, device="cuda")
    loss, counts, seq_tokens, lse = M.moe_balance_loss(everything, ids[:5].contiguous())
    assert (loss == 0).all() and (counts == 0).all() and (seq_tokens == 0).all() and (lse == 0).all()


def test_nan_and_infinite_logits_show(M):
    for bad in (math.nan, math.inf):
        lg = _inputs(70, 24, 2, 4)
        ids, _ = M.moe_route_topk(lg, 2)
        lg[66, 5] = bad
        loss = M.moe_balance_loss(lg, ids)[0]
        assert torch.isnan(loss).all()


def test_ids_out_of_range_and_repeated(M):
    lg = _inputs(80, 24, 4, 5)
    ids = torch.randint(0, 24, (80, 4), generator=torch.Generator().manual_seed(6)).to(torch.int32)
    ids[3] = torch.tensor([-1, 24, 5, 1 << 30], dtype=torch.int32)
    ids[4] = 7
    _check(M, lg, 4, ids=ids.cuda())


def test_no_tokens(M):
    lg, ids = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, seq_tokens, lse = M.moe_balance_loss(lg, ids)
    assert (loss == 0).all() and (counts == 0).all() and (seq_tokens == 0).all() and lse.shape == (0,)
    d = M.moe_router_bwd(lg, ids, torch.empty(0, 2, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert d.shape == (0, 8)


def test_many_tokens_and_sequences(M):
    """Sums over many chunks against 64 bits, vectorised (the row-by-row form
    is too slow here): 20000 tokens, 1000 sequences."""
    T, E, k, S = 20000, 96, 6, 1000
    lg = _inputs(T, E, k, 7)
    ids, _ = M.moe_route_topk(lg, k)
    cuts = torch.randint(0, T + 1, (S - 1,), generator=torch.Generator().manual_seed(8)).sort().values
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])])
    loss, counts, seq_tokens, lse = M.moe_balance_loss(lg, ids, seq_offsets=off.to(torch.int32).cuda())
    x = lg.cpu().double()
    rlse = torch.logsumexp(x, 1)
    seq = torch.searchsorted(off, torch.arange(T), right=True) - 1
    p = torch.zeros(S, E, dtype=torch.float64).index_add_(0, seq, torch.exp(x - rlse[:, None]))
    c = torch.zeros(S * E, dtype=torch.int64).index_add_(0, (seq[:, None] * E + ids.cpu().long()).reshape(-1),
                                                        torch.ones(T * k, dtype=torch.int64)).view(S, E)
    n = torch.bincount(seq, minlength=S)
    assert torch.equal(counts.cpu().long(), c) and torch.equal(seq_tokens.cpu().long()[:S], n)
    nn = n.clamp(min=1).double()[:, None]
    ref = ((c * E / (k * nn)) * (p / nn)).sum(1)[n > 0].mean().item(), (rlse ** 2).mean().item()
    rel = _rel(lg)
    assert abs(loss[0].item() - ref[0]) <= 4 * rel * ref[0] and abs(loss[1].item() - ref[1]) <= 4 * rel * (ref[1] + 1)


def test_more_sequences_than_tokens(M):
    """Sequence search over many, mostly empty, sequences, in one chunk and in several."""
    g = torch.Generator().manual_seed(11)
    for T, S in ((50, 9000), (300, 5000)):
        off = torch.randint(0, T + 1, (S + 1,), generator=g).sort().values.tolist()
        _check(M, _inputs(T, 12, 2, T), 2, None, off)


def test_offsets_outside_the_batch_are_clamped(M):
    lg = _inputs(100, 16, 2, 12)
    ids, _ = M.moe_route_topk(lg, 2)
    d = torch.tensor([1.0, 1.0], device="cuda")
    for bad, good in (([-5, 40, 1000], [0, 40, 100]), ([200, 300], [100, 100]), ([-9, -1], [0, 0])):
        res = []
        for off in (bad, good):
            off = torch.tensor(off, dtype=torch.int32, device="cuda")
            out = M.moe_balance_loss(lg, ids, seq_offsets=off)
            res.append(out + (M.moe_router_bwd(lg, ids, lse=out[3], counts=out[1], seq_tokens=out[2], d_loss=d, seq_offsets=off),))
        assert all(torch.equal(a, b) for a, b in zip(*res))


def test_binding_refusals_on_the_device(M):
    lg = _inputs(10, 16, 2, 13)
    ids, w = M.moe_route_topk(lg, 2)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    bad = [lambda: M.moe_balance_loss(lg, ids.long()), lambda: M.moe_balance_loss(lg.t(), ids),
           lambda: M.moe_balance_loss(lg, ids[:5]), lambda: M.moe_balance_loss(lg, ids, token_mask=w[:, 0]),
           lambda: M.moe_balance_loss(lg, ids, seq_offsets=i32(0)), lambda: M.moe_balance_loss(lg, ids, seq_offsets=i32(0, 10).cpu()),
           lambda: M.moe_router_bwd(lg, ids, w, w[:5].contiguous()), lambda: M.moe_router_bwd(lg, ids, w, w.double()),
           lambda: M.moe_router_bwd(lg, ids, w, w, d_logits=lg[:5]),
           lambda: M.moe_balance_loss(lg.new_zeros((1 << 24) + 1, 1), ids.new_zeros((1 << 24) + 1, 1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_gradient_against_differences(M):
    """Central differences of loss(logits) = 3 balance + 0.5 z + sum weights * c
    in 64 bits, selection and counts held."""
    T, E, k = 12, 20, 3
    lg = _inputs(T, E, k, 9)
    ids, w = M.moe_route_topk(lg, k)
    c = torch.randn(T, k, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    off = [0, 5, 5, 11]
    mask = torch.ones(T, dtype=torch.uint8)
    mask[2] = 0
    loss, counts, seq_tokens, lse = M.moe_balance_loss(lg, ids, mask.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"))
    d = M.moe_router_bwd(lg, ids, w, c.float().cuda(), lse, counts, seq_tokens, torch.tensor([3.0, 0.5], device="cuda"),
                         mask.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda")).cpu().double()

    def total(x):
        rl, _, _, _, valid = R.balance(x, ids, mask, torch.tensor(off))
        ww = torch.softmax(x.gather(1, ids.cpu().long()), 1)
        return 3 * rl[0] + 0.5 * rl[1] + (ww * c * valid[:, None]).sum()

    x = lg.cpu().double()
    h = 1e-5
    for t, e in ((0, 0), (0, int(ids[0, 0])), (2, 3), (4, int(ids[4, 2])), (10, 7), (11, 0)):
        up, dn = x.clone(), x.clone()
        up[t, e] += h
        dn[t, e] -= h
        diff = (total(up) - total(dn)).item() / (2 * h)
        # differences: h^2 of third derivatives (below 100 here) and 1e-16 / h of rounding; the gradient: fp32
        assert abs(diff - d[t, e].item()) <= 100 * h * h + 1e-14 / h + 8 * _rel(lg) * 10


def test_given_output_other_stream_and_graph(M):
    lg = _inputs(200, 50, 4, 10)
    ids, w = M.moe_route_topk(lg, 4)
    dw = torch.randn(200, 4, device="cuda")
    dl = torch.tensor([1.0, 2.0], device="cuda")
    off = torch.tensor([0, 90, 180], dtype=torch.int32, device="cuda")

    def step(x, **kw):
        loss, counts, seq_tokens, lse = M.moe_balance_loss(x, ids, seq_offsets=off, **kw)
        return loss, counts, M.moe_router_bwd(x, ids, w, dw, lse, counts, seq_tokens, dl, seq_offsets=off, **kw)

    want = step(lg)
    out = torch.full((200, 50), 9.0, device="cuda")
    assert M.moe_router_bwd(lg, ids, w, dw, d_logits=out, seq_offsets=off) is out and (out[180:] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(lg, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = lg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static)
    for i in range(4):
        static.copy_(_inputs(200, 50, 4, 20 + i))
        want = step(static)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
