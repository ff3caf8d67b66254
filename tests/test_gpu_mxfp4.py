"""GPU tests of the dense MXFP4 operators against plain 64-bit forms: codes
and scales bit for bit, products within the fp32 sums' and the output
rounding's bounds (mx_reference.product_bound)."""
import math

import pytest
import torch

import mx_reference as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    import mxfp4_quantized_weights_amd as mod
    return mod


def _matrix(rows, cols, dtype, seed, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if spread:
        x *= torch.exp2(torch.randint(-spread, spread + 1, (rows, cols), generator=g).float())
    return x.to(dtype)


def _check_quant(M, x, **kw):
    qr, sr, qc, sc = M.moe_mxfp4_quant(x.cuda() if not x.is_cuda else x, rows=True, cols=True, **kw)
    torch.cuda.synchronize()
    for q, s, v in ((qr, sr, x), (qc, sc, x.t())):
        code, b = R.quantise(v)
        assert torch.equal(s.cpu().long(), b)
        assert torch.equal(q.cpu(), R.pack(code))
    return qr, sr, qc, sc


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (33, 31), (31, 33), (127, 129), (128, 128), (129, 127),
                                       (1, 4096), (300, 1), (256, 1000), (130, 4000)])
def test_quant_both_ways(M, rows, cols, dtype):
    _check_quant(M, _matrix(rows, cols, dtype, rows * 5000 + cols, spread=6))


def test_quant_one_way_equals_both_and_moe_quant_act(M):
    x = _matrix(70, 200, BF16, 1, spread=3).cuda()
    qr, sr, qc, sc = M.moe_mxfp4_quant(x, rows=True, cols=True)
    a = M.moe_mxfp4_quant(x)
    assert torch.equal(a[0], qr) and torch.equal(a[1], sr) and a[2] is None and a[3] is None
    b = M.moe_mxfp4_quant(x, rows=False, cols=True)
    assert torch.equal(b[2], qc) and torch.equal(b[3], sc) and b[0] is None and b[1] is None
    q, s = M.moe_quant_act(x, 256, "mxfp4")
    assert torch.equal(q, qr) and torch.equal(s, sr)


def test_quant_every_midpoint_and_scale(M):
    """Every grid value and midpoint and its fp32 neighbours at scales over
    fp32's whole range, subnormals and signed zeros included."""
    mids = sorted(set(R.GRID) | {(a + b) / 2 for a, b in zip(R.GRID, R.GRID[1:])} | {7.0, 7.99})
    base = torch.tensor(mids + [-m for m in mids], dtype=torch.float32)
    rows = []
    for e in (-149, -140, -127, -126, -100, -1, 0, 1, 60, 125):
        v = torch.ldexp(base.double(), torch.tensor(e)).float()
        near = torch.cat([v, torch.nextafter(v, torch.tensor(math.inf)), torch.nextafter(v, torch.tensor(-math.inf))])
        near = near[torch.isfinite(near)]
        lead = torch.ldexp(torch.tensor(4.0, dtype=torch.float64), torch.tensor(e)).float()
        pad = (-len(near)) % 31
        near = torch.cat([near, torch.zeros(pad)]).view(-1, 31)
        rows.append(torch.cat([lead.expand(len(near), 1), near], 1))
    x = torch.cat(rows)
    _check_quant(M, x)
    _check_quant(M, x.t().contiguous())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_infinities_and_nan(M, dtype):
    x = _matrix(70, 150, dtype, 3)
    x[0, 5] = math.inf
    x[1, 140] = -math.inf
    x[69, 33] = math.nan
    x[40] = 0
    x[41] = -0.0
    x[:, 77] = torch.finfo(dtype).min
    qr, sr, qc, sc = _check_quant(M, x)
    back = M.moe_mxfp4_dequant(qr, sr, 150, F32).cpu()
    assert torch.isnan(back[0, :32]).all() and torch.isfinite(back[0, 32:]).all()
    y = M.moe_mxfp4_matmul(qr, sr, *M.moe_mxfp4_quant(torch.ones(8, 150, device="cuda"))[:2]).cpu()
    nan_rows = torch.isnan(y.float()).all(1)
    assert nan_rows.nonzero().flatten().tolist() == [0, 1, 69]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_strides_and_alignment(M, dtype):
    big = _matrix(200, 300, dtype, 4).cuda()
    for view in (big[3:90, 8:208], big[1:, 1:], big[:, 5:6], big[5:6], big[::2, :100], big[::3, 3:]):
        _check_quant(M, view)


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (0, 0)])
def test_quant_of_nothing(M, rows, cols):
    qr, sr, qc, sc = M.moe_mxfp4_quant(torch.empty(rows, cols, device="cuda"), rows=True, cols=True)
    assert qr.shape == (rows, R.up128(cols) // 2) and sr.shape == (rows, R.up128(cols) // 32)
    assert qc.shape == (cols, R.up128(rows) // 2) and sc.shape == (cols, R.up128(rows) // 32)
    assert M.moe_mxfp4_dequant(qr, sr, cols).shape == (rows, cols)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [1, 7, 8, 100, 128, 999])
def test_dequant_every_code_and_scale(M, cols, dtype):
    g = torch.Generator().manual_seed(cols)
    n = 256
    q = torch.randint(0, 256, (n, R.up128(cols) // 2), generator=g).to(torch.uint8)
    s = torch.randint(0, 256, (n, R.up128(cols) // 32), generator=g)
    s[:, 0] = torch.arange(n)                   # every scale byte
    ref = R.values(R.unpack(q), s)[:, :cols].to(torch.float32).to(dtype)
    out = torch.full((n, cols + 9), 3.0, dtype=dtype, device="cuda")
    for view in (out[:, :cols], out[:, 1:1 + cols]):
        out.fill_(3.0)
        M.moe_mxfp4_dequant(q.cuda(), s.to(torch.uint8).cuda(), cols, out=view)
        assert torch.equal(view.cpu().isnan(), ref.isnan())
        assert torch.equal(view.cpu().nan_to_num(7), ref.nan_to_num(7))
        assert (out != 3.0).sum() == (view != 3.0).sum()   # nothing beside the view


def _operand(rows, K, seed, spread=2):
    """Random codes and scales, zero codes past K."""
    g = torch.Generator().manual_seed(seed)
    code = torch.randint(0, 16, (rows, R.up128(K)), generator=g).to(torch.uint8)
    code[:, K:] = 0
    b = torch.randint(127 - spread, 128 + spread, (rows, R.up128(K) // 32), generator=g)
    return R.pack(code).cuda(), b.to(torch.uint8).cuda(), R.values(code, b)


def test_binding_refusals_on_the_device(M):
    q, s, _ = _operand(8, 256, 1)
    x = torch.zeros(4, 256, device="cuda")
    bad = [lambda: M.moe_mxfp4_linear(x, q, s[:, :4]), lambda: M.moe_mxfp4_linear(x[:, :100], q, s),
           lambda: M.moe_mxfp4_linear(x, q.cpu(), s), lambda: M.moe_mxfp4_linear(x.t(), q, s),
           lambda: M.moe_mxfp4_linear(x, q, s, out=torch.zeros(4, 9, device="cuda")),
           lambda: M.moe_mxfp4_linear(x, q, s, out=torch.zeros(1, 8, device="cuda").expand(4, 8)),
           lambda: M.moe_mxfp4_linear(x, q, s, out_dtype=torch.float16),
           lambda: M.moe_mxfp4_matmul(q, s, q, s, accumulate=True),
           lambda: M.moe_mxfp4_matmul(q[:, :100].contiguous(), s, q, s),
           lambda: M.moe_mxfp4_matmul(q[::2], s[::2], q, s), lambda: M.moe_mxfp4_dequant(q, s, 300),
           lambda: M.moe_mxfp4_linear_bwd(x, dw=x), lambda: M.moe_mxfp4_linear_bwd(x, x_col=(q, s), dx=x),
           lambda: M.moe_mxfp4_linear_bwd(x[:, :8], w_col=(q, s)),
           lambda: M.moe_mxfp4_quant(x, rows=False),
           lambda: M.moe_mxfp4_quant(x.new_zeros((1 << 24) + 1, 1)),
           lambda: M.moe_mxfp4_linear(x.new_zeros(1, 0), q.new_zeros((1 << 24) + 1, 0), q.new_zeros((1 << 24) + 1, 0))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(M.MoeError):                        # rows that overlap
        M.moe_mxfp4_quant(x[:1].expand(4, 256))
    with pytest.raises(M.MoeError):                        # only fp32 sums accumulate
        M.moe_mxfp4_matmul(q, s, q, s, out=torch.zeros(8, 8, dtype=BF16, device="cuda"), accumulate=True)


SIZES = [(1, 1, 1), (1, 16, 128), (1, 2048, 4096), (3, 257, 1000), (16, 100, 160), (17, 33, 64), (31, 65, 384),
         (32, 32, 512), (33, 1000, 640), (64, 300, 2048), (65, 129, 257), (100, 288, 4096), (128, 128, 128),
         (129, 257, 896), (255, 256, 513), (288, 512, 4001), (257, 1023, 1100), (300, 4000, 1000), (513, 770, 300),
         (1000, 130, 5000), (2, 8192, 96), (7, 31, 16000), (100, 288, 300), (40, 50, 256), (33, 1000, 64), (48, 90, 4500), (63, 35, 3500),
         (100, 70, 2683), (65, 130, 3200), (100, 200, 5188), (40, 300, 6000), (64, 64, 8200),
         (2000, 2050, 1100), (3300, 3900, 600), (3333, 3901, 513)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul(M, m, n, k, dtype):
    a, sa, av = _operand(m, k, 11 * m + n + k)
    b, sb, bv = _operand(n, k, 7 * n + m + k)
    out = M.moe_mxfp4_matmul(a, sa, b, sb, out_dtype=dtype)
    assert out.dtype == dtype
    ref, mass = R.product(av, bv)
    err = (out.cpu().double() - ref).abs()
    assert (err <= R.product_bound(ref, mass, k, dtype)).all(), err.max()
    again = M.moe_mxfp4_matmul(a, sa, b, sb, out_dtype=dtype)
    assert torch.equal(out, again)


def test_matmul_wide_scales(M):
    """Scales over their whole range: products at both ends of fp32."""
    m, n, k = 40, 50, 256
    a, sa, _ = _operand(m, k, 1)
    b, sb, _ = _operand(n, k, 2)
    ca, cb = R.unpack(a.cpu()), R.unpack(b.cpu())
    for lo, hi in ((0, 60), (60, 100), (200, 250), (1, 253)):
        for lo2, hi2 in ((0, 60), (100, 130), (200, 250)):
            g = torch.Generator().manual_seed(lo + lo2)
            ba = torch.randint(lo, hi, sa.shape, generator=g)
            bb = torch.randint(lo2, hi2, sb.shape, generator=g)
            ref, mass = R.product(R.values(ca, ba), R.values(cb, bb))
            out = M.moe_mxfp4_matmul(a, ba.to(torch.uint8).cuda(), b, bb.to(torch.uint8).cuda(), out_dtype=F32).cpu().double()
            safe = mass < 2.0 ** 126
            # below 2^-126 the sums may be flushed: an absolute allowance of K such terms
            bound = R.product_bound(ref, mass, k, F32) + (k + 2) * 2.0 ** -126
            assert ((out - ref).abs() <= bound)[safe].all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(5, 33, 256), (64, 100, 512), (50, 70, 200), (200, 300, 1024), (300, 520, 4096),
                                   (64, 100, 4096), (60, 70, 5120), (2000, 2050, 512), (3300, 3900, 512)])
def test_matmul_strided_out_and_accumulate(M, m, n, k, dtype):
    a, sa, av = _operand(m, k, 5)
    b, sb, bv = _operand(n, k, 6)
    ref, mass = R.product(av, bv)
    for off in (0, 1, 8):
        big = torch.full((m + 2, n + 16), 3.0, dtype=dtype, device="cuda")
        view = big[1:1 + m, off:off + n]
        M.moe_mxfp4_matmul(a, sa, b, sb, out=view)
        bound = R.product_bound(ref, mass, k, dtype)
        assert ((view.cpu().double() - ref).abs() <= bound).all()
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:1 + m, off:off + n] = False
        assert (big[keep] == 3.0).all()
        if dtype == F32:
            before = view.clone()
            M.moe_mxfp4_matmul(a, sa, b, sb, out=view, accumulate=True)
            want = before.cpu().double() + ref
            assert ((view.cpu().double() - want).abs() <= bound + 2.0 ** -23 * (want.abs() + mass)).all()
            assert (big[keep] == 3.0).all()


def test_matmul_empty_sums_and_sides(M):
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 4), 7.0, device="cuda")
    M.moe_mxfp4_matmul(e(3, 0), e(3, 0), e(4, 0), e(4, 0), out=out, accumulate=True)
    assert (out == 7.0).all()
    M.moe_mxfp4_matmul(e(3, 0), e(3, 0), e(4, 0), e(4, 0), out=out)
    assert (out == 0.0).all()
    assert M.moe_mxfp4_matmul(e(0, 64), e(0, 4), e(4, 64), e(4, 4)).shape == (0, 4)
    assert M.moe_mxfp4_matmul(e(4, 64), e(4, 4), e(0, 64), e(0, 4)).shape == (4, 0)
    y = M.moe_mxfp4_linear(torch.empty(3, 0, device="cuda"), e(4, 0), e(4, 0))
    assert (y == 0).all() and y.shape == (3, 4)
    dx, dw = M.moe_mxfp4_linear_bwd(torch.empty(0, 4, device="cuda"), x_col=(e(5, 0), e(5, 0)), w_col=(e(5, 64), e(5, 4)))
    assert dx.shape == (0, 5) and (dw == 0).all() and dw.shape == (4, 5)
    dx, dw = M.moe_mxfp4_linear_bwd(torch.empty(6, 0, device="cuda"), x_col=(e(5, 64), e(5, 4)), w_col=(e(5, 0), e(5, 0)))
    assert (dx == 0).all() and dx.shape == (6, 5) and dw.shape == (0, 5)


def _check_linear(M, x, n, seed, dtype=BF16):
    m, k = x.shape
    w, sw, wv = _operand(n, k, seed)
    out = M.moe_mxfp4_linear(x, w, sw, out_dtype=dtype)
    ref, mass = R.product(R.quantised_values(x), wv[:, :k])
    assert ((out.cpu().double() - ref).abs() <= R.product_bound(ref, mass, k, dtype)).all()
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 13, 16, 17, 31, 32, 33, 64, 100, 129, 300])
@pytest.mark.parametrize("n,k", [(2048, 4096), (4000, 1000), (100, 33), (33, 4200)])
def test_linear(M, m, n, k, dtype):
    x = _matrix(m, k, dtype, m + n, spread=2).cuda()
    x[m // 2, k // 3] = 100
    _check_linear(M, x, n, m, dtype)


@pytest.mark.parametrize("m", [1, 7, 16, 40])
def test_linear_views_and_nan(M, m):
    big = _matrix(m + 4, 1100, BF16, m).cuda()
    for off in (0, 1, 8):
        _check_linear(M, big[2:2 + m, off:off + 1000], 200, 9)
    x = big[:m, :1000].clone()
    x[m - 1, 999] = math.nan
    y = _check_nan(M, x)
    assert torch.isnan(y[m - 1]).all() and torch.isfinite(y[:m - 1]).all()


def _check_nan(M, x):
    w, sw, _ = _operand(200, x.shape[1], 9)
    return M.moe_mxfp4_linear(x, w, sw).float().cpu()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 40, 100), (130, 257, 300), (257, 100, 513), (1000, 288, 640)])
def test_linear_bwd(M, m, n, k, dtype):
    """Against the formulas; and both gradients alone, accumulated, and as
    differences of the layer's own loss (it is linear in w and x once they
    and dy are quantised)."""
    dy = _matrix(m, n, dtype, m, spread=1).cuda()
    x = _matrix(m, k, BF16, n).cuda()
    w = _matrix(n, k, F32, k).cuda()
    x_col, w_col = M.moe_mxfp4_quant(x, rows=False, cols=True)[2:], M.moe_mxfp4_quant(w, rows=False, cols=True)[2:]
    dx, dw = M.moe_mxfp4_linear_bwd(dy, x_col, w_col, dx_dtype=dtype)
    xv, wv = R.quantised_values(x.t()), R.quantised_values(w.t())        # [k, m], [k, n]
    ref, mass = R.product(R.quantised_values(dy), wv)
    assert ((dx.cpu().double() - ref).abs() <= R.product_bound(ref, mass, n, dtype)).all()
    ref, mass = R.product(R.quantised_values(dy.t()), xv)
    bound = R.product_bound(ref, mass, m, F32)
    assert ((dw.cpu().double() - ref).abs() <= bound).all()
    assert dx.dtype == dtype and dw.dtype == F32
    only, none = M.moe_mxfp4_linear_bwd(dy, w_col=w_col, dx_dtype=dtype)
    assert torch.equal(only, dx) and none is None
    none, only = M.moe_mxfp4_linear_bwd(dy, x_col=x_col)
    assert torch.equal(only, dw) and none is None
    twice = dw.clone()
    M.moe_mxfp4_linear_bwd(dy, x_col=x_col, dw=twice, accumulate=True)
    assert ((twice.cpu().double() - 2 * ref).abs() <= 2 * bound + 2.0 ** -23 * 2 * mass).all()


def test_linear_bwd_against_differences(M):
    """L(x, w) = sum dy * (x w^T) with x, w and dy on the MXFP4 grid along
    both axes (every value +-1, +-2 or 0, every group's largest 4), so that no
    quantisation rounds: one element moved by h changes L by h * gradient."""
    m, n, k = 96, 64, 128
    g = torch.Generator().manual_seed(3)

    def grid(r, c):
        v = torch.randint(-2, 3, (r, c), generator=g).float()
        v[torch.arange(r), torch.arange(r) % 32 % c] = 4      # row groups; columns follow below
        for lo in range(0, c, 32):
            v[torch.arange(r), lo + torch.arange(r) % min(32, c - lo)] = 4
        return v

    x, w, dy = grid(m, k), grid(n, k), grid(m, n)
    for v in (x, w, dy):
        assert torch.equal(R.quantised_values(v), v.double()) and torch.equal(R.quantised_values(v.t()), v.t().double())
    q = lambda v: M.moe_mxfp4_quant(v.cuda(), rows=True, cols=True)
    dx, dw = M.moe_mxfp4_linear_bwd(dy.cuda(), q(x)[2:], q(w)[2:], dx_dtype=F32)

    def loss(xx, ww):
        y = M.moe_mxfp4_matmul(*q(xx)[:2], *q(ww)[:2], out_dtype=F32).cpu().double()
        return (y * dy.double()).sum().item()

    for i, j in ((0, 5), (17, 100), (95, 127)):
        for mat, grad, which in ((x, dx, 0), (w, dw, 1)):
            i = min(i, mat.shape[0] - 1)
            old = mat[i, j].item()
            new = 2.0 if old in (-2.0, 0.0, 1.0, 4.0) else -2.0
            if old == 4.0:
                continue
            moved = mat.clone()
            moved[i, j] = new
            diff = loss(moved, w) - loss(x, w) if which == 0 else loss(x, moved) - loss(x, w)
            assert diff == (new - old) * grad[i, j].item()


def test_products_past_32_bit_offsets(M):
    """Rows whose element offset passes 2^32, in the input and the output."""
    rows, ld = 70000, 65536
    big = torch.empty(rows, ld, dtype=BF16, device="cuda")
    x = big[:, 65000:65200]
    x.copy_(torch.randn(rows, 200, device="cuda"))
    q, s, _, _ = M.moe_mxfp4_quant(x)
    code, b = R.quantise(x[-100:])
    assert torch.equal(q[-100:].cpu(), R.pack(code)) and torch.equal(s[-100:].cpu().long(), b)
    w, sw, wv = _operand(136, 200, 1)
    out = big[:, 1000:1136]
    M.moe_mxfp4_matmul(q, s, w, sw, out=out)
    ref, mass = R.product(R.values(code, b), wv)
    assert ((out[-100:].cpu().double() - ref).abs() <= R.product_bound(ref, mass, 200, BF16)).all()
    M.moe_mxfp4_dequant(q, s, 200, out=big[:, 2000:2200])
    assert torch.equal(big[-100:, 2000:2200].cpu().double(), R.values(code, b)[:, :200])


@pytest.mark.parametrize("m,n,k", [(2000, 2050, 1100), (3300, 3900, 600), (1000, 1000, 700), (4097, 4100, 520), (8100, 8100, 520)])
def test_repeated_runs_give_the_same_bits(M, m, n, k):
    """Many runs one behind the other: a load that overtook a read of what it
    writes over would show in some of them."""
    a, sa, _ = _operand(m, k, 1)
    b, sb, _ = _operand(n, k, 2)
    want = M.moe_mxfp4_matmul(a, sa, b, sb, out_dtype=F32)
    outs = [torch.empty_like(want) for _ in range(10)]
    for _ in range(10):
        for o in outs:
            M.moe_mxfp4_matmul(a, sa, b, sb, out=o)
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("k", [400, 512, 600, 700, 900, 1100, 1200, 1700, 2048])
def test_several_tiles_per_workgroup(M, k):
    """More large tiles than compute units, whole and ragged ones, at lengths
    that end anywhere in a group of four blocks: the same bits as products of
    parts, which go through other tiles in the same order."""
    m, n = 8100, 8100
    a, sa, _ = _operand(m, k, 1)
    b, sb, _ = _operand(n, k, 2)
    for dtype in (BF16, F32):
        out = torch.full((m, n + 4), 3.0, dtype=dtype, device="cuda")
        M.moe_mxfp4_matmul(a, sa, b, sb, out=out[:, :n])
        parts = [M.moe_mxfp4_matmul(a[i:i + 700], sa[i:i + 700], b, sb, out_dtype=dtype) for i in range(0, m, 700)]
        assert torch.equal(out[:, :n], torch.cat(parts)) and (out[:, n:] == 3.0).all()
    before = out.clone()
    M.moe_mxfp4_matmul(a, sa, b, sb, out=out[:, :n], accumulate=True)
    # fp32: the sum, rounded, added and rounded once more; of a sum with itself both are exact
    assert torch.equal(out[:, :n], 2 * before[:, :n]) and (out[:, n:] == 3.0).all()


@pytest.mark.parametrize("rows,k,n", [(1 << 24, 40, 33), (1 << 24, 520, 40), (70, 520, 1 << 24), (5, 130, 1 << 24), (66000, 512, 66000)])
def test_largest_sides(M, rows, k, n):
    """Sides of 2^24, and results past 2^32 elements: the first, some in the
    middle and the last rows and columns as in products of those alone."""
    def codes(r, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        kp = (k + 127) // 128 * 128
        q = torch.randint(0, 256, (r, kp // 2), generator=g, device="cuda", dtype=torch.uint8)
        q[:, k // 2:] = 0
        return q, torch.randint(118, 130, (r, kp // 32), generator=g, device="cuda", dtype=torch.uint8)

    (a, sa), (b, sb) = codes(rows, 1), codes(n, 2)
    out = M.moe_mxfp4_matmul(a, sa, b, sb)
    pick = lambda size: [slice(i, min(i + 70, size)) for i in ({0, size // 2 - 3, size - 70} if size > 200 else {0})]
    for i in pick(rows):
        for j in pick(n):
            want = M.moe_mxfp4_matmul(a[i].contiguous(), sa[i].contiguous(), b[j].contiguous(), sb[j].contiguous(), out_dtype=F32)
            got = out[i, j].float()
            # bf16 of the same sum, in an order of its own perhaps: half a step, and K roundings of the terms' size (<= 36 * 2^4 each)
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + k * k * 36 * 16 * 2.0 ** -24).all()
    del out, a, sa, b, sb
    torch.cuda.empty_cache()


def test_longest_sums(M):
    """K = 2^24, the longest: ones times ones with a power of two per row, sums
    that fp32 holds exactly; row offsets of up to 2 GB."""
    K = 1 << 24
    for m, n in ((260, 40), (3, 33)):
        one = lambda rows: torch.full((rows, K // 2), 0x22, dtype=torch.uint8, device="cuda")   # 1.0, 1.0
        sc = lambda rows: (120 + torch.arange(rows, device="cuda") % 9).to(torch.uint8)[:, None].expand(rows, K // 32).contiguous()
        sa, sb = sc(m), sc(n)
        out = M.moe_mxfp4_matmul(one(m), sa, one(n), sb, out_dtype=F32)
        want = float(K) * torch.exp2(sa[:, :1].float() - 127) * torch.exp2(sb[:, 0].float() - 127)
        assert torch.equal(out, want)


def test_two_streams_at_once(M):
    """The same products on two streams together, each with its own scratch."""
    a, sa, _ = _operand(100, 4096, 1)
    b, sb, _ = _operand(288, 4096, 2)
    x = _matrix(40, 4096, BF16, 3).cuda()
    want = M.moe_mxfp4_matmul(a, sa, b, sb), M.moe_mxfp4_linear(x, b, sb)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            got.append((M.moe_mxfp4_matmul(a, sa, b, sb, stream=s), M.moe_mxfp4_linear(x, b, sb, stream=s)))
    for s in streams:
        s.synchronize()
    assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))


def test_other_stream_and_graph(M):
    """On a stream of its own, and captured (its backward too) and replayed on
    new inputs with eager calls in between."""
    x, n = _matrix(40, 1000, BF16, 1).cuda(), 500
    w = _matrix(n, 1000, F32, 2).cuda()
    wq, wsc, wc, wcs = M.moe_mxfp4_quant(w, rows=True, cols=True)
    eager = M.moe_mxfp4_linear(x, wq, wsc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = M.moe_mxfp4_linear(x, wq, wsc, stream=side)
    y2 = M.moe_mxfp4_linear(x, wq, wsc, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, eager) and torch.equal(y2, eager)

    def step(xx):
        q = M.moe_mxfp4_quant(xx, rows=True, cols=True)
        out = M.moe_mxfp4_matmul(*q[:2], wq, wsc, out_dtype=F32)
        dx, dw = M.moe_mxfp4_linear_bwd(out, q[2:], (wc, wcs))
        return out, M.moe_mxfp4_linear(xx, wq, wsc), M.moe_mxfp4_linear(xx[:3], wq, wsc), dx, dw

    static = x.clone()
    with torch.cuda.stream(side):
        step(static)
    side.synchronize()
    graphs = []
    for _ in range(2):                          # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(static)
        graphs.append((graph, outs))
    for i in range(4):
        static.copy_(_matrix(40, 1000, BF16, 50 + i))
        want = step(static)
        for graph, outs in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
