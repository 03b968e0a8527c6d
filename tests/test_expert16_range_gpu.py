"""The 16-bit expert operators over the whole range of their types: small and
large values whose squares, products or exponentials leave fp32's range or
precision on the way although the result does not.  Against 64-bit formulas."""
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("F", [64, 1032])
def test_routing_weight_gradient_has_fp32_precision(M, F, dtype):
    """drow_w for rows of one gate value each, from -86 to 20: every term of a
    row has the same error of its exponential, which nothing averages out.

    Roundings in units of 2^-24 of a term: exponential 4 (2 ulp), 1 + t 1, reciprocal
    4, t / (1 + t) 1, a s 1, dh and up 2; the sums add F / 8 + 8 of the sum of the terms
    (at most F / 32 chunks a thread with 5 additions each, then 8 steps)."""
    a = torch.arange(-86, 20.25, 0.25).to(dtype)
    R = a.numel()
    g = torch.Generator().manual_seed(1)
    gu = torch.cat([a[:, None].expand(R, F), (torch.rand(R, F, generator=g) + 0.5).to(dtype)], 1).contiguous()
    dh, w = (torch.rand(R, F, generator=g) + 0.5).to(dtype), torch.ones(R)
    _, got = M.swiglu_backward(dh.cuda(), gu.cuda(), w.cuda())
    ad = a.double()
    ref = (ad / (1 + torch.exp(-ad))) * (dh.double() * gu[:, F:].double()).sum(1)
    tol = (16 + F / 8 + 8) * 2.0 ** -24 * ref.abs()
    err = (got.cpu().double() - ref).abs()
    assert (err <= tol).all(), (err / tol.clamp_min(1e-300)).max().item()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("weights", [False, True])
def test_closed_gate_beside_factors_whose_product_overflows(M, weights, dtype):
    """A gate so low that SiLU and its slope are 0 in 64 bits gives zeros for any
    finite up, dh and weight, although their products leave fp32's range."""
    R, F = 5, 72
    low = torch.finfo(dtype).min
    gu = torch.full((R, 2 * F), 2.0e38).to(dtype)
    gu[:, :F] = low
    gu[1, :F] = -1000.0
    dh = torch.full((R, F), -1.0e38).to(dtype)
    w = torch.full((R,), 64.0).cuda() if weights else None
    h = M.swiglu(gu.cuda(), w)
    dgu, drow = M.swiglu_backward(dh.cuda(), gu.cuda(), w)
    for t in (h, dgu) + ((drow,) if weights else ()):
        assert torch.isfinite(t).all() and not t.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_that_brings_a_large_product_back(M, dtype):
    """up times weight, and dh times up, are beyond fp32; with SiLU's factor the
    results are not.  One rounding to the type and at most 32 of 2^-24, the
    exponential's among them (2^-16 where it is the hardware's, for bf16 outputs)."""
    R, F = 3, 64
    a = torch.tensor([-60.0, -30.0, -8.0]).to(dtype)
    up, w = torch.full((R, F), 2.0e38).to(dtype), torch.tensor([64.0, 16.0, 4.0])
    d = torch.tensor([-1e8, 1e3, 4.0])[:, None].expand(R, F).to(dtype)
    gu = torch.cat([a[:, None].expand(R, F), up], 1).contiguous()
    A, U, D, W = a.double()[:, None], up.double(), d.double(), w.double()[:, None]
    s = 1 / (1 + torch.exp(-A))
    h = M.swiglu(gu.cuda(), w.cuda())
    dgu, drow = M.swiglu_backward(d.contiguous().cuda(), gu.cuda(), w.cuda())
    small = 32 * 2.0 ** -24 + (2.0 ** -16 if dtype is BF16 else 0)
    u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -24
    ref = [W * A * s * U, torch.cat([W * D * U * s * (1 + A * (1 - s)), W * D * A * s], 1), (D * A * s * U).sum(1)]
    for got, r, tol in ((h, ref[0], u + small), (dgu, ref[1], u + small + 64 * 2.0 ** -24),
                        (drow, ref[2], (32 + F / 8) * 2.0 ** -24)):
        assert r.abs().max() < 3e38
        assert ((got.double().cpu() - r).abs() <= tol * r.abs()).all()


# ----------------------------------------------------------------- block norms
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def within(got, ref, terms, steps, what):
    """One rounding to the type, `steps` of 2^-24 of the terms, half a subnormal."""
    got = got.cpu().double()
    tol = U[BF16 if what[1] is BF16 else F32] * ref.abs() + steps * 2.0 ** -24 * terms + 2.0 ** -134
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def wide_rows(T, D, dtype):
    """x and y of ordinary rows and, in turn, of rows whose squares, or products
    of two tensors, are beyond fp32."""
    x, y = randn(1, T, D), randn(2, T, D)
    low = torch.finfo(dtype).min
    for r in range(T):
        kind = r % 8
        if kind == 1:
            y[r] = low / 4 if r % 16 == 1 else low  # one value, the type's lowest
        elif kind == 2:
            y[r] *= 1e30
        elif kind == 3:
            x[r] *= 1e30
        elif kind == 4:
            x[r] *= 1e25
            y[r] *= 1e33
        elif kind == 5:
            x[r] *= 1e17
            y[r] *= 1e17
        elif kind == 6:
            x[r] = low
        # kinds 0 and 7 stay
    return x.to(dtype), y.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(9, 512), (700, 512), (25, 4104), (330, 4104), (330, 8200)])
@pytest.mark.parametrize("alpha,gates", [(0.75, 1), (1e-3, 1), (1e19, 1), (0.75, 0)])
def test_norms_of_rows_whose_squares_leave_fp32(M, T, D, alpha, gates, dtype):
    eps = 1e-6
    x, y = wide_rows(T, D, dtype)
    post, pre = 1 + 0.2 * randn(3, D), 1 + 0.2 * randn(4, D)
    gate = 0.5 + randn(5, 1, D).abs().clamp_max(2) if gates else None
    xd, yd = x.double(), y.double()
    n = alpha * (gate.double() if gates else 1.0) * yd / ((yd * yd).mean(1, keepdim=True) + eps).sqrt() * post.double()
    xo, terms = xd + n, xd.abs() + n.abs()
    h = xo / ((xo * xo).mean(1, keepdim=True) + eps).sqrt() * pre.double()
    limit = torch.finfo(dtype).max
    fits = (xo.abs() <= limit).all(1)  # x at the lowest value and n of the same sign
    assert fits.sum() > T // 2
    got_x, got_h = M.block_norm(x.cuda(), y.cuda(), post.cuda(), gate.cuda() if gates else None, pre.cuda(), alpha, eps)
    within(got_x[fits.cuda()], xo[fits], terms[fits], 64, ("x_out", dtype))
    within(got_h[fits.cuda()], h[fits], (h.abs() * (1 + terms / xo.abs().clamp_min(1e-300)))[fits], 64, ("h", dtype))
    alone = M.block_norm(x.cuda(), gamma_pre=pre.cuda(), eps=eps)[1]
    ref = xd / ((xd * xd).mean(1, keepdim=True) + eps).sqrt() * pre.double()
    within(alone, ref, 2 * ref.abs(), 64, ("h of x", dtype))


def test_norms_keep_infinities_and_nans_in_their_rows(M):
    x, y = randn(1, 40, 264), randn(2, 40, 264)
    p = torch.ones(264).cuda()
    want = M.block_norm(x.cuda(), y.cuda(), p, None, p)
    x2, y2 = x.clone(), y.clone()
    x2[3, 5], y2[7, 0], y2[9, 100] = float("inf"), float("nan"), float("-inf")
    got = M.block_norm(x2.cuda(), y2.cuda(), p, None, p)
    rest = [r for r in range(40) if r not in (3, 7, 9)]
    assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][rest], want[1][rest])
    assert all(not torch.isfinite(got[1][r]).all() for r in (3, 7, 9))


def norm_gradients(x, y, dxo, dh, post, gate, pre, alpha, eps):
    """The gradients in 64 bits and the sums of absolute terms of each."""
    x, y, dxo, dh = (t.double() for t in (x, y, dxo, dh))
    post, pre, a = post.double(), pre.double(), alpha * gate.double()
    r1 = ((y * y).mean(1, keepdim=True) + eps).rsqrt()
    r2 = ((x * x).mean(1, keepdim=True) + eps).rsqrt()
    v, xn, yn = dh * pre, x * r2, y * r1
    d = dxo + r2 * v - r2 * xn * (v * xn).mean(1, keepdim=True)
    da = dxo.abs() + (r2 * v).abs() + (r2 * xn).abs() * (v * xn).abs().mean(1, keepdim=True)
    q, qa = a * post * d, (a * post).abs() * da
    dy = r1 * q - r1 * yn * (q * yn).mean(1, keepdim=True)
    dya = r1 * qa + (r1 * yn).abs() * (qa * yn.abs()).mean(1, keepdim=True)
    tp, tg, tq = a * d * yn, alpha * post * d * yn, dh * xn
    ta, ga = (a * yn).abs() * da, (alpha * post * yn).abs() * da
    return {"dx": (d, da), "dy": (dy, dya), "dgamma_post": (tp.sum(0), ta.sum(0)),
            "dgate": (tg.sum(0, keepdim=True), ga.sum(0, keepdim=True)), "dgamma_pre": (tq.sum(0), tq.abs().sum(0))}


def check_norm_gradients(M, x, y, dxo, dh, eps, alpha=0.75):
    D = x.shape[1]
    post, pre, gate = 1 + 0.2 * randn(13, D), 1 + 0.2 * randn(14, D), 0.5 + randn(15, 1, D).abs().clamp_max(2)
    ref = norm_gradients(x, y, dxo, dh, post, gate, pre, alpha, eps)
    cu = lambda t: t.cuda()
    got = M.block_norm_backward(cu(x), cu(y), cu(dxo), cu(dh), cu(post), cu(gate), cu(pre), alpha, eps)
    for (name, (r, terms)), g in zip(ref.items(), got):
        rows = x.shape[0] if name.startswith("dg") else 0
        # dgamma and dgate are fp32 whatever the rows are
        within(g, r, terms, 64 + rows, (name, x.dtype if name in ("dx", "dy") else F32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(7, 264), (700, 512), (330, 4104), (9, 8200)])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_norm_gradients_of_small_rows(M, T, D, eps, dtype):
    """1 / rms cubed is beyond fp32 where a row is zero beside a small eps."""
    x, y = randn(1, T, D), randn(2, T, D)
    for r in range(T):
        x[r] *= [1.0, 0.0, 0.0, 1e-12, 1e-10][r % 5]
        y[r] *= [1.0, 0.0, 1.0, 1e-11, 1e-12][r % 5]
    dh, dxo = randn(3, T, D), randn(4, T, D)
    dxo[1::2] = 0  # what comes through the norm is not hidden behind dx_out
    check_norm_gradients(M, x.to(dtype), y.to(dtype), dxo.to(dtype), dh.to(dtype), eps)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(17, 264), (700, 512), (330, 4104), (18, 8200)])
@pytest.mark.parametrize("gates", [1, "many"])
def test_norm_gradients_of_large_rows(M, T, D, gates, dtype):
    """Rows whose squares, or whose gradients over squares, are beyond fp32."""
    x, y = randn(1, T, D), randn(2, T, D)
    scale = [1.0, 1e13, 1e15, 1e17, 1e19, 1e25, 1e33, 1e5]
    for r in range(T):
        x[r] *= scale[r % 8]
        y[r] *= scale[(r + r // 8) % 8]
    low = torch.finfo(dtype).min
    x[3], y[5], x[7], y[7] = low, low, low, low / 2
    dh, dxo = randn(3, T, D), randn(4, T, D)
    dxo[1::2] = 0
    x, y, dh, dxo = (t.to(dtype) for t in (x, y, dh, dxo))
    if gates == 1:
        check_norm_gradients(M, x, y, dxo, dh, 1e-6)
        return
    # gate by gate
    G = {17: 17, 700: 7, 330: 110, 18: 2}[T]
    post, pre, gate = 1 + 0.2 * randn(13, D), 1 + 0.2 * randn(14, D), 0.5 + randn(15, G, D).abs().clamp_max(2)
    cu = lambda t: t.cuda()
    dx, dy, _, dgate, _ = M.block_norm_backward(cu(x), cu(y), cu(dxo), cu(dh), cu(post), cu(gate), cu(pre), 0.75, 1e-6)
    S = T // G
    for g in (0, G // 2, G - 1):
        s = slice(g * S, (g + 1) * S)
        ref = norm_gradients(x[s], y[s], dxo[s], dh[s], post, gate[g:g + 1], pre, 0.75, 1e-6)
        within(dx[s], *ref["dx"], 64, ("dx", dtype))
        within(dy[s], *ref["dy"], 64, ("dy", dtype))
        within(dgate[g:g + 1], *ref["dgate"], 64 + S, ("dgate", F32))
