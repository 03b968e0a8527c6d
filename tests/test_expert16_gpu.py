"""The 16-bit expert operators on the GPU against plain 64-bit formulas.

Tolerances.  An output rounded once to its type is off by at most u |ref|, with
u = 2^-8 for bf16 (8 significant bits, round to nearest), 2^-11 for fp16 and
2^-24 for fp32; among the subnormals it is off by half their spacing, 2^-134,
2^-25 and 2^-150.  What is computed in fp32 before that adds:
  - a product summed over L terms: the tensor cores add 16 products to the
    fp32 accumulator at a time, each time off by at most 2^-23 of the largest
    partial sum, which sum |a b| bounds: L / 16 steps, taken twice over for the
    order of the sums, and 16 more: (L / 8 + 16) 2^-23 sum |a b|;
  - the elementwise operators: at most 64 rounded operations of 2^-24 each,
    relative to the sum of the absolute values of the terms;
  - sums over rows: one more 2^-24 for each row.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES16 = [torch.bfloat16, torch.float16]
ALL = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def randn(seed, dtype, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def close(got, ref, terms, steps, what):
    """|got - ref| <= u |ref| + steps 2^-24 terms, element by element."""
    ref = ref.double()
    tol = U[got.dtype] * ref.abs() + steps * 2.0 ** -24 * terms.double() + SUBNORMAL[got.dtype]
    err = (got.detach().cpu().double() - ref).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, (what, worst, err.max().item())


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


# ------------------------------------------------------------ grouped products
def mm_steps(length):
    return 2 * (length / 8 + 16)


def grouped_reference(x, w, dy, counts):
    """y, dx, dw and the sums of absolute terms of each, in 64 bits."""
    x, w, dy = x.double(), w.double(), dy.double()
    R, K = x.shape
    E, N, _ = w.shape
    out = [torch.zeros(s, dtype=torch.float64) for s in ((R, N), (R, K), (E, N, K)) for _ in (0, 1)]
    r = 0
    for e, c in enumerate(counts):
        s = slice(r, r + c)
        out[0][s], out[1][s] = x[s] @ w[e].T, x[s].abs() @ w[e].abs().T
        out[2][s], out[3][s] = dy[s] @ w[e], dy[s].abs() @ w[e].abs()
        out[4][e], out[5][e] = dy[s].T @ x[s], dy[s].abs().T @ x[s].abs()
        r += c
    return out


GROUPED = [
    # counts of the segments, N, K
    ([1], 8, 8),
    ([0, 1, 0], 16, 64),
    ([0, 0], 64, 64),                         # no rows at all
    ([3, 0, 5], 72, 40),
    ([1] * 8, 256, 512),                      # one token's experts
    ([1, 2, 0, 7, 1], 768, 264),
    ([64], 136, 128),
    ([9, 55, 0, 0, 1, 8], 1536, 256),         # few rows, several of one expert
    ([65, 63, 64, 0, 1], 264, 72),
    ([255, 1, 256, 257, 0, 31], 328, 200),    # around one and two tiles of rows
    ([513, 16, 0, 15, 17], 520, 1032),
    ([1000], 2048, 64),
    ([33] * 40, 64, 2048),
    ([2, 120, 0, 700, 5, 48, 130, 1], 128, 768),
    ([1, 0, 2, 1] * 24, 520, 1096),           # about one row an expert, widths of 8
    ([2331], 264, 200),                       # one long segment, few tiles
    ([40, 33, 0, 50], 1048, 104),
]


@pytest.mark.parametrize("dtype", DTYPES16)
@pytest.mark.parametrize("counts,N,K", GROUPED)
def test_grouped_products(M, counts, N, K, dtype):
    R, E = sum(counts), len(counts)
    x, dy = randn(1, dtype, R, K), randn(2, dtype, R, N, scale=0.5)
    w = randn(3, dtype, E, N, K, scale=K ** -0.5)
    y, ya, dx, dxa, dw, dwa = grouped_reference(x, w, dy, counts)
    off = offsets_of(counts).cuda()
    xd, wd, dyd = x.cuda(), w.cuda(), dy.cuda()
    ws = M.workspace(M.grouped_mm_workspace_size(R, E, N, K))
    close(M.grouped_mm(xd, wd, off, ws=ws), y, ya, mm_steps(K), "y")
    close(M.grouped_mm_dx(dyd, wd, off, ws=ws), dx, dxa, mm_steps(N), "dx")
    got = M.grouped_mm_dw(dyd, xd, off, ws=ws)
    close(got, dw, dwa, mm_steps(max(counts)), "dw")
    for e, c in enumerate(counts):
        if c == 0:
            assert not got[e].any()
    assert M.get_device_error(ws) == M.MOE_OK


@pytest.mark.parametrize("dtype", DTYPES16)
@pytest.mark.parametrize("counts,N,K", [
    ([70], 88, 2072),              # shares of the summed index: of y,
    ([100, 0, 37], 232, 4104),
    ([40], 2056, 136),             # of dx,
    ([2100], 96, 80),              # of dw
    ([6001, 0, 1], 104, 136),      # whose second and third segment have less rows than shares
    ([17, 4080], 40, 264),
    ([60, 59], 2056, 2064),        # of y and dx
])
def test_grouped_products_of_few_tiles(M, counts, N, K, dtype):
    """Few tiles with a long summed index are shared out and added up."""
    R, E = sum(counts), len(counts)
    assert M.grouped_mm_workspace_size(R, E, N, K) > 256
    test_grouped_products(M, counts, N, K, dtype)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_grouped_products_of_few_tiles_keep_segments_apart(M, bad):
    """Shares of one expert's sums see nothing of another's rows and weights;
    bit for bit the same again, and in a graph; bad offsets are reported."""
    counts, N, K = [2101, 2051], 96, 80
    x, dy = randn(1, torch.bfloat16, sum(counts), K).cuda(), randn(2, torch.bfloat16, sum(counts), N).cuda()
    off = offsets_of(counts).cuda()
    ws = M.workspace(M.grouped_mm_workspace_size(sum(counts), 2, N, K))
    assert ws.numel() > 256
    want = M.grouped_mm_dw(dy, x, off, ws=ws)
    assert torch.equal(M.grouped_mm_dw(dy, x, off, ws=ws), want)
    for e, s in ((0, slice(0, counts[0])), (1, slice(counts[0], None))):
        x2, dy2 = torch.full_like(x, bad), torch.full_like(dy, bad)
        x2[s], dy2[s] = x[s], dy[s]
        assert torch.equal(M.grouped_mm_dw(dy2, x2, off, ws=ws)[e], want[e])
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.grouped_mm_dw(dy, x, off, dw=out, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and M.get_device_error(ws) == M.MOE_OK
    M.grouped_mm_dw(dy, x, torch.tensor([0, 4153, 4152], dtype=torch.int32).cuda(), ws=ws)
    assert M.STATUS[M.get_device_error(ws)] == "MOE_ERR_DEVICE_RANGE"
    assert torch.equal(M.grouped_mm_dw(dy, x, off, ws=ws), want)


@pytest.mark.parametrize("dtype", DTYPES16)
@pytest.mark.parametrize("counts,N,K", [
    ([1, 0, 2], 72, 1096),
    ([7], 264, 4104),
    ([0, 9, 1, 1], 136, 2056),     # a second block of an expert's rows
    ([1] * 8, 512, 4096),
    ([3, 3], 3400, 1024),
    ([30], 1032, 72),
])
def test_grouped_products_of_few_rows(M, counts, N, K, dtype):
    """A handful of rows: K shared by 4, 8 or 16 warps."""
    test_grouped_products(M, counts, N, K, dtype)


def test_grouped_products_of_few_tiles_leave_other_rows(M):
    R, N, K = 150, 64, 4096
    x, w = randn(1, torch.bfloat16, R, K).cuda(), randn(2, torch.bfloat16, 2, N, K).cuda()
    off = torch.tensor([10, 80, 140], dtype=torch.int32).cuda()
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16).cuda()
    M.grouped_mm(x, w, off, y=y)
    ref = torch.cat([x[10:80].double() @ w[0].double().T, x[80:140].double() @ w[1].double().T]).cpu()
    terms = torch.cat([x[10:80].double().abs() @ w[0].double().abs().T, x[80:140].double().abs() @ w[1].double().abs().T]).cpu()
    assert (y[:10] == 7).all() and (y[140:] == 7).all()
    close(y[10:140], ref, terms, mm_steps(K), "y")


@pytest.mark.parametrize("dtype", DTYPES16)
def test_grouped_products_are_exact_on_small_integers_and_bilinear(M, dtype):
    """Small whole numbers: every product, sum and rounding is exact, so the
    results equal the definition's, and the gradients equal the differences of
    the bilinear form <dy, y(x, w)> in single entries of x and w."""
    g = torch.Generator().manual_seed(5)
    counts, N, K = [3, 0, 17, 4], 24, 40
    R, E = sum(counts), len(counts)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).to(dtype).cuda()
    x, w, dy, off = whole(R, K), whole(E, N, K), whole(R, N), offsets_of(counts).cuda()

    def form(x, w):
        return (M.grouped_mm(x, w, off).double() * dy.double()).sum().item()

    dx, dw = M.grouped_mm_dx(dy, w, off), M.grouped_mm_dw(dy, x, off)
    base = form(x, w)
    for r, k in ((0, 0), (2, 39), (3, 7), (19, 8), (23, 39)):
        x2 = x.clone()
        x2[r, k] += 1
        assert form(x2, w) - base == dx[r, k].item()
    for e, n, k in ((0, 0, 0), (0, 23, 39), (1, 3, 3), (2, 8, 16), (3, 23, 0)):
        w2 = w.clone()
        w2[e, n, k] += 1
        assert form(x, w2) - base == dw[e, n, k].item()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_grouped_products_keep_segments_apart(M, bad):
    """Rows and weights of other experts, and what stands behind the last
    segment, never reach a result, not even as 0 * NaN."""
    dtype, counts, N, K = torch.bfloat16, [5, 40, 0, 21, 300], 136, 72
    R, E = sum(counts), len(counts)
    x, dy = randn(1, dtype, R + 64, K), randn(2, dtype, R + 64, N)
    w = randn(3, dtype, E, N, K)
    ref = grouped_reference(x[:R], w, dy[:R], counts)
    off = offsets_of(counts)
    for e in (0, 1, 3, 4):
        x2, w2, dy2 = (torch.full_like(t, bad) for t in (x, w, dy))
        s = slice(off[e], off[e + 1])
        x2[s], dy2[s], w2[e] = x[s], dy[s], w[e]
        xd, wd, dyd, od = x2.cuda()[:R], w2.cuda(), dy2.cuda()[:R], off.cuda()
        close(M.grouped_mm(xd, wd, od)[s], ref[0][s], ref[1][s], mm_steps(K), "y")
        close(M.grouped_mm_dx(dyd, wd, od)[s], ref[2][s], ref[3][s], mm_steps(N), "dx")
        got = M.grouped_mm_dw(dyd, xd, od)
        close(got[e], ref[4][e], ref[5][e], mm_steps(counts[e]), "dw")
        assert not got[2].any()


def test_grouped_products_report_bad_offsets(M):
    """A segment outside the rows counts as empty and sets the error word."""
    dtype, N, K, R, E = torch.bfloat16, 64, 64, 40, 4
    x, dy, w = randn(1, dtype, R, K).cuda(), randn(2, dtype, R, N).cuda(), randn(3, dtype, E, N, K).cuda()
    for off in ([0, 10, 5, 20, 40], [0, 10, 20, 30, 41], [-1, 10, 20, 30, 40], [0, 10, 20, 2 ** 30, 40]):
        od = torch.tensor(off, dtype=torch.int32).cuda()
        ws = M.workspace(M.grouped_mm_workspace_size(R, E, N, K))
        for call in (lambda: M.grouped_mm(x, w, od, ws=ws), lambda: M.grouped_mm_dx(dy, w, od, ws=ws),
                     lambda: M.grouped_mm_dw(dy, x, od, ws=ws)):
            call()
            assert M.STATUS[M.get_device_error(ws)] == "MOE_ERR_DEVICE_RANGE"
            assert M.get_device_error(ws) == M.MOE_OK  # cleared


def test_grouped_products_with_weights_past_32_bits(M):
    """More than 2^31 weights: the last expert's products and gradient."""
    dtype, E, N, K = torch.bfloat16, 130, 4096, 4104
    counts = [0] * (E - 1) + [70]
    x, dy, w1 = randn(1, dtype, 70, K), randn(2, dtype, 70, N), randn(3, dtype, 1, N, K, scale=0.02)
    w = torch.zeros(E, N, K, dtype=dtype, device="cuda")
    w[-1] = w1[0].cuda()
    ref = grouped_reference(x, w1, dy, [70])
    off = offsets_of(counts).cuda()
    close(M.grouped_mm(x.cuda(), w, off), ref[0], ref[1], mm_steps(K), "y")
    close(M.grouped_mm_dx(dy.cuda(), w, off), ref[2], ref[3], mm_steps(N), "dx")
    w.fill_(1)
    M.grouped_mm_dw(dy.cuda(), x.cuda(), off, dw=w)
    close(w[-1], ref[4][0], ref[5][0], mm_steps(70), "dw")
    assert not w[:-1].any()


def test_grouped_products_repeat_bit_for_bit_on_streams_and_graphs(M):
    dtype, counts, N, K = torch.float16, [7, 0, 130, 64, 1], 512, 640
    R, E = sum(counts), len(counts)
    x, dy, w = randn(1, dtype, R, K).cuda(), randn(2, dtype, R, N).cuda(), randn(3, dtype, E, N, K).cuda()
    off = offsets_of(counts).cuda()
    ws = M.workspace(M.grouped_mm_workspace_size(R, E, N, K))
    first = [M.grouped_mm(x, w, off, ws=ws), M.grouped_mm_dx(dy, w, off, ws=ws), M.grouped_mm_dw(dy, x, off, ws=ws)]
    out = [torch.full_like(t, 3) for t in first]

    def calls(stream=None):
        M.grouped_mm(x, w, off, y=out[0], ws=ws, stream=stream)
        M.grouped_mm_dx(dy, w, off, dx=out[1], ws=ws, stream=stream)
        M.grouped_mm_dw(dy, x, off, dw=out[2], ws=ws, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # back to back on one workspace
        calls(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            calls()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    assert M.get_device_error(ws) == M.MOE_OK


# ------------------------------------------------------------ gated activation
def swiglu_reference(gu, dh, row_w, row_map):
    R, F = dh.shape
    a, u, d = gu.double()[:, :F], gu.double()[:, F:], dh.double()
    w = torch.ones(R, 1, dtype=torch.float64) if row_w is None else row_w.double()[row_map.long()][:, None]
    s = 1 / (1 + torch.exp(-a))
    h = w * a * s * u
    da, daa = w * d * u * s * (1 + a * (1 - s)), (w * d * u * s).abs() * (1 + a.abs())
    du = w * d * a * s
    terms = d * a * s * u
    return h, torch.cat([da, du], 1), torch.cat([daa, du.abs()], 1), terms.sum(1), terms.abs().sum(1)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("R,F", [(1, 8), (8, 768), (3, 264), (129, 1024), (77, 1032), (5, 4096), (300, 72), (2, 16384)])
@pytest.mark.parametrize("weights", ["none", "identity", "map"])
def test_swiglu(M, R, F, dtype, weights):
    gu, dh = randn(1, dtype, R, 2 * F, scale=2.0), randn(2, dtype, R, F)
    gu[0, :4] = torch.tensor([100.0, -100.0, 0.0, -20.0])  # both ends of the sigmoid
    row_w = None if weights == "none" else torch.rand(R, generator=torch.Generator().manual_seed(3))
    row_map = torch.randperm(R, generator=torch.Generator().manual_seed(4)).int() if weights == "map" else torch.arange(R).int()
    h, dgu, dgua, dw, dwa = swiglu_reference(gu, dh, row_w, row_map)
    wd = row_w.cuda() if row_w is not None else None
    md = row_map.cuda() if weights == "map" else None
    close(M.swiglu(gu.cuda(), wd, md), h, h.abs(), 64, "h")
    got, got_w = M.swiglu_backward(dh.cuda(), gu.cuda(), wd, md)
    close(got, dgu, dgua, 64, "dgu")
    if row_w is None:
        assert got_w is None
    else:
        close(got_w.cpu()[row_map.long()], dw, dwa, 64 + F / 8, "drow_w")
    again = gu.cuda()
    M.swiglu_backward(dh.cuda(), again, wd, md, dgu=again)  # in place
    assert torch.equal(again, got)


def test_swiglu_gradient_against_differences(M):
    """Derivative of <dh, h> along the signs of its gradient, where it is
    largest, by central differences.  With step d
    the cut-off error is below d^2 / 6 times the third derivative along the
    direction (|SiLU'''| < 1.2, |values| < 4: below 40 for each entry), and the
    rounding of fp32 outputs adds 2^-24 |h| / d for each."""
    R, F, d = 6, 64, 2.0 ** -8
    gu, dh = randn(1, torch.float32, R, 2 * F), randn(2, torch.float32, R, F)
    row_w = torch.rand(R, generator=torch.Generator().manual_seed(3)) + 0.5
    dgu, dw = M.swiglu_backward(dh.cuda(), gu.cuda(), row_w.cuda())
    vg, vw = dgu.sign().cpu(), dw.sign().cpu()
    f = lambda t: (M.swiglu((gu + t * vg).cuda(), (row_w + t * vw).cuda()).cpu().double() * dh.double()).sum().item()
    want = (dgu.cpu().double() * vg.double()).sum().item() + (dw.cpu().double() * vw.double()).sum().item()
    n = R * F
    tol = n * (d * d / 6 * 40 + 64 * 2.0 ** -24 * 40 / d) * dh.abs().mean().item()
    assert abs((f(d) - f(-d)) / (2 * d) - want) <= tol
    assert abs(want) > 3 * tol  # the comparison says something


def test_swiglu_skips_entries_outside_the_map(M):
    R, F = 4, 64
    gu, dh = randn(1, torch.float32, R, 2 * F).cuda(), randn(2, torch.float32, R, F).cuda()
    row_w = torch.ones(R).cuda()
    row_map = torch.tensor([2, -1, 4, 0], dtype=torch.int32).cuda()
    h = M.swiglu(gu, row_w, row_map)
    ones = M.swiglu(gu)
    assert torch.equal(h[0], ones[0]) and torch.equal(h[3], ones[3]) and not h[1:3].any()
    drow = torch.full((R,), 7.0).cuda()
    dgu, _ = M.swiglu_backward(dh, gu, row_w, row_map, drow_w=drow)
    assert not dgu[1:3].any() and drow[1] == 7 and drow[3] == 7 and drow[0] != 7 and drow[2] != 7


@pytest.mark.parametrize("dtype", ALL)
def test_swiglu_of_the_lowest_gate(M, dtype):
    """SiLU and its slope at the type's lowest values are zero, whatever the
    other factors (nothing in between may overflow)."""
    R, F = 3, 64
    low = torch.finfo(dtype).min
    gu, dh = randn(1, dtype, R, 2 * F, scale=8.0), randn(2, dtype, R, F, scale=8.0)
    gu[:, :F:2] = low
    gu[:, 1:F:4] = low / 2
    row_w = torch.full((R,), 8.0)
    h = M.swiglu(gu.cuda(), row_w.cuda())
    dgu, drow = M.swiglu_backward(dh.cuda(), gu.cuda(), row_w.cuda())
    h, dgu = h.cpu(), dgu.cpu()
    rest = gu[:, :F] > low / 2
    for t in (h, dgu[:, :F], dgu[:, F:]):
        assert not t[~rest].any() and torch.isfinite(t.float()).all()
    # and they add nothing to the routing weight's gradient
    a, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    terms = torch.where(rest, d * a / (1 + torch.exp(-a)) * u, 0.0)
    close(drow.cpu(), terms.sum(1), terms.abs().sum(1), 64 + F / 8, "drow_w")


# ----------------------------------------------------------------- block norms
def norm_reference(x, y, dx_out, dh, post, gate, pre, alpha, eps):
    """Forward at (x, y), backward at (x as the stored stream, y); with the
    sums of absolute terms."""
    x = x.double()
    T, D = x.shape
    one = torch.ones(D, dtype=torch.float64)
    g = gate.double().repeat_interleave(T // gate.shape[0], 0) if gate is not None else torch.ones(T, D, dtype=torch.float64)
    po = post.double() if post is not None else one
    out = {}
    if y is not None:
        y = y.double()
        r1 = ((y * y).mean(1, keepdim=True) + eps).rsqrt() if post is not None else torch.ones(T, 1, dtype=torch.float64)
        n = y * r1 * po
        xo = x + alpha * g * n
        out["x_out"] = (xo, x.abs() + (alpha * g * n).abs())
    else:
        xo = x
    if pre is not None:
        pr = pre.double()
        h = xo * ((xo * xo).mean(1, keepdim=True) + eps).rsqrt() * pr
        grow = (out["x_out"][1] / xo.abs().clamp_min(1e-30)) if y is not None else 1.0
        out["h"] = (h, h.abs() * grow + h.abs())
    # backward
    d = dx_out.double() if dx_out is not None else torch.zeros(T, D, dtype=torch.float64)
    da = d.abs()
    if pre is not None:
        r2 = ((x * x).mean(1, keepdim=True) + eps).rsqrt()
        v = dh.double() * pr
        d = d + r2 * v - x * r2 ** 3 * (v * x).mean(1, keepdim=True)
        da = da + (r2 * v).abs() + x.abs() * r2 ** 3 * (v * x).abs().mean(1, keepdim=True)
        t = dh.double() * x * r2
        out["dgamma_pre"] = (t.sum(0), t.abs().sum(0))
    out["dx"] = (d, da)
    if y is not None:
        q, qa = alpha * g * po * d, (alpha * g * po).abs() * da
        if post is not None:
            dy = r1 * q - y * r1 ** 3 * (q * y).mean(1, keepdim=True)
            dya = r1 * qa + y.abs() * r1 ** 3 * (qa * y.abs()).mean(1, keepdim=True)
            t, ta = alpha * g * d * y * r1, (alpha * g * y * r1).abs() * da
            out["dgamma_post"] = (t.sum(0), ta.sum(0))
        else:
            dy, dya = q, qa
        out["dy"] = (dy, dya)
        if gate is not None:
            t, ta = alpha * d * n, (alpha * n).abs() * da
            G = gate.shape[0]
            out["dgate"] = (t.reshape(G, T // G, D).sum(1), ta.reshape(G, T // G, D).sum(1))
    return out


NORMS = [
    # T, D, G (0: no gate), gamma_post, y, gamma_pre, dx_out
    (1, 8, 1, True, True, True, True),
    (2, 2048, 1, True, True, True, True),
    (5, 264, 5, True, True, True, True),       # a gate for every row
    (33, 72, 11, True, True, True, False),
    (700, 136, 7, True, True, True, True),     # gate rows that cross blocks
    (701, 1024, 1, True, True, False, True),
    (64, 1032, 0, True, True, True, True),
    (40, 520, 2, False, True, True, True),
    (9, 768, 1, False, True, False, True),
    (17, 2056, 0, True, False, True, True),    # the first norm alone
    (6, 4104, 3, True, True, True, True),
    (3, 7168, 1, True, True, True, True),
    (4, 8200, 2, True, True, True, True),
    (2, 16384, 1, True, True, True, True),
    (1216, 64, 1216, True, True, True, True),
]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("params", ["same", "fp32"])
@pytest.mark.parametrize("T,D,G,has_post,has_y,has_pre,has_dxo", NORMS)
def test_block_norm(M, T, D, G, has_post, has_y, has_pre, has_dxo, dtype, params):
    p = dtype if params == "same" else torch.float32
    alpha, eps = 0.75, 1e-5
    x, y = randn(1, dtype, T, D, scale=2.0), randn(2, dtype, T, D)
    y[T // 2] = 0  # a row of zeros: its norm is bounded by eps alone
    if not has_y:
        y, has_post, G = None, False, 0
    post = (1 + randn(3, torch.float32, D, scale=0.2)).to(p) if has_post else None
    gate = randn(4, p, G, D) if G else None
    pre = (1 + randn(5, torch.float32, D, scale=0.2)).to(p) if has_pre else None
    dxo = randn(6, dtype, T, D) if has_dxo or not has_pre else None
    dh = randn(7, dtype, T, D) if has_pre else None
    ref = norm_reference(x, y, dxo, dh, post, gate, pre, alpha, eps)
    cu = lambda t: None if t is None else t.cuda()
    kw = dict(gamma_post=cu(post), gate=cu(gate), gamma_pre=cu(pre), alpha=alpha, eps=eps)
    xo, h = M.block_norm(cu(x), cu(y), **kw)
    assert (xo is None) == (y is None) and (h is None) == (pre is None)
    if xo is not None:
        close(xo, *ref["x_out"], 64, "x_out")
        xi = x.cuda()
        assert M.block_norm(xi, cu(y), **kw, x_out=xi)[0] is xi and torch.equal(xi, xo)  # in place
    if h is not None:
        close(h, *ref["h"], 64, "h")
    grads = dict(zip(("dx", "dy", "dgamma_post", "dgate", "dgamma_pre"),
                     M.block_norm_backward(cu(x), cu(y), cu(dxo), cu(dh), **kw)))
    for name, got in grads.items():
        assert (got is None) == (name not in ref), name
        if got is not None:
            rows = T if name in ("dgamma_post", "dgamma_pre") else T // max(G, 1) if name == "dgate" else 0
            close(got, *ref[name], 64 + rows, name)
    again = M.block_norm_backward(cu(x), cu(y), cu(dxo), cu(dh), **kw)
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, grads.values()))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,D,G", [
    (6999, 64, 2333),   # gates shorter than the rows of a row group, some shared by two
    (7000, 64, 3500),   # and none shared
    (7000, 64, 1000),   # longer
    (1200, 4104, 400),
    (1200, 4104, 24),
    (608, 8200, 304),
    (610, 8200, 122),
])
def test_block_norm_of_many_gates(M, T, D, G, dtype):
    test_block_norm(M, T, D, G, True, True, True, True, dtype, "same")


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("D", [264, 2048, 5120, 8200])
def test_block_norm_gradient_in_place(M, D, dtype):
    """dx may be dx_out."""
    T = 310
    x, y, dxo, dh = (randn(i, dtype, T, D).cuda() for i in range(4))
    post, gate, pre = (randn(4 + i, dtype, *s).cuda() for i, s in enumerate([(D,), (5, D), (D,)]))
    want = M.block_norm_backward(x, y, dxo, dh, post, gate, pre)
    ws = M.workspace(M.block_norm_backward_workspace_size(T, D, 5))
    dx, dy = dxo.clone(), torch.empty_like(y)
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dtype]
    st = M.lib().moe_block_norm_backward(code, code, T, D, 5, 1.0, 1e-6, post.data_ptr(), gate.data_ptr(), pre.data_ptr(),
                                         x.data_ptr(), y.data_ptr(), dx.data_ptr(), dh.data_ptr(), dx.data_ptr(), dy.data_ptr(),
                                         None, None, None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == M.MOE_OK and torch.equal(dx, want[0]) and torch.equal(dy, want[1])


def test_block_norm_gradient_against_differences(M):
    """Derivative of <dx_out, x_out> + <dh, h> along the signs of its gradient
    in every input, by central differences in fp32: cut-off below d^2 / 6 times a third derivative
    of at most 100 for each entry, rounding below 64 2^-24 |values| / d."""
    T, D, G, alpha, eps, d = 12, 64, 3, 0.5, 1e-3, 2.0 ** -8
    names = ["x", "y", "gamma_post", "gate", "gamma_pre"]
    shapes = [(T, D), (T, D), (D,), (G, D), (D,)]
    at = [randn(i, torch.float32, *s) + (1.0 if len(s) == 1 else 0.0) for i, s in enumerate(shapes)]
    dxo, dh = randn(40, torch.float32, T, D), randn(41, torch.float32, T, D)

    def f(t):
        v = {n: (a + t * b).cuda() for n, a, b in zip(names, at, along)}
        xo, h = M.block_norm(**v, alpha=alpha, eps=eps)
        return (xo.cpu().double() * dxo.double()).sum().item() + (h.cpu().double() * dh.double()).sum().item()

    v = {n: a.cuda() for n, a in zip(names, at)}
    xo, _ = M.block_norm(**v, alpha=alpha, eps=eps)
    v["x_out"] = xo
    del v["x"]
    grads = M.block_norm_backward(**v, dx_out=dxo.cuda(), dh=dh.cuda(), alpha=alpha, eps=eps)
    along = [t.sign().cpu() for t in grads]
    want = sum(t.cpu().double().abs().sum().item() for t in grads)
    tol = 2 * T * D * (d * d / 6 * 100 + 64 * 2.0 ** -24 * 4 / d)
    assert abs((f(d) - f(-d)) / (2 * d) - want) <= tol
    assert abs(want) > 3 * tol


@pytest.mark.parametrize("T", [3, 700])
def test_block_norm_where_the_block_cancels_the_stream(M, T):
    """x' = x + alpha gate n of a hundredth of its terms' size: its mean square
    has to come from x' itself, not from sums of squares that cancel."""
    D, alpha, eps = 512, 0.75, 1e-6
    y = randn(2, torch.float32, T, D)
    post, pre, gate = (1 + randn(i, torch.float32, D, scale=0.2) for i in (3, 4, 5))
    gate = gate[None]
    yd = y.double()
    n = alpha * gate.double() * yd * ((yd * yd).mean(1, keepdim=True) + eps).rsqrt() * post.double()
    x = (-0.99 * n).float()
    ref = norm_reference(x, y, y, y, post, gate, pre, alpha, eps)
    xo, h = M.block_norm(x.cuda(), y.cuda(), post.cuda(), gate.cuda(), pre.cuda(), alpha, eps)
    close(xo, *ref["x_out"], 64, "x_out")
    close(h, *ref["h"], 64, "h")


def test_block_norm_of_no_rows(M):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    gate = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    xo, h = M.block_norm(x, x.clone(), p, gate, p)
    assert xo.shape == h.shape == (0, 64)
    dx, dy, dpost, dgate, dpre = M.block_norm_backward(x, x.clone(), x.clone(), x.clone(), p, gate, p)
    assert dx.shape == dy.shape == (0, 64) and not dpost.any() and not dgate.any() and not dpre.any()
    assert M.swiglu(torch.empty(0, 64, device="cuda")).shape == (0, 32)


def test_operators_on_a_side_stream(M):
    """Every operator runs on the stream it is given, behind what that stream holds."""
    T, D = 50, 512
    s = torch.cuda.Stream()
    x, y, p = randn(1, torch.bfloat16, T, D).cuda(), randn(2, torch.bfloat16, T, D).cuda(), torch.ones(D, dtype=torch.bfloat16).cuda()
    ref = M.block_norm(x, y, p, None, p)
    gref = M.block_norm_backward(x, y, x, y, p, None, p)
    sref = M.swiglu(x)
    torch.cuda.synchronize()
    x2 = torch.zeros_like(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(5):
            big = big @ big * 1e-4
        x2.copy_(x)
        got = M.block_norm(x2, y, p, None, p)
        ggot = M.block_norm_backward(x2, y, x2, y, p, None, p)
        sgot = M.swiglu(x2)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and torch.equal(sgot, sref)
    assert all(a is None or torch.equal(a, b) for a, b in zip(ggot, gref))


def test_outputs_belong_to_the_given_stream(M):
    """What a call allocates comes from the pool of the stream that writes it."""
    s = torch.cuda.Stream()
    x, w, p = randn(1, torch.bfloat16, 64, 64).cuda(), randn(2, torch.bfloat16, 2, 64, 64).cuda(), torch.ones(64, dtype=torch.bfloat16).cuda()
    off, half, rw = torch.tensor([0, 30, 64], dtype=torch.int32).cuda(), x[:, :32].contiguous(), torch.ones(64).cuda()
    torch.cuda.synchronize()
    outs = [M.grouped_mm(x, w, off, stream=s), M.grouped_mm_dx(x, w, off, stream=s), M.grouped_mm_dw(x, x, off, stream=s),
            M.swiglu(x, stream=s), *M.swiglu_backward(half, x, rw, stream=s)]
    s.synchronize()
    outs += [*M.block_norm(x, x, p, None, p, stream=s), *M.block_norm_backward(x, x, x, x, p, None, p, stream=s)]
    s.synchronize()
    pools = {}
    for seg in torch.cuda.memory_snapshot():
        pools[range(seg["address"], seg["address"] + seg["total_size"])] = seg["stream"]
    for t in outs:
        if t is not None:
            assert [v for k, v in pools.items() if t.data_ptr() in k] == [s.cuda_stream]
    assert torch.cuda.current_stream() != s
