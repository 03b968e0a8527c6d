"""Layer norm, rows to 8-bit codes and 8-bit grouped products on the GPU against
plain 64-bit formulas.

Tolerances.  An output rounded once to its type is off by at most u |ref| (u = 2^-8
bf16, 2^-11 fp16, 2^-24 fp32), among the subnormals by half their spacing.  Before that:
  - layer norm: a row's sums are trees of at most 64 fp32 additions, taken of x' and of
    x' less its mean: every normalised value is off by at most 64 2^-24 of
    N = (|x'| + |mean|) / std, which stands for |n| in the terms below; 128 roundings
    where a product of two such sums enters (gradients);
  - sums over rows: one more 2^-24 for each row;
  - 8-bit products: the sum is exact below 2^24, then three fp32 roundings; beyond,
    (K / 8 + 16) 2^-23 sum |a b| as for the 16-bit products (16 products at a time
    are added to the accumulator);
  - codes are exact, and scales rounded once.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
SUBNORMAL = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def randn(seed, dtype, *shape, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def close(got, ref, terms, steps, what):
    """|got - ref| <= u |ref| + steps 2^-24 terms, element by element."""
    ref = ref.double()
    tol = U[got.dtype] * ref.abs() + steps * 2.0 ** -24 * terms.double() + SUBNORMAL[got.dtype]
    err = (got.detach().cpu().double() - ref).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, (what, worst, err.max().item())


def dev(*ts):
    return [t.cuda() if t is not None else None for t in ts]


# ------------------------------------------------------------------ layer norm
def norm_reference(x, gamma, beta, eps):
    """x' in 64 bits: normalised rows, their bound N, 1 / std, h and its terms."""
    mean = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    n = (x - mean) * r
    big = (x.abs() + mean.abs()) * r
    g = gamma.double() if gamma is not None else torch.ones(x.shape[1], dtype=torch.float64)
    b = beta.double() if beta is not None else torch.zeros(x.shape[1], dtype=torch.float64)
    return n, big, r, g, n * g + b, big * g.abs() + b.abs()


SHAPES = [(1, 8), (1, 2048), (3, 264), (7, 4096), (2, 4104), (5, 8192), (3, 8200), (2, 16384), (150, 72), (153, 1288),
          (700, 768), (1213, 2048), (311, 7168), (1000, 8), (4001, 32)]


@pytest.mark.parametrize("dtype,ptype", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("T,D", SHAPES)
def test_layer_norm(M, T, D, dtype, ptype):
    x, y = randn(1, dtype, T, D, scale=2.0, shift=0.5), randn(2, dtype, T, D)
    gamma, beta = randn(3, ptype, D, scale=0.3, shift=1.0), randn(4, ptype, D, scale=0.2)
    xd, yd, gd, bd = dev(x, y, gamma, beta)
    xo = x.double() + y.double()
    _, _, _, _, h, terms = norm_reference(xo, gamma, beta, 1e-5)
    got_x, got_h = M.layer_norm(xd, yd, gd, bd)
    close(got_x, xo, xo.abs(), 2, "x_out")
    close(got_h, h, terms, 64, "h")
    _, _, _, _, h, terms = norm_reference(x.double(), gamma, beta, 1e-5)
    none, got_h = M.layer_norm(xd, gamma=gd, beta=bd)
    assert none is None
    close(got_h, h, terms, 64, "h without y")


@pytest.mark.parametrize("dtype,ptype", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("T,D", SHAPES)
def test_layer_norm_backward(M, T, D, dtype, ptype):
    x, dh, dxo = randn(1, dtype, T, D, scale=2.0, shift=0.5), randn(2, dtype, T, D, scale=0.1), randn(3, dtype, T, D, scale=0.1)
    gamma, beta = randn(4, ptype, D, scale=0.3, shift=1.0), randn(5, ptype, D)
    xd, dhd, dxod, gd, bd = dev(x, dh, dxo, gamma, beta)
    n, big, r, g, _, _ = norm_reference(x.double(), gamma, beta, 1e-5)
    dh64 = dh.double()
    v = dh64 * g
    dx = r * (v - v.mean(1, keepdim=True) - n * (v * n).mean(1, keepdim=True))
    terms = r * (v.abs() + v.abs().mean(1, keepdim=True) + big * (v.abs() * big).mean(1, keepdim=True))
    ws = M.workspace(M.layer_norm_backward_workspace_size(T, D))
    got = M.layer_norm_backward(xd, dhd, dxod, gd, bd, ws=ws)
    close(got[0], dx + dxo.double(), terms + dxo.double().abs(), 128, "dx")
    close(got[1], (dh64 * n).sum(0), (dh64.abs() * big).sum(0), 128 + T, "dgamma")
    close(got[2], dh64.sum(0), dh64.abs().sum(0), 64 + T, "dbeta")
    again = M.layer_norm_backward(xd, dhd, dxod, gd, bd, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # without the stream's gradient, without parameters
    v, big_v = dh64, dh64.abs()
    dx = r * (v - v.mean(1, keepdim=True) - n * (v * n).mean(1, keepdim=True))
    terms = r * (big_v + big_v.mean(1, keepdim=True) + big * (big_v * big).mean(1, keepdim=True))
    got = M.layer_norm_backward(xd, dhd)
    assert got[1] is None and got[2] is None
    close(got[0], dx, terms, 128, "dx alone")


def test_layer_norm_against_differences(M):
    """dx, dgamma and dbeta against differences of the 64-bit formula."""
    T, D, eps, step = 3, 16, 1e-2, 1e-6
    x, dh = randn(1, F32, T, D), randn(2, F32, T, D)
    gamma, beta = randn(3, F32, D), randn(4, F32, D)

    def loss(a, g, b):
        return (norm_reference(a, g, b, eps)[4] * dh.double()).sum()

    dx, dgamma, dbeta = M.layer_norm_backward(*dev(x, dh), None, *dev(gamma, beta), eps=eps)
    args = [x.double(), gamma.double(), beta.double()]
    for which, got in ((0, dx), (1, dgamma), (2, dbeta)):
        for i in range(args[which].numel()):
            lo, hi = [a.clone() for a in args], [a.clone() for a in args]
            lo[which].view(-1)[i] -= step
            hi[which].view(-1)[i] += step
            d = (loss(*hi) - loss(*lo)) / (2 * step)
            # the third derivatives' step^2 and 64-bit rounding over the step: 1e-8 of terms up to 1e3
            assert abs(got.view(-1)[i].item() - d.item()) < 1e-5 * max(1.0, abs(d.item())), (which, i)


@pytest.mark.parametrize("T", [2, 400])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_far_rows(M, T, dtype):
    """Rows far from zero, constant, tiny and near the type's ends."""
    D = 1032
    rows = [randn(1, dtype, D, shift=300.0), torch.full((D,), 7.0).to(dtype), randn(2, dtype, D, scale=1e-18),
            randn(3, dtype, D, scale=1e30), randn(4, dtype, D, scale=1e-3, shift=-2e37), torch.zeros(D).to(dtype),
            randn(5, dtype, D, scale=1e22, shift=3e24)]
    x = torch.stack([rows[i % len(rows)] for i in range(T)])
    if T == 2:
        x = torch.stack([rows[3], rows[4]])
    n, big, r, _, h, terms = norm_reference(x.double(), None, None, 1e-5)
    _, got = M.layer_norm(x.cuda())
    close(got, h, terms, 64, "h")
    dh = randn(6, dtype, T, D)
    v = dh.double()
    dx = r * (v - v.mean(1, keepdim=True) - n * (v * n).mean(1, keepdim=True))
    terms = r * (v.abs() + v.abs().mean(1, keepdim=True) + big * (v.abs() * big).mean(1, keepdim=True))
    # r of the largest rows may be among fp32's subnormals
    got = M.layer_norm_backward(x.cuda(), dh.cuda())[0]
    close(got, dx, terms + 2.0 ** -120, 128, "dx")


def test_layer_norm_not_finite(M):
    x = randn(1, F32, 200, 64)
    x[3, 5], x[7, 0] = float("inf"), float("nan")
    _, h = M.layer_norm(x.cuda())
    bad = torch.isnan(h).any(1).cpu()
    assert bad[3] and bad[7] and bad.sum() == 2


@pytest.mark.parametrize("T", [4, 1000])
def test_layer_norm_in_place(M, T):
    x, y = randn(1, BF16, T, 512).cuda(), randn(2, BF16, T, 512).cuda()
    xo, h = M.layer_norm(x, y)
    x2 = x.clone()
    xo2, h2 = M.layer_norm(x2, y, x_out=x2)
    assert xo2.data_ptr() == x2.data_ptr() and torch.equal(xo, x2) and torch.equal(h, h2)


def test_layer_norm_no_rows(M):
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    g = torch.ones(64, dtype=BF16, device="cuda")
    xo, h = M.layer_norm(x, x, g, g)
    assert xo.shape == h.shape == (0, 64)
    dx, dg, db = M.layer_norm_backward(x, x, None, g, g)
    assert dx.shape == (0, 64) and not dg.any() and not db.any()


# --------------------------------------------------------------- rows to codes
def codes_reference(x):
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    # exact numerators: the quotient falls on the right side of every border
    codes = torch.where(top > 0, torch.round(127 * x / top.clamp_min(1e-300)), torch.zeros_like(x))
    return codes.to(torch.int8), (top[:, 0] / 127).float()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,D", [(1, 16), (8, 768), (5, 512), (33, 528), (4, 1024), (3, 2048), (2, 2064), (3, 4096),
                                 (2, 8192), (2, 8208), (1, 16384), (1, 32768), (1000, 272)])
def test_quantize_rows(M, T, D, dtype):
    x = randn(T + D, dtype, T, D)
    x[0, :8] = 0
    codes, scales = M.quantize_rows(x.cuda())
    want, want_s = codes_reference(x)
    assert torch.equal(codes.cpu(), want)
    assert torch.equal(scales.cpu(), want_s)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_rows_borders_and_ends(M, dtype):
    """Ties between two codes, rows of zeros, subnormals and the type's ends."""
    big = torch.finfo(dtype).max
    tie = torch.arange(-127, 129).float() / 2
    rows = []
    for unit in (1.0, 2.0 ** -10, 2.0 ** 6):
        r = torch.cat([tie[:-1], torch.tensor([127.0])]) * unit
        rows.append(r)
    rows.append(torch.zeros(256))
    rows.append(torch.full((256,), torch.finfo(dtype).tiny))
    rows.append(torch.linspace(-1, 1, 256) * 2.0 ** (-133 if dtype == BF16 else -24 if dtype == F16 else -140))
    rows.append(torch.linspace(-1, 1, 256) * big)
    x = torch.stack(rows).to(dtype)
    codes, scales = M.quantize_rows(x.cuda())
    want, want_s = codes_reference(x)
    assert torch.equal(codes.cpu(), want)
    assert torch.equal(scales.cpu(), want_s)


def test_quantize_rows_not_finite(M):
    x = randn(1, F32, 6, 64)
    x[1, 3], x[4, 60] = float("-inf"), float("nan")
    codes, scales = M.quantize_rows(x.cuda())
    assert torch.isnan(scales).cpu().tolist() == [False, True, False, False, True, False]
    assert not codes[1].any() and not codes[4].any()


def test_quantize_rows_map(M):
    """Rows of a permutation; entries out of range give zeros."""
    T, k, D = 37, 3, 208
    x = randn(1, BF16, T, D)
    ids = torch.stack([torch.randperm(16, generator=torch.Generator().manual_seed(i))[:k] for i in range(T)]).to(torch.int32)
    p = M.permute(ids.cuda(), 16)
    codes, scales = M.quantize_rows(x.cuda(), p["sorted"], k)
    want, want_s = codes_reference(x)
    src = p["sorted"].cpu().long() // k
    assert torch.equal(codes.cpu(), want[src]) and torch.equal(scales.cpu(), want_s[src])
    m = torch.tensor([0, -1, T * k, T * k - 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    codes, scales = M.quantize_rows(x.cuda(), m.cuda(), k)
    assert torch.equal(codes[0].cpu(), want[0]) and torch.equal(codes[3].cpu(), want[T - 1])
    for i in (1, 2, 4, 5):
        assert not codes[i].any() and scales[i] == 0
    none, s = M.quantize_rows(x.cuda(), m.cuda()[:0], k)
    assert none.shape == (0, D) and s.shape == (0,)


@pytest.mark.parametrize("T,R,D,dtype", [(301, 9000, 2048, BF16), (700, 81000, 208, F16), (64, 1500, 12304, F32),
                                         (1, 600, 32768, BF16)])
def test_quantize_rows_taken_several_times(M, T, R, D, dtype):
    """Rows quantised once and copied: any map, entries out of range, given spaces and none,
    and the same codes as of each row by itself."""
    k = 3
    x = randn(1, dtype, T, D)
    if T > 9:
        x[9, 7] = float("inf")
    m = torch.randint(-k, (T + 1) * k, (R,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    need = M.quantize_rows_workspace_size(T, R, D)
    assert need > T * D
    src = torch.div(m, k, rounding_mode="floor").long()
    there = (src >= 0) & (src < T)
    want, want_s = codes_reference(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))
    if T > 9:
        want[9], want_s[9] = 0, float("nan")
    src = src.clamp(0, T - 1)
    want, want_s = want[src] * there[:, None], torch.where(there, want_s[src], torch.zeros(()))
    space = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    for ws in (None, space[256:256 + need]):
        codes, scales = M.quantize_rows(x.cuda(), m.cuda(), k, ws=ws)
        assert torch.equal(codes.cpu(), want)
        assert torch.equal(scales.cpu().nan_to_num(-1), want_s.nan_to_num(-1))
    assert (space[:256] == 0x5A).all() and (space[256 + need:] == 0x5A).all()
    xd, md, codes, scales = *dev(x, m), torch.empty_like(codes), torch.empty_like(scales)
    torch.cuda.synchronize()
    assert M.lib().moe_quantize_rows({BF16: 0, F16: 1, F32: 2}[dtype], xd.data_ptr(), md.data_ptr(), k, T, R, D,
                                     codes.data_ptr(), scales.data_ptr(), None, 0, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(codes.cpu(), want)
    with pytest.raises(RuntimeError):
        M.quantize_rows(x.cuda(), m.cuda(), k, ws=space[:need - 256])


# ------------------------------------------------------------- 8-bit products
def codes(seed, *shape, lo=-127, hi=128):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int8)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def product_case(counts, N, K, seed=0, lo=-127, hi=128):
    R, E = sum(counts), len(counts)
    x, w = codes(seed + 1, R, K, lo=lo, hi=hi), codes(seed + 2, E, N, K, lo=lo, hi=hi)
    xs, ws = randn(seed + 3, F32, R).abs() + 0.1, (randn(seed + 4, F32, E, N).abs() + 0.1) / (5000 * K ** 0.5)
    ref = torch.zeros(R, N, dtype=torch.float64)
    most = torch.zeros(R, N, dtype=torch.float64)
    r = 0
    for e, c in enumerate(counts):
        s = slice(r, r + c)
        scale = xs[s, None].double() * ws[e].double()
        ref[s] = x[s].double() @ w[e].double().T * scale
        most[s] = x[s].double().abs() @ w[e].double().abs().T * scale
        r += c
    return x, xs, w, ws, offsets_of(counts), ref, most


PRODUCTS = [
    ([1], 8, 16),
    ([0, 1, 0], 16, 64),
    ([0, 0], 64, 64),                         # no rows at all
    ([3, 0, 5], 72, 48),
    ([1] * 8, 256, 512),                      # one token's experts
    ([1, 2, 0, 7, 1], 768, 272),
    ([9, 20, 0, 0, 1, 2], 136, 2048),
    ([64], 136, 128),
    ([33], 8, 16),
    ([9, 55, 0, 0, 1, 8], 1536, 256),
    ([65, 63, 64, 0, 1], 264, 80),
    ([191, 1, 192, 193, 0, 31], 328, 208),    # around one and two tiles of rows
    ([385, 16, 0, 15, 17], 520, 1040),
    ([1000], 2048, 64),
    ([33] * 40, 64, 2048),
    ([2, 120, 0, 700, 5, 48, 130, 1], 128, 768),
    ([1, 0, 2, 1] * 24, 520, 1104),           # about one row an expert
    ([40] + [0] * 200 + [3], 520, 144),
    ([2331], 264, 208),
    ([40, 33, 0, 50], 1048, 1296),            # more stages than the ring's, odd ends
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("counts,N,K", PRODUCTS)
def test_grouped_mm_i8(M, counts, N, K, dtype):
    x, xs, w, ws, off, ref, _ = product_case(counts, N, K)
    space = M.workspace(M.grouped_mm_i8_workspace_size(len(xs), len(counts), N, K))
    got = M.grouped_mm_i8(*dev(x, xs, w, ws, off), dtype=dtype, ws=space)
    assert got.dtype == dtype
    close(got, ref, ref.abs(), 4, "y")
    assert M.get_device_error(space) == M.MOE_OK


SHORT = [([1, 0, 3, 1, 0, 9] * 2, 1000, 176), ([2, 1, 0, 1] * 25, 328, 16), ([1, 0, 2, 17, 0, 12], 1048, 336),
         ([1, 1, 0, 1] * 30, 200, 512)]


@pytest.mark.parametrize("counts,N,K", SHORT)
def test_grouped_mm_i8_few_rows_short_k(M, counts, N, K):
    """Many experts of few rows each and a short K: warps with weight rows of their own, some
    of them behind N."""
    x, xs, w, ws, off, ref, _ = product_case(counts, N, K)
    close(M.grouped_mm_i8(*dev(x, xs, w, ws, off)), ref, ref.abs(), 4, "y")


MANY = [([1500, 0, 700, 9, 130], 264, 2048), ([40, 33, 0, 64, 65] * 13, 72, 2064), ([300, 1, 200], 520, 8448)]


@pytest.mark.parametrize("counts,N,K", MANY)
def test_grouped_mm_i8_many_rows(M, counts, N, K):
    """Rows widened beside the product: tiles of many rows and of few, one row a unit; the same
    outputs every time, on two streams at once and as a graph."""
    x, xs, w, ws, off, ref, _ = product_case(counts, N, K)
    args = dev(x, xs, w, ws, off)
    spaces = [M.workspace(M.grouped_mm_i8_workspace_size(len(xs), len(counts), N, K)) for _ in range(2)]
    got = M.grouped_mm_i8(*args, ws=spaces[0])
    close(got, ref, ref.abs(), 4, "y")
    streams = [torch.cuda.Stream() for _ in spaces]
    torch.cuda.synchronize()
    outs = [M.grouped_mm_i8(*args, ws=space, stream=s) for _ in range(15) for s, space in zip(streams, spaces)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, got) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = M.grouped_mm_i8(*args, ws=spaces[0])
    for seed in (1, 2):
        args[0].copy_(codes(seed, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, M.grouped_mm_i8(*args, ws=spaces[1]))
        assert torch.equal(y, got) == (seed == 1)  # (those are the case's own codes)
    assert all(M.get_device_error(space) == M.MOE_OK for space in spaces)


def test_grouped_mm_i8_many_rows_outside_the_segments(M):
    counts, N, K = [900, 0, 1300], 72, 2048
    x, xs, w, ws, off, ref, _ = product_case(counts, N, K)
    big, scale = torch.zeros(len(x) + 50, K, dtype=torch.int8), torch.ones(len(x) + 50)
    big[20:20 + len(x)], scale[20:20 + len(x)] = x, xs
    y = torch.full((len(x) + 50, N), 7.0, dtype=BF16, device="cuda")
    space = M.workspace(M.grouped_mm_i8_workspace_size(len(big), 3, N, K))
    M.grouped_mm_i8(*dev(big, scale, w, ws, off + 20), y=y, ws=space)
    close(y[20:20 + len(x)], ref, ref.abs(), 4, "y")
    assert (y[:20] == 7).all() and (y[20 + len(x):] == 7).all()
    y.fill_(7)
    M.grouped_mm_i8(*dev(big, scale, w, ws, torch.tensor([0, 900, 800, 2200], dtype=torch.int32)), y=y, ws=space)
    assert M.get_device_error(space) == 6 and (y == 7).all()


@pytest.mark.parametrize("counts", [[7, 1], [40, 90]])
def test_grouped_mm_i8_largest_codes(M, counts):
    """All codes at -128, and sums beyond 2^24."""
    x, xs, w, ws, off, ref, most = product_case(counts, 264, 4112, lo=-128, hi=-127)
    got = M.grouped_mm_i8(*dev(x, xs, w, ws, off))
    close(got, ref, most, 2 * (4112 / 8 + 16), "y")


@pytest.mark.parametrize("R", [20, 300])
def test_grouped_mm_i8_rows_outside_the_segments(M, R):
    """Rows in front of the first segment and behind the last stay as they were."""
    counts = [0, 5, 3, R - 14]
    x, xs, w, ws, off, ref, _ = product_case(counts, 72, 64)
    big = torch.zeros(R + 9, 64, dtype=torch.int8)
    big[4:4 + len(x)] = x
    scale = torch.ones(R + 9)
    scale[4:4 + len(x)] = xs
    y = torch.full((R + 9, 72), 7.0, dtype=BF16, device="cuda")
    out = M.grouped_mm_i8(*dev(big, scale, w, ws, off + 4), y=y)
    assert out.data_ptr() == y.data_ptr()
    close(y[4:4 + len(x)], ref, ref.abs(), 4, "y")
    assert (y[:4] == 7).all() and (y[4 + len(x):] == 7).all()


@pytest.mark.parametrize("offsets", [[0, 10, 5, 20], [0, 5, 21, 21], [-3, 4, 9, 20], [0, 2 ** 31 - 1, 20, 20]])
@pytest.mark.parametrize("R", [20, 200])
def test_grouped_mm_i8_bad_offsets(M, offsets, R):
    """Decreasing or beyond the rows: the error word, and nothing is written."""
    x, xs, w, ws, _, _, _ = product_case([R, 0, 0], 72, 64)
    off = torch.tensor(offsets, dtype=torch.int32)
    off[off == 21] = R + 1
    space = M.workspace(M.grouped_mm_i8_workspace_size(R, 3, 72, 64))
    y = torch.full((R, 72), 7.0, dtype=BF16, device="cuda")
    M.grouped_mm_i8(*dev(x, xs, w, ws, off), y=y, ws=space)
    assert M.get_device_error(space) == 6
    assert (y == 7).all()
    assert M.get_device_error(space) == 0


def test_a_not_finite_row_spoils_its_own_outputs_alone(M):
    x = randn(1, BF16, 70, 64)
    x[11, 3] = float("inf")
    q, s = M.quantize_rows(x.cuda())
    w, ws = codes(2, 1, 72, 64).cuda(), torch.ones(1, 72, device="cuda")
    y = M.grouped_mm_i8(q, s, w, ws, torch.tensor([0, 70], dtype=torch.int32).cuda())
    bad = torch.isnan(y).any(1).cpu()
    assert bad[11] and bad.sum() == 1


def test_workspace_for_many_rows_does_for_fewer(M):
    counts = [150, 90]
    x, xs, w, ws, off, ref, _ = product_case(counts, 264, 208)
    space = M.workspace(M.grouped_mm_i8_workspace_size(4096, 2, 264, 208))
    for _ in range(3):
        close(M.grouped_mm_i8(*dev(x, xs, w, ws, off), ws=space), ref, ref.abs(), 4, "y")
    sizes = [M.grouped_mm_i8_workspace_size(r, 8, 520, 272) for r in range(0, 600, 7)]
    assert sizes == sorted(sizes)


# ------------------------------------------------------------------- together
def eight_bit_block(M, x, ids, rw, gamma, beta, w13, s13, w2, s2, space):
    """Layer norm, 8-bit gate_up, gated activation, 8-bit down, combine."""
    k = ids.shape[1]
    E = w13.shape[0]
    _, h = M.layer_norm(x, gamma=gamma, beta=beta)
    p = M.permute(ids, E)
    q, qs = M.quantize_rows(h, p["sorted"], k)
    gu = M.grouped_mm_i8(q, qs, w13, s13, p["offsets"], ws=space)
    act = M.swiglu(gu, rw.view(-1), p["sorted"])
    q2, qs2 = M.quantize_rows(act)
    yp = M.grouped_mm_i8(q2, qs2, w2, s2, p["offsets"], ws=space)
    return h, p, q, qs, gu, act, q2, qs2, yp, M.combine(yp, p["inv"], torch.ones_like(rw))


@pytest.mark.parametrize("T", [1, 5, 90])
def test_a_block_with_8_bit_experts(M, T):
    """Each step against its formula on what the step before gave; then once more as a graph,
    on another stream, with other inputs."""
    E, k, d, f = 8, 2, 256, 192
    g = torch.Generator().manual_seed(T)
    w13, w2 = codes(1, E, 2 * f, d).cuda(), codes(2, E, d, f).cuda()
    s13, s2 = torch.full((E, 2 * f), 1e-3).cuda(), torch.full((E, d), 1e-3).cuda()
    gamma, beta = randn(3, BF16, d, shift=1.0).cuda(), randn(4, BF16, d).cuda()
    x = randn(5, BF16, T, d).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    rw = torch.rand(T, k, generator=g).cuda()
    space = M.workspace(max(M.grouped_mm_i8_workspace_size(T * k, E, 2 * f, d), M.grouped_mm_i8_workspace_size(T * k, E, d, f)))
    args = (M, x, ids, rw, gamma, beta, w13, s13, w2, s2, space)
    h, p, q, qs, gu, act, q2, qs2, yp, out = eight_bit_block(*args)
    _, _, _, _, ref, terms = norm_reference(x.cpu().double(), gamma.cpu(), beta.cpu(), 1e-5)
    close(h, ref, terms, 64, "h")
    src = p["sorted"].cpu().long() // k
    want, want_s = codes_reference(h.cpu())
    assert torch.equal(q.cpu(), want[src]) and torch.equal(qs.cpu(), want_s[src])
    want, want_s = codes_reference(act.cpu())
    assert torch.equal(q2.cpu(), want) and torch.equal(qs2.cpu(), want_s)
    off = p["offsets"].tolist()
    for e in range(E):
        s = slice(off[e], off[e + 1])
        for a, b, w, sw, y in ((q, qs, w13, s13, gu), (q2, qs2, w2, s2, yp)):
            ref = a[s].cpu().double() @ w[e].cpu().double().T * b[s].cpu().double()[:, None] * sw[e].cpu().double()
            close(y[s], ref, ref.abs(), 4, "product")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eight_bit_block(*args)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = eight_bit_block(*args)[-1]
    x.copy_(randn(6, BF16, T, d))
    graph.replay()
    torch.cuda.synchronize()
    again = captured.clone()
    assert torch.equal(again, eight_bit_block(*args)[-1]) and not torch.equal(again, out)
    assert M.get_device_error(space) == M.MOE_OK
