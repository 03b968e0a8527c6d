"""The operators of expert blocks at the ends of what they take: sums of 8-bit products
around and beyond 2^24, as many experts as there may be, the widest layers, and layer norms of
rows of one value and of few rows far from zero.  Tolerances as in test_expert_block_ops_gpu
and test_expert_layer_gpu."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_expert_block_ops_gpu import BF16, F16, F32, close, codes, dev, norm_reference, offsets_of, randn  # noqa: E402
from tests.test_expert_layer_gpu import case, check, reference  # noqa: E402
from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


# --------------------------------------------------------------- 8-bit sums
FEW, MANY = [7, 1, 4], [40, 90]  # rows of the experts: for the kernel of few rows and the other one


def cancelling(counts, N, K, seed=0):
    """Odd codes of 101 to 127 whose products grow to a large sum in the first half of K and
    take nearly all of it back in the second; the sums in 64 bits, and those of |a b|."""
    g = torch.Generator().manual_seed(seed)
    R, E, half = sum(counts), len(counts), K // 2
    odd = lambda *s: torch.randint(50, 64, s, generator=g, dtype=torch.int8) * 2 + 1  # noqa: E731
    x, w = odd(R, half), odd(E, N, half)
    back = torch.where(torch.rand(E, N, half, generator=g) < 8 / half, (w.int() - 2).to(torch.int8), w)
    x, w = torch.cat([x, x], 1), torch.cat([w, -back], 2)
    ref, most = torch.zeros(R, N, dtype=torch.float64), torch.zeros(R, N, dtype=torch.float64)
    r = 0
    for e, c in enumerate(counts):
        a, b = x[r:r + c].double(), w[e].double()
        ref[r:r + c], most[r:r + c] = a @ b.T, a.abs() @ b.abs().T
        r += c
    assert most.max() / 2 < 2 ** 31 and (ref.abs() < 16384).all() and ref.count_nonzero() > ref.numel() / 2
    return x, w, ref, most


def product(M, x, w, counts, dtype):
    one, scales = torch.full((len(x),), 0.5), torch.full(w.shape[:2], 0.25)
    return M.grouped_mm_i8(*dev(x, one, w, scales, offsets_of(counts)), dtype=dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K,counts", [(1040, FEW), (1040, MANY), (2064, FEW), (2064, MANY), (4112, FEW), (32768, FEW)])
def test_exact_sums_that_cancel(M, K, counts, dtype):
    """Partial sums up to 2^24 (K 2064: 1032 products of at most 16129), with few rows up to 2^31:
    nothing is rounded but the output."""
    x, w, ref, most = cancelling(counts, 72, K)
    assert counts is FEW or most.max() / 2 <= 2 ** 24
    close(product(M, x, w, counts, dtype), ref / 8, ref.abs() / 8, 0, "y")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K", [4112, 8192, 32768])
def test_sums_beyond_2_to_the_24_that_cancel(M, K, dtype):
    """Many rows: the sum is held in fp32, 16 products added at a time."""
    x, w, ref, most = cancelling(MANY, 72, K)
    assert most.max() / 2 > 2 ** 24
    close(product(M, x, w, MANY, dtype), ref / 8, most / 8, 2 * (K / 8 + 16), "y")


# ------------------------------------------------------------- many experts
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k", [(3, 8), (8, 5), (32, 8)])
@pytest.mark.parametrize("E", [257, 513, 1023, 1024])
def test_layers_of_many_experts(M, E, T, k, dtype):
    x, lg, w13, w2 = case(E + T, T, k, E, 64, 64, dtype)
    for t in range(T):  # experts at both ends and around the threads' and lanes' shares
        for j, e in enumerate((E - 1, 0, E - 2, 255, 256)):
            lg[t, e] += 5.0 * ((t + j) % 3 == 0)
    lg[0, 0] = 9.0
    lg[T - 1] = torch.linspace(0, 1, E)  # the last ones in order
    want, tol, ids = reference(x, lg, w13, w2, k)
    assert (ids == E - 1).any() and (ids == 0).any() and (ids[T - 1] == np.arange(E - 1, E - 1 - k, -1)).all()
    ws, got_ids = M.workspace(M.expert_layer_workspace_size(T, k, E, 64, 64)), torch.empty(T, k, dtype=torch.int32, device="cuda")
    got = M.expert_layer(*dev(x, lg, w13, w2), k, ids=got_ids, ws=ws)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    check(got, want, tol)
    assert M.get_device_error(ws) == M.MOE_OK


@pytest.mark.parametrize("E", [257, 513, 1023, 1024])
@pytest.mark.parametrize("R", [31, 128, 300, 5000, 100000])
def test_8_bit_products_of_many_experts(M, E, R):
    """Few rows, and tiles of 64 and of 192 rows; the first and last experts have some."""
    N, K = 72, 64
    g = torch.Generator().manual_seed(E + R)
    e = torch.cat([torch.tensor([0, E - 1, E - 1, E - 2, 255, 256]), torch.randint(0, E, (R - 6,), generator=g)]).sort().values
    counts = torch.bincount(e, minlength=E).tolist()
    assert sum(counts) == R
    x, w, xs, sw = codes(1, R, K), codes(2, E, N, K), randn(3, F32, R).abs() + 0.1, (randn(4, F32, E, N).abs() + 0.1) / 4000
    ref = torch.bmm(w[e].double(), x.double()[:, :, None])[:, :, 0] if R <= 5000 else torch.zeros(R, N, dtype=torch.float64)
    if R > 5000:
        at = np.concatenate([[0], np.cumsum(counts)])
        for i in range(E):
            ref[at[i]:at[i + 1]] = x[at[i]:at[i + 1]].double() @ w[i].double().T
    ref = ref * xs.double()[:, None] * sw[e].double()
    space = M.workspace(M.grouped_mm_i8_workspace_size(R, E, N, K))
    got = M.grouped_mm_i8(*dev(x, xs, w, sw, offsets_of(counts)), ws=space)
    close(got, ref, ref.abs(), 4, "y")
    assert M.get_device_error(space) == M.MOE_OK


# ------------------------------------------------------------------- widths
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,d,f", [(2, 2, 2, 32768, 64), (2, 2, 2, 64, 32768), (6, 2, 3, 64, 32704), (20, 1, 2, 32704, 64),
                                       (20, 1, 2, 128, 32768), (32, 2, 3, 16448, 128)])
def test_widest_layers(M, T, k, E, d, f, dtype):
    x, lg, w13, w2 = case(T + d, T, k, E, d, f, dtype)
    want, tol, ids = reference(x, lg, w13, w2, k)
    ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
    got = M.expert_layer(*dev(x, lg, w13, w2), k, ws=ws)
    check(got, want, tol)
    assert M.get_device_error(ws) == M.MOE_OK


# --------------------------------------------------------------- layer norms
@pytest.mark.parametrize("D", [8, 1032, 2048, 5000, 16384])
@pytest.mark.parametrize("T", [2, 200])
@pytest.mark.parametrize("value", [0.0, 7.0, -300.0, 1e4, 3e9, 1e19, -2e37])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_one_value(M, T, D, value, dtype):
    """h is beta.  The mean is off by at most 65 2^-24 of the value (a tree of 64 additions, the
    division), all c = x - mean are that; the mean of c is off by 65 2^-24 of it, and the
    variance is held to at least 2^-22 c^2, 2^-11 c the deviation: |h - beta| is at most
    66 2^-24 2^11, and the products of 2^11 are rounded by 2^-13.
    dx is r (v - mean v) with an r of at most 1 / sqrt(eps)."""
    eps = 1e-5
    x = torch.full((T, D), value).to(dtype)
    beta = randn(1, dtype, D)
    _, got = M.layer_norm(x.cuda(), beta=beta.cuda(), eps=eps)
    off = (got.cpu().double() - beta.double()).abs()
    assert (off <= 68 * 2.0 ** -13 + 2.0 ** -8 * (beta.double().abs() + 2.0 ** -6) * (dtype == BF16)).all(), off.max().item()
    dh = randn(2, dtype, T, D)
    dx = M.layer_norm_backward(x.cuda(), dh.cuda(), eps=eps)[0].cpu().double()
    v = dh.double() - dh.double().mean(1, keepdim=True)
    r = (dx * v).sum(1, keepdim=True) / (v * v).sum(1, keepdim=True).clamp_min(1e-30)
    most = eps ** -0.5
    assert (r >= -1e-30).all() and (r <= most * (1 + 2.0 ** -7)).all()
    if abs(value) <= 1e4:  # c is at most 0.04, the variance's floor 4e-10: r as it should be
        assert (r >= most * (1 - 2.0 ** -7)).all()
    # along v, but for n mean(v n), of n up to 68 2^-13 and a mean (a difference of sums) of 134
    # 2^-13 mean |v|: 2^-12.8; and for dx's rounding, in dx and in the estimate of r
    rest = (dx - r * v).abs()
    tol = r.abs() * (dh.double().abs().mean(1, keepdim=True) * 2.0 ** -12 + v.abs() * 2.0 ** -7) + 2.0 ** -8 * dx.abs() + 2.0 ** -120
    assert (rest <= tol).all(), (rest / tol).max().item()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_rows_far_from_zero(M, dtype):
    D, T = 1032, 2
    x = torch.stack([randn(1, dtype, D, shift=300.0), randn(5, dtype, D, scale=1e22, shift=3e24)])
    n, big, r, _, h, terms = norm_reference(x.double(), None, None, 1e-5)
    _, got = M.layer_norm(x.cuda())
    close(got, h, terms, 64, "h")
    dh = randn(6, dtype, T, D)
    v = dh.double()
    dx = r * (v - v.mean(1, keepdim=True) - n * (v * n).mean(1, keepdim=True))
    terms = r * (v.abs() + v.abs().mean(1, keepdim=True) + big * (v.abs() * big).mean(1, keepdim=True))
    got = M.layer_norm_backward(x.cuda(), dh.cuda())[0]
    close(got, dx, terms + 2.0 ** -120, 128, "dx")
