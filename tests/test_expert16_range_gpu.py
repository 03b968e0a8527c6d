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
