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
