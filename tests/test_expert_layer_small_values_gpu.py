"""The layer for a few tokens in fp16 where its activations are small, against its formula in
64 bits.

Tolerance of an output in units of 2^-24 besides the rounding to fp16 (2^-11 |ref|, 2^-25
among the subnormals):
  - a product of L terms: s(L) = 2 (L / 8 + 16) of sum |a b|;
  - h = SiLU(a) u: 1.1 |u| of the error of a, |SiLU(a)| of that of u, and 16 of |h|; the
    weight p: 16 of |p h|;
  - p h is kept as two fp16 numbers, the second one its rounding error times 2^11: off by
    2^-11 of 2^-11 |p h|, and by at least half of fp16's smallest number, 2^-25, times 2^-11.
"""
import pytest

torch = pytest.importorskip("torch")

from tests.test_expert_layer_gpu import case, choose, randn, steps  # noqa: E402
from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def reference(x, logits, w13, w2, k):
    T, d = x.shape
    f, one = w2.shape[2], 2.0 ** -24
    ids, p = choose(logits, k)
    out, tol = torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            w, wd, xt = w13[ids[t, j]].double(), w2[ids[t, j]].double(), x[t].double()
            (a, u), (ba, bu) = (w @ xt).split(f), (w.abs() @ xt.abs()).split(f)
            s = a * torch.sigmoid(a)
            ph = float(p[t, j]) * s * u
            dph = float(p[t, j]) * one * steps(d) * (1.1 * ba * u.abs() + s.abs() * bu) + (32 * one + 2.0 ** -22) * ph.abs() + 2.0 ** -36
            out[t] += wd @ ph
            tol[t] += wd.abs() @ (dph + one * steps(f) * ph.abs())
    return out, tol + 2.0 ** -11 * out.abs() + 2.0 ** -25


@pytest.mark.parametrize("scale", [1e-1, 1e-2, 5e-3, 1e-3, 1e-4])
@pytest.mark.parametrize("T,k,E,d,f", [
    (1, 8, 16, 512, 768),
    (3, 8, 8, 256, 768),      # up to 4 tokens: values and errors in one product
    (7, 8, 16, 512, 768),     # up to 8
    (13, 4, 64, 256, 768),    # experts of up to four tokens
    (14, 8, 12, 256, 320),    # of up to 8 and more
    (30, 8, 10, 192, 768),    # of more than 16
])
def test_small_activations(M, T, k, E, d, f, scale):
    """Outputs of unit weights down: no more is lost than one rounding of the output."""
    x, lg, w13, _ = case(T + E, T, k, E, d, f, F16)
    x, w2 = (x.float() * scale).half(), randn(7, F16, E, d, f)
    want, tol = reference(x, lg, w13, w2, k)
    ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k, ws=ws).cpu().double()
    err = (got - want).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), ((err / tol).max().item(), err.square().mean().sqrt().item())
    assert M.get_device_error(ws) == M.MOE_OK


@pytest.mark.parametrize("T", [1, 6, 20])
def test_weights_that_make_an_expert_negligible(M, T):
    """One expert with nearly all the weight, and one whose weight alone makes p h small."""
    k, E, d, f = 2, 4, 192, 320
    x, lg, w13, w2 = case(T, T, k, E, d, f, F16)
    lg = torch.where(lg > lg.mean(1, keepdim=True), lg, lg - 12.0)
    want, tol = reference(x, lg, w13, w2, k)
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k).cpu().double()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("T", [1, 6, 20])
def test_large_activations(M, T):
    """p h up to fp16's largest number: the rounding error times 2^11 stays within the range."""
    k, E, d, f = 1, 2, 64, 192
    x, lg, w13, w2 = case(T, T, k, E, d, f, F16)
    x = torch.ones_like(x)
    w13 = torch.zeros_like(w13)
    w13[:, :f, 0] = torch.linspace(1.0, 256.0, f).half()
    w13[:, f:, 0] = 255.875                               # times 256: 65504
    w2 = (w2.float() * 2.0 ** -6).half()
    want, tol = reference(x, lg, w13, w2, k)
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k).cpu().double()
    assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all()
