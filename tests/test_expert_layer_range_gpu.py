"""Activations of the layer for a few tokens that leave fp16's range: the tokens of that expert
get infinities, and the error word says so."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_expert_layer_gpu import case, choose  # noqa: E402
from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
RANGE = 8


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def call(M, x, lg, w13, w2, k):
    ws = M.workspace(M.expert_layer_workspace_size(len(x), k, len(w2), x.shape[1], w2.shape[2]))
    out = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k, ws=ws).cpu()
    return out, M.get_device_error(ws), ws


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 6, 20])
def test_every_expert_beyond_the_range(M, T, dtype):
    k, E, d, f = 1, 2, 64, 192
    x, lg, w13, w2 = case(T, T, k, E, d, f, dtype)
    x, w13 = torch.ones_like(x), torch.zeros_like(w13)
    w13[:, :f, 0] = torch.linspace(1.0, 256.0, f).to(dtype)
    w13[:, f:, 0] = 255.9375  # 256 in fp16 and bf16: the last feature of h is 65536
    out, error, _ = call(M, x, lg, w13, w2, k)
    assert error == (RANGE if dtype == F16 else M.MOE_OK)
    assert torch.isfinite(out).all() == (dtype == BF16)


@pytest.mark.parametrize("T", [4, 6, 20])
def test_one_expert_beyond_the_range(M, T):
    """Tokens without it are as they were, and the next call too."""
    k, E, d, f = 2, 8, 192, 128
    x, lg, w13, w2 = case(5, T, k, E, d, f, F16)
    lg[0, 3], lg[1, 3] = 9.0, -9.0
    clean, error, _ = call(M, x, lg, w13, w2, k)
    assert error == M.MOE_OK
    has = torch.from_numpy((choose(lg, k)[0] == 3).any(1))
    assert has[0] and not has[1]
    far = w13.clone()
    far[3] = torch.where(far[3] < 0, -400.0, 400.0).half() * torch.sign(x[0]).abs()
    far[3, 0], far[3, f] = torch.sign(x[0]) * 40, torch.sign(x[0]) * 40  # of token 0: some 6000 each
    got, error, ws = call(M, x, lg, far, w2, k)
    assert error == RANGE
    assert torch.equal(got[~has], clean[~has]) and not torch.isfinite(got[0]).any()
    again = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k, ws=ws).cpu()
    assert torch.equal(again, clean) and M.get_device_error(ws) == M.MOE_OK


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_inputs_that_are_not_finite_are_no_range_error(M, value):
    T, k, E, d, f = 6, 2, 8, 192, 128
    x, lg, w13, w2 = case(2, T, k, E, d, f, F16)
    x[2, 5] = value
    out, error, _ = call(M, x, lg, w13, w2, k)
    assert error == M.MOE_OK
    assert not torch.isfinite(out[2]).any() and torch.isfinite(out[[0, 1, 3, 4, 5]]).all()
