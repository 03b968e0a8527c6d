"""One workspace of the grouped products for batches of any size up to the largest."""
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("E,N,K", [(2, 1024, 4096), (1, 256, 7168), (2, 2056, 2064), (4, 88, 2072)])
def test_workspace_of_the_largest_batch_does_for_smaller_ones(M, E, N, K):
    most = 4096
    ws = M.workspace(M.grouped_mm_workspace_size(most, E, N, K))
    x, dy, w = randn(1, most, K), randn(2, most, N), randn(3, E, N, K)
    for R in (1, 20, 33, 70, 100, 300, 512, 1000, 2048, most):
        off = torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32).cuda()
        xs, ds = x[:R], dy[:R]
        for fn, a, b in ((M.grouped_mm, xs, w), (M.grouped_mm_dx, ds, w), (M.grouped_mm_dw, ds, xs)):
            assert torch.equal(fn(a, b, off, ws=ws), fn(a, b, off)), (fn, R)
    assert M.get_device_error(ws) == M.MOE_OK


def test_a_product_asks_for_its_own_shares_only(M):
    """The few-rows product has none; dx of the same rows has, and is refused without room for them."""
    R, E, N, K = 24, 1, 4096, 256
    x, dy, w = randn(1, R, K), randn(2, R, N), randn(3, E, N, K)
    off, ws = torch.tensor([0, R], dtype=torch.int32).cuda(), M.workspace(256)
    assert M.grouped_mm_workspace_size(R, E, N, K) > 256
    assert torch.equal(M.grouped_mm(x, w, off, ws=ws), M.grouped_mm(x, w, off))
    with pytest.raises(M.MoeError, match="WORKSPACE"):
        M.grouped_mm_dx(dy, w, off, ws=ws)


def test_an_output_that_does_not_fit_is_out_of_memory(M):
    """As everywhere in torch, so that a caller may free memory and try again."""
    E, N, K = 1024, 32768, 32768  # 2 TiB of gradients
    x, dy = torch.empty(0, K, dtype=torch.bfloat16, device="cuda"), torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        M.grouped_mm_dw(dy, x, off)
    assert M.grouped_mm_dw(dy[:, :64].contiguous(), x[:, :64].contiguous(), off).shape == (E, 64, 64)


@pytest.mark.parametrize("D", [136, 2048, 4104])
@pytest.mark.parametrize("gates", [1, 2])
def test_norm_gradients_workspace_of_the_largest_batch_does_for_smaller_ones(M, D, gates):
    most = 4096
    ws = M.workspace(M.block_norm_backward_workspace_size(most, D, gates))
    x, y, dxo, dh = (randn(i, most, D) for i in range(4))
    post, pre, gate = randn(5, D), randn(6, D), randn(7, gates, D)
    for T in (2, 150, 304, 306, 456, 1000, most):
        args = (x[:T], y[:T], dxo[:T], dh[:T], post, gate, pre)
        got, want = M.block_norm_backward(*args, ws=ws), M.block_norm_backward(*args)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), T
