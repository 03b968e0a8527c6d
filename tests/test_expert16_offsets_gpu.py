"""Offsets out of place: nothing is computed and nothing written, in the tensor-core
kernels and in the one for few rows, and the error word says so."""
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


@pytest.mark.parametrize("R", [24, 40])  # y by the few-rows kernel, and by the tiles
@pytest.mark.parametrize("where", ["falls", "beyond", "negative", "far", "last"])
def test_nothing_is_written_where_a_segment_is_out_of_place(M, R, where):
    N, K, E = 64, 64, 4
    off = [0, 5, 12, 20, R]
    if where == "falls":
        off[2] = 3
    elif where == "beyond":
        off[4] = R + 1
    elif where == "negative":
        off[0] = -1
    elif where == "far":
        off[3] = 2 ** 30
    else:
        off[3], off[4] = R, R - 1
    x, dy, w = randn(1, R, K), randn(2, R, N), randn(3, E, N, K)
    od = torch.tensor(off, dtype=torch.int32).cuda()
    ws = M.workspace(M.grouped_mm_workspace_size(R, E, N, K))
    assert ws.numel() == 256  # no shares: the products write their outputs themselves
    for fn, a, b, shape in ((M.grouped_mm, x, w, (R, N)), (M.grouped_mm_dx, dy, w, (R, K)), (M.grouped_mm_dw, dy, x, (E, N, K))):
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        fn(a, b, od, out, ws)
        assert M.STATUS[M.get_device_error(ws)] == "MOE_ERR_DEVICE_RANGE"
        assert (out == 7).all(), fn
    good = torch.tensor([0, 5, 12, 20, R], dtype=torch.int32).cuda()
    y = M.grouped_mm(x, w, good, ws=ws)  # and the next call is not affected
    assert M.get_device_error(ws) == M.MOE_OK and torch.isfinite(y).all()


@pytest.mark.parametrize("counts,N,K", [([70], 88, 2072), ([40], 2056, 136), ([2100], 96, 80), ([60, 59], 2056, 2064)])
def test_shared_out_sums_write_nothing_where_a_segment_is_out_of_place(M, counts, N, K):
    """Nor what an earlier call left in the workspace."""
    R, E = sum(counts), len(counts)
    x, dy, w = randn(1, R, K), randn(2, R, N), randn(3, E, N, K)
    good = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(E)], dtype=torch.int32).cuda()
    bad = good.clone()
    bad[0] = 5
    bad[-1] = R + 1
    ws = M.workspace(M.grouped_mm_workspace_size(R, E, N, K))
    assert ws.numel() > 256
    for fn, a, b in ((M.grouped_mm, x, w), (M.grouped_mm_dx, dy, w), (M.grouped_mm_dw, dy, x)):
        want = fn(a, b, good, ws=ws)
        out = torch.full_like(want, 7.0)
        fn(a, b, bad, out, ws)
        assert M.STATUS[M.get_device_error(ws)] == "MOE_ERR_DEVICE_RANGE"
        assert (out == 7).all(), fn
        assert torch.equal(fn(a, b, good, ws=ws), want)
