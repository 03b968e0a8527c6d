"""Calls of the layer norm's gradients that the header allows: over their inputs, captured and
replayed with other inputs, on two streams, and in a workspace for more rows."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_expert_block_ops_gpu import BF16, F16, F32, randn  # noqa: E402
from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

CODE = {BF16: 0, F16: 1, F32: 2}


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(3, 2048), (700, 768), (1213, 2048), (311, 7168), (5, 16384), (400, 8200)])
@pytest.mark.parametrize("over", ["dh", "dx_out"])
def test_gradients_in_place(M, T, D, dtype, over):
    x, dh, dxo = randn(1, dtype, T, D).cuda(), randn(2, dtype, T, D).cuda(), randn(3, dtype, T, D).cuda()
    gamma, beta = randn(4, dtype, D).cuda(), randn(5, dtype, D).cuda()
    want = M.layer_norm_backward(x, dh, dxo, gamma, beta)
    ws = M.workspace(M.layer_norm_backward_workspace_size(T, D))
    dx = dh if over == "dh" else dxo
    dg, db = torch.empty_like(gamma), torch.empty_like(beta)
    torch.cuda.synchronize()
    assert M.lib().moe_layer_norm_backward(CODE[dtype], CODE[dtype], T, D, 1e-5, gamma.data_ptr(), x.data_ptr(), dh.data_ptr(),
                                           dxo.data_ptr(), dx.data_ptr(), dg.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(),
                                           torch.cuda.current_stream().cuda_stream) == M.MOE_OK
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), want))


@pytest.mark.parametrize("T,D", [(7, 4096), (1213, 2048)])
def test_gradients_as_a_graph_and_on_two_streams(M, T, D):
    gamma, beta = randn(4, BF16, D).cuda(), randn(5, BF16, D).cuda()
    inputs = [[randn(10 * i + j, BF16, T, D).cuda() for j in range(3)] for i in range(3)]
    wants = [M.layer_norm_backward(*a, gamma, beta) for a in inputs]
    spaces = [M.workspace(M.layer_norm_backward_workspace_size(4096, D)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in spaces]
    torch.cuda.synchronize()
    outs = [(M.layer_norm_backward(*inputs[i % 3], gamma, beta, ws=ws, stream=s), wants[i % 3])
            for i in range(12) for s, ws in zip(streams, spaces)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got, want in outs for a, b in zip(got, want))
    held = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        got = M.layer_norm_backward(*held, gamma, beta, ws=spaces[0])
    for i in (0, 1, 2, 0):
        for a, b in zip(held, inputs[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, wants[i]))
