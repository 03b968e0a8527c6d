"""The operators of expert blocks in 8 and 16 bits refuse bad arguments on the host,
before any launch (no GPU needed).

Every call here that carries made-up pointers is one the library must reject
or that has nothing to do, so nothing is ever launched with them.
"""
import pytest

from tests.util import build_lib

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BF16, F16, F32 = 0, 1, 2
P = 0x100000  # 16-byte aligned, never dereferenced
BIG = 1 << 40
ROWS = 2 ** 31 - 2 ** 24  # one more than there may be


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


def test_layer_norm_rejects_bad_arguments(M):
    def call(dt=BF16, pt=BF16, T=4, D=64, eps=1e-5, gamma=P, beta=P, x=P, y=P, x_out=P, h=P):
        return M.lib().moe_layer_norm(dt, pt, T, D, eps, gamma, beta, x, y, x_out, h, None)

    assert call(T=-1) == INVALID
    assert call(D=0) == INVALID
    for eps in (0.0, -1e-5, float("inf"), float("nan")):
        assert call(eps=eps) == INVALID
    assert call(dt=3) == UNSUPPORTED
    assert call(pt=F16) == UNSUPPORTED          # neither the rows' type nor fp32
    assert call(D=60) == UNSUPPORTED
    assert call(D=16392) == UNSUPPORTED
    assert call(T=ROWS) == UNSUPPORTED
    for hole in ("x", "y", "x_out", "h"):
        assert call(**{hole: None}) == INVALID, hole
    for hole in ("gamma", "beta", "x", "y", "x_out", "h"):
        assert call(**{hole: P + 8}) == MISALIGNED, hole
    assert call(T=0) == OK
    assert call(T=0, x=None, h=None) == OK


def test_layer_norm_backward_rejects_bad_arguments(M):
    def call(dt=BF16, pt=F32, T=4, D=64, eps=1e-5, gamma=P, x=P, dh=P, dxo=P, dx=P, dg=P, db=P, ws=P, wsb=BIG):
        return M.lib().moe_layer_norm_backward(dt, pt, T, D, eps, gamma, x, dh, dxo, dx, dg, db, ws, wsb, None)

    assert call(T=-1) == INVALID
    assert call(D=0) == INVALID
    assert call(eps=0.0) == INVALID
    assert call(D=12) == UNSUPPORTED
    assert call(dt=F16, pt=BF16) == UNSUPPORTED
    assert call(gamma=None) == INVALID          # dgamma has its parameter
    for hole in ("x", "dh", "dx", "ws"):
        assert call(**{hole: None}) == INVALID, hole
    for hole in ("gamma", "x", "dh", "dxo", "dx", "dg", "db", "ws"):
        assert call(**{hole: P + 4}) == MISALIGNED, hole
    need = M.layer_norm_backward_workspace_size(4, 64)
    assert need > 256
    assert call(wsb=need - 1) == WORKSPACE
    assert M.layer_norm_backward_workspace_size(-1, 64) == 0
    assert M.layer_norm_backward_workspace_size(4, 0) == 0
    sizes = [M.layer_norm_backward_workspace_size(t, 64) for t in range(0, 1000, 13)]
    assert sizes == sorted(sizes)


def test_quantize_rows_rejects_bad_arguments(M):
    def call(dt=BF16, x=P, m=P, k=2, T=8, R=16, D=64, codes=P, scales=P, ws=P, wsb=BIG):
        return M.lib().moe_quantize_rows(dt, x, m, k, T, R, D, codes, scales, ws, wsb, None)

    assert call(T=-1) == INVALID
    assert call(R=-1) == INVALID
    assert call(D=0) == INVALID
    assert call(k=0) == INVALID
    assert call(m=None) == INVALID              # as many rows as x has, without a map
    assert call(dt=3) == UNSUPPORTED
    assert call(D=40) == UNSUPPORTED
    assert call(D=32784) == UNSUPPORTED
    assert call(R=ROWS) == UNSUPPORTED
    assert call(T=ROWS) == UNSUPPORTED
    for hole in ("x", "codes", "scales"):
        assert call(**{hole: None}) == INVALID, hole
    for hole in ("x", "m", "codes", "scales", "ws"):
        assert call(**{hole: P + 8}) == MISALIGNED, hole
    need = M.quantize_rows_workspace_size(1000, 9000, 2048)
    assert need >= 1000 * (2048 + 4)
    assert call(T=1000, R=9000, D=2048, k=9, wsb=need - 1) == WORKSPACE
    for sizes in ((8000, 8000, 2048), (500, 4000, 2048), (1000, 8000, 2056), (0, 8, 64), (8, -1, 64), (8, ROWS, 64), (2, 4, 64)):
        assert M.quantize_rows_workspace_size(*sizes) == 0
    assert call(R=0) == OK
    assert call(R=0, x=None, codes=None, scales=None) == OK


def test_grouped_mm_i8_rejects_bad_arguments(M):
    def call(dt=BF16, x=P, xs=P, w=P, ws=P, off=P, R=64, E=8, N=64, K=64, y=P, space=P, wsb=BIG):
        return M.lib().moe_grouped_mm_i8(dt, x, xs, w, ws, off, R, E, N, K, y, space, wsb, None)

    assert call(R=-1) == INVALID
    assert call(E=0) == INVALID
    assert call(E=1025) == INVALID
    assert call(N=0) == INVALID
    assert call(K=0) == INVALID
    assert call(dt=F32) == UNSUPPORTED
    assert call(N=60) == UNSUPPORTED
    assert call(K=40) == UNSUPPORTED            # a multiple of 8, not of 16
    assert call(N=32776) == UNSUPPORTED
    assert call(K=32784) == UNSUPPORTED
    assert call(R=ROWS) == UNSUPPORTED
    for hole in ("x", "xs", "w", "ws", "off", "y", "space"):
        assert call(**{hole: None}) == INVALID, hole
        assert call(**{hole: P + 8}) == MISALIGNED, hole
    need = M.grouped_mm_i8_workspace_size(64, 8, 64, 64)
    assert call(wsb=need - 1) == WORKSPACE
    assert call(R=0, x=None, xs=None, w=None, ws=None, y=None) == OK
    assert M.grouped_mm_i8_workspace_size(-1, 8, 64, 64) == 0
    assert M.grouped_mm_i8_workspace_size(16, 8, 64, 64) >= 256


def test_python_refuses_other_types_and_shapes(M):
    torch = pytest.importorskip("torch")
    bf = dict(dtype=torch.bfloat16)
    x = torch.zeros(4, 64, **bf)
    i8 = torch.zeros(4, 64, dtype=torch.int8)
    w = torch.zeros(2, 8, 64, dtype=torch.int8)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: M.layer_norm(torch.zeros(4, 64, dtype=torch.float64)),
                 lambda: M.layer_norm(torch.zeros(64, **bf)),
                 lambda: M.layer_norm(x, torch.zeros(4, 32, **bf)),
                 lambda: M.layer_norm(x, gamma=torch.zeros(32, **bf)),
                 lambda: M.layer_norm(x, gamma=torch.zeros(64, **bf), beta=torch.zeros(64)),
                 lambda: M.layer_norm_backward(x, torch.zeros(4, 64)),
                 lambda: M.quantize_rows(i8),
                 lambda: M.quantize_rows(x, torch.zeros(4, dtype=torch.int64)),
                 lambda: M.quantize_rows(x, torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: M.grouped_mm_i8(x, torch.zeros(4), w, torch.zeros(2, 8), off),
                 lambda: M.grouped_mm_i8(i8, torch.zeros(4), w, torch.zeros(2, 16), off),
                 lambda: M.grouped_mm_i8(i8, torch.zeros(4, **bf), w, torch.zeros(2, 8), off),
                 lambda: M.grouped_mm_i8(i8, torch.zeros(4), w, torch.zeros(2, 8), off, dtype=torch.float64),
                 lambda: M.grouped_mm_i8(i8, torch.zeros(4), w, torch.zeros(2, 8), off),   # host tensors
                 lambda: M.layer_norm(x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        M.grouped_mm_i8(i8, torch.zeros(4), w, torch.zeros(2, 8), off, dtype="bfloat16")
    with pytest.raises(TypeError):
        M.quantize_rows(x, k=1.5)


def test_expert_layer_rejects_bad_arguments(M):
    def call(dt=BF16, x=P, lg=P, w13=P, w2=P, T=4, k=2, E=8, d=128, f=64, out=P, ids=P, ws=P, wsb=BIG):
        return M.lib().moe_expert_layer(dt, x, lg, w13, w2, T, k, E, d, f, out, ids, ws, wsb, None)

    assert call(T=-1) == INVALID
    assert call(k=0) == INVALID
    assert call(k=9) == INVALID                 # more than the experts
    assert call(E=0) == INVALID
    assert call(E=1025) == INVALID
    assert call(d=0) == INVALID
    assert call(f=-64) == INVALID
    assert call(dt=F32) == UNSUPPORTED
    assert call(T=33) == UNSUPPORTED
    assert call(T=2 ** 31 - 1) == UNSUPPORTED
    assert call(T=32, k=9, E=64) == UNSUPPORTED
    assert call(T=1, k=33, E=64) == UNSUPPORTED
    assert call(d=96) == UNSUPPORTED
    assert call(f=32) == UNSUPPORTED
    assert call(d=32832) == UNSUPPORTED
    assert call(f=32832) == UNSUPPORTED
    for hole in ("x", "lg", "w13", "w2", "out", "ws"):
        assert call(**{hole: None}) == INVALID, hole
    for hole in ("x", "lg", "w13", "w2", "out", "ids", "ws"):
        assert call(**{hole: P + 8}) == MISALIGNED, hole
    need = M.expert_layer_workspace_size(4, 2, 8, 128, 64)
    assert need > 256
    assert call(wsb=need - 1) == WORKSPACE
    assert call(T=0, x=None, lg=None, w13=None, w2=None, out=None) == OK
    assert M.expert_layer_workspace_size(33, 2, 8, 128, 64) == 0
    assert M.expert_layer_workspace_size(4, 2, 8, 100, 64) == 0
    assert M.expert_layer_workspace_size(4, 0, 8, 128, 64) == 0


def test_python_expert_layer_refuses(M):
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    x, lg, w13, w2 = z(4, 64), z(4, 8, t=torch.float32), z(8, 128, 64), z(8, 64, 64)
    for call in (lambda: M.expert_layer(x, lg, w13, w2, 2),                         # host tensors
                 lambda: M.expert_layer(x, z(4, 8), w13, w2, 2),
                 lambda: M.expert_layer(x, z(3, 8, t=torch.float32), w13, w2, 2),
                 lambda: M.expert_layer(x, lg, z(8, 64, 64), w2, 2),
                 lambda: M.expert_layer(x, lg, w13, z(8, 64, 64, t=torch.float16), 2),
                 lambda: M.expert_layer(x, lg, w13, w2, 2, ids=z(4, 3, t=torch.int32)),
                 lambda: M.expert_layer(z(64), lg, w13, w2, 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        M.expert_layer(x, lg, w13, w2)
    with pytest.raises(TypeError):
        M.expert_layer(x, lg, w13, w2, None)
