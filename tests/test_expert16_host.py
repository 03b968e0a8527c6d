"""The 16-bit expert operators refuse bad arguments on the host, before any
launch (no GPU needed).

Every call here that carries made-up pointers is one the library must reject
or that has nothing to do, so nothing is ever launched with them.
"""
import pytest

from tests.util import build_lib

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BF16, F16, F32 = 0, 1, 2
P = 0x100000  # 16-byte aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


@pytest.mark.parametrize("fn", ["moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw"])
def test_grouped_products_reject_bad_arguments(M, fn):
    def call(dt=BF16, a=P, b=P, off=P, R=16, E=8, N=64, K=64, out=P, ws=P, wsb=BIG):
        return getattr(M.lib(), fn)(dt, a, b, off, R, E, N, K, out, ws, wsb, None)

    assert call(R=-1) == INVALID
    assert call(E=0) == INVALID
    assert call(E=1025) == INVALID
    assert call(N=0) == INVALID
    assert call(K=-8) == INVALID
    assert call(dt=F32) == UNSUPPORTED
    assert call(dt=7) == UNSUPPORTED
    assert call(N=60) == UNSUPPORTED            # not a multiple of 8
    assert call(K=4) == UNSUPPORTED
    assert call(N=32776) == UNSUPPORTED
    assert call(K=32776) == UNSUPPORTED
    for hole in ("a", "b", "off", "out", "ws"):
        assert call(**{hole: None}) == INVALID, hole
        assert call(**{hole: P + 8}) == MISALIGNED, hole
    assert call(wsb=255) == WORKSPACE
    assert call(R=0, off=None) == INVALID
    if fn != "moe_grouped_mm_dw":               # no rows: a no-op, nothing launched
        assert call(R=0) == OK
        assert call(R=0, a=None, b=None, out=None) == OK
    else:                                       # dw of no rows is zeros and has to be there
        assert call(R=0, out=None) == INVALID


def test_workspace_sizes(M):
    lib = M.lib()
    assert lib.moe_grouped_mm_workspace_size(16, 8, 64, 64) >= 256
    assert lib.moe_grouped_mm_workspace_size(-1, 8, 64, 64) == 0
    assert lib.moe_grouped_mm_workspace_size(16, 0, 64, 64) == 0
    assert lib.moe_block_norm_backward_workspace_size(16, 64, 4) > 256
    assert lib.moe_block_norm_backward_workspace_size(16, 64, 5) == 0
    assert lib.moe_block_norm_backward_workspace_size(16, 0, 1) == 0


def test_swiglu_rejects_bad_arguments(M):
    lib = M.lib()

    def fwd(dt=BF16, gu=P, w=P, m=P, R=4, F=64, h=P):
        return lib.moe_swiglu(dt, gu, w, m, R, F, h, None)

    def bwd(dt=BF16, dh=P, gu=P, w=P, m=P, R=4, F=64, dgu=P, dw=P):
        return lib.moe_swiglu_backward(dt, dh, gu, w, m, R, F, dgu, dw, None)

    for call in (fwd, bwd):
        assert call(R=-1) == INVALID
        assert call(F=0) == INVALID
        assert call(F=12) == UNSUPPORTED
        assert call(F=32776) == UNSUPPORTED
        assert call(dt=3) == UNSUPPORTED
        assert call(gu=None) == INVALID
        assert call(gu=P + 2) == MISALIGNED
        assert call(w=P + 4) == MISALIGNED
        assert call(m=P + 4) == MISALIGNED
        assert call(w=None) == INVALID           # a map without weights
        assert call(R=0) == OK
    assert fwd(h=None) == INVALID
    assert fwd(h=P + 8) == MISALIGNED
    assert bwd(dh=None) == INVALID
    assert bwd(dgu=None) == INVALID
    assert bwd(w=None, m=None) == INVALID        # a gradient of weights that are not there
    assert bwd(dw=P + 4) == MISALIGNED


def test_block_norm_rejects_bad_arguments(M):
    lib = M.lib()

    def fwd(dt=BF16, pt=BF16, T=4, D=64, G=1, alpha=1.0, eps=1e-6, post=P, gate=P, pre=P, x=P, y=P, xo=P, h=P):
        return lib.moe_block_norm(dt, pt, T, D, G, alpha, eps, post, gate, pre, x, y, xo, h, None)

    def bwd(dt=BF16, pt=BF16, T=4, D=64, G=1, alpha=1.0, eps=1e-6, post=P, gate=P, pre=P, x=P, y=P, dxo=P, dh=P, dx=P,
            dy=P, dpost=P, dgate=P, dpre=P, ws=P, wsb=BIG):
        return lib.moe_block_norm_backward(dt, pt, T, D, G, alpha, eps, post, gate, pre, x, y, dxo, dh, dx, dy, dpost,
                                           dgate, dpre, ws, wsb, None)

    for call in (fwd, bwd):
        assert call(T=-1) == INVALID
        assert call(D=0) == INVALID
        assert call(G=0) == INVALID
        assert call(G=3) == INVALID              # does not divide the rows
        assert call(eps=0.0) == INVALID
        assert call(eps=float("nan")) == INVALID
        assert call(alpha=float("inf")) == INVALID
        assert call(D=68) == UNSUPPORTED
        assert call(D=16392) == UNSUPPORTED
        assert call(dt=5) == UNSUPPORTED
        assert call(pt=F16) == UNSUPPORTED       # bf16 tensors take bf16 or fp32 parameters
        assert call(dt=F32, pt=BF16) == UNSUPPORTED
        assert call(y=None) == INVALID           # a norm and a gate of a block that is not there
        assert call(x=P + 8) == MISALIGNED
        assert call(gate=P + 8) == MISALIGNED
    assert fwd(x=None) == INVALID
    assert fwd(xo=None) == INVALID
    assert fwd(h=None) == INVALID                # gamma_pre without its output
    assert fwd(pre=None) == INVALID              # h without gamma_pre
    assert fwd(y=None, post=None, gate=None) == INVALID                               # x_out without y
    assert fwd(y=None, post=None, gate=None, xo=None, pre=None, h=None) == INVALID    # nothing wanted
    assert fwd(T=0) == OK
    assert bwd(dx=None) == INVALID
    assert bwd(dy=None) == INVALID
    assert bwd(dh=None) == INVALID
    assert bwd(pre=None, dpre=None) == INVALID   # dh without gamma_pre
    assert bwd(pre=None, dpre=None, dh=None, dxo=None) == INVALID                     # no gradient comes in
    assert bwd(post=None) == INVALID             # a gradient without its parameter
    assert bwd(gate=None) == INVALID
    assert bwd(ws=None) == INVALID
    assert bwd(wsb=256) == WORKSPACE
    assert bwd(T=0, dpost=None, dgate=None, dpre=None) == OK


def test_binding_checks_shapes_and_types(M):
    """Shapes and types are refused before any library call, host tensors too."""
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    x, w, dy, off = z(4, 16), z(2, 24, 16), z(4, 24), i32(3)
    ws = torch.zeros(1024, dtype=torch.uint8)
    for call in (
            lambda: M.grouped_mm(x, z(2, 24, 8), off, ws=ws),                     # K differs
            lambda: M.grouped_mm(x, w.half(), off, ws=ws),                        # types differ
            lambda: M.grouped_mm(x, w, i32(4), ws=ws),                            # offsets of another E
            lambda: M.grouped_mm(x, w, off.long(), ws=ws),
            lambda: M.grouped_mm(x, w, off, y=z(4, 16), ws=ws),
            lambda: M.grouped_mm(x.double(), w.double(), off, ws=ws),
            lambda: M.grouped_mm_dx(dy, z(2, 16, 16), off, ws=ws),
            lambda: M.grouped_mm_dw(dy, z(5, 16), off, ws=ws),
            lambda: M.grouped_mm_dw(dy, x, off, dw=z(2, 16, 24), ws=ws),
            lambda: M.swiglu(z(4, 15)),
            lambda: M.swiglu(z(4, 16), z(4)),                                     # weights not fp32
            lambda: M.swiglu(z(4, 16), z(5, dt=torch.float32)),
            lambda: M.swiglu_backward(z(4, 16), z(4, 16)),
            lambda: M.block_norm(x, z(4, 8), z(16), None, z(16)),
            lambda: M.block_norm(x, x, z(8)),
            lambda: M.block_norm(x, x, z(16), z(3, 16), z(16)),                   # 3 does not divide 4
            lambda: M.block_norm(x, x, z(16), None, z(16, dt=torch.float32)),     # parameters of two types
            lambda: M.block_norm_backward(x, x, x.float(), x, z(16), None, z(16)),
            lambda: M.grouped_mm(x, w, off, ws=ws),                               # host tensors
            lambda: M.swiglu(z(4, 16)),
            lambda: M.block_norm(x, x, z(16), None, z(16))):
        with pytest.raises(ValueError):
            call()


def test_binding_rejects_strided_tensors(M):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="contiguous|device"):
        M.swiglu(torch.zeros(32, 4).t())
