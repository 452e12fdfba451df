"""Host-side checks of the sequence-block operators' entry points: sizes,
workspaces and refusals, all before anything touches a device (CPU)."""

import ctypes
import os

import pytest

from tests import harness

OK, INVALID, UNSUPPORTED, SMALL, MISALIGNED = 0, 1, 2, 3, 4
P, ODD = 1 << 20, (1 << 20) + 8  # addresses that are never read


@pytest.fixture(scope="module")
def L():
    if not os.path.exists("/usr/local/cuda/bin/nvcc") and not os.path.exists(
            os.path.join(harness.ROOT, "layer_rnn_gb300", "liblayer_rnn.so")):
        pytest.skip("no nvcc and no prebuilt library")
    harness.ensure_built()
    from layer_rnn_gb300 import binding
    return binding.lib()


@pytest.fixture(params=[0, 1], ids=["f32", "bf16"])
def h(L, request):
    p = ctypes.c_void_p()
    assert L.rnn_ops_create(ctypes.byref(p), request.param, 0) == OK
    yield p
    assert L.rnn_ops_destroy(p) == OK


def test_create_refuses(L):
    p = ctypes.c_void_p()
    assert L.rnn_ops_create(None, 0, 0) == INVALID
    assert L.rnn_ops_create(ctypes.byref(p), 2, 0) == INVALID
    assert L.rnn_ops_create(ctypes.byref(p), 0, 0x2) == INVALID  # a flag of the recurrent layers
    assert p.value is None
    assert L.rnn_ops_destroy(None) == OK
    assert L.rnn_ops_check_status(None, None) == INVALID


def test_scan_workspace(L, h):
    b = ctypes.c_int64()
    size = lambda T, N, H, D: (L.rnn_scan_workspace_size(h, T, N, H, D, ctypes.byref(b)), b.value)  # noqa: E731
    assert size(64, 2, 8, 1) == (OK, 256) and size(65, 2, 8, 1) == (OK, 256)
    assert size(6400, 3, 100, 2) == (OK, 100 * 3 * 100 * 2 * 4 + 0 if 240000 % 256 == 0 else 240128)
    assert size(0, 1, 1, 1)[0] == INVALID and size(1, 1, 1, 3)[0] == INVALID
    assert size(1, 1 << 16, 1 << 15, 1)[0] == UNSUPPORTED
    assert L.rnn_scan_workspace_size(h, 1, 1, 1, 1, None) == INVALID
    assert L.rnn_scan_workspace_size(None, 1, 1, 1, 1, ctypes.byref(b)) == INVALID


def test_scan_forward_refuses(L, h):
    def call(T=4, N=2, H=8, D=1, gate=0, lengths=None, gx=P, ldg=0, h0=None, y=P, ldy=0, hy=None,
             ws=None, nb=0):
        return L.rnn_scan_forward(h, None, T, N, H, D, gate, lengths, gx, ldg, h0, y, ldy, hy, ws, nb)

    for bad in (dict(T=0), dict(N=0), dict(H=0), dict(D=0), dict(D=3), dict(gate=2), dict(gx=None),
                dict(y=None), dict(ldg=15), dict(ldy=7), dict(ldg=-16)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(gx=ODD), dict(y=ODD), dict(h0=ODD), dict(hy=ODD), dict(ws=ODD, nb=1 << 20),
                dict(lengths=P + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(ws=P, nb=63) == SMALL
    assert call(T=1 << 31) == UNSUPPORTED and call(N=1 << 20, H=1 << 11) == UNSUPPORTED


def test_scan_backward_and_step_refuse(L, h):
    def call(T=4, N=2, H=8, D=1, gate=0, lengths=None, gx=P, ldg=0, dy=P, ldy=0, dhy=None, dgx=P,
             dh0=None, ws=P, nb=1 << 20):
        return L.rnn_scan_backward(h, None, T, N, H, D, gate, lengths, gx, ldg, dy, ldy, dhy, dgx, dh0,
                                   ws, nb)

    for bad in (dict(T=0), dict(gx=None), dict(dy=None), dict(dgx=None), dict(ws=None), dict(D=4)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dgx=ODD), dict(dh0=ODD), dict(dhy=ODD), dict(dy=ODD)):
        assert call(**bad) == MISALIGNED, bad
    assert call(nb=63) == SMALL
    step = lambda N=2, H=8, gate=0, gx=P, ldg=0, a=P, b=P, y=P, ldy=0: L.rnn_scan_step(  # noqa: E731
        h, None, N, H, gate, gx, ldg, a, b, y, ldy)
    assert step(N=0) == INVALID and step(a=None) == INVALID and step(b=None) == INVALID
    assert step(gx=None) == INVALID and step(ldg=1) == INVALID and step(a=ODD) == MISALIGNED


def test_w4_refuses(L, h):
    bf = 1 if ctypes.cast(h, ctypes.POINTER(ctypes.c_int))[0] == 1 else 0  # the handle starts with its type

    def call(M=1, R=4, K=64, group=32, x=P, q=P, ldq=0, s=P, z=None, y=P):
        return L.rnn_w4_matvec(h, None, M, R, K, group, x, q, ldq, s, z, y)

    for bad in (dict(M=0), dict(R=0), dict(K=0), dict(group=16), dict(group=0), dict(x=None), dict(q=None),
                dict(s=None), dict(y=None), dict(ldq=16), dict(ldq=33), dict(ldq=40)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=ODD), dict(q=ODD), dict(y=ODD), dict(s=P + (1 if bf else 2))):
        assert call(**bad) == MISALIGNED, bad
    assert call(K=65537) == UNSUPPORTED and call(R=1 << 31) == UNSUPPORTED
    quant = lambda R=4, K=64, group=32, W=P, q=P, ldq=0, s=P, z=None: L.rnn_w4_quantize(  # noqa: E731
        h, None, R, K, group, W, q, ldq, s, z)
    assert quant(W=None) == INVALID and quant(group=8) == INVALID and quant(W=ODD) == MISALIGNED


def test_w4_refuses_pitches_beyond_its_offsets(L, h):
    call = lambda R, ldq: L.rnn_w4_matvec(h, None, 1, R, 64, 32, P, P, ldq, P, None, P)  # noqa: E731
    assert call(4, (1 << 22) + 16) == UNSUPPORTED and call(4, 1 << 40) == UNSUPPORTED
    assert call((1 << 31) - 1024, 0) == UNSUPPORTED
    assert L.rnn_w4_quantize(h, None, 4, 64, 32, P, P, (1 << 22) + 16, P, None) == UNSUPPORTED


def test_glu_workspace_and_refusals(L, h):
    b = ctypes.c_int64()
    size = lambda M, K, F, bwd: (L.rnn_glu_workspace_size(h, M, K, F, bwd, ctypes.byref(b)), b.value)  # noqa: E731
    assert size(1, 64, 64, 0) == (OK, 256)
    assert size(1000, 64, 64, 1)[1] >= size(1000, 64, 64, 0)[1] >= 256
    assert size(1000, 64, 64, 1)[1] >= 2 * 1000 * 64 * 2
    for bad in ((0, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (1, 1, 1, 2)):
        assert size(*bad)[0] == INVALID
    assert size(1 << 24, 1, 1, 0)[0] == UNSUPPORTED and size(1, 1, 1 << 23, 0)[0] == UNSUPPORTED

    def fwd(M=4, K=8, F=8, act=0, x=P, W=P, y=P, ws=P, nb=1 << 40):
        return L.rnn_glu_forward(h, None, M, K, F, act, x, W, y, ws, nb)

    def bwd(M=4, K=8, F=8, act=0, x=P, W=P, dy=P, dx=P, dW=P, ws=P, nb=1 << 40):
        return L.rnn_glu_backward(h, None, M, K, F, act, x, W, dy, dx, dW, ws, nb)

    for call in (fwd, bwd):
        for bad in (dict(M=0), dict(K=-1), dict(F=0), dict(act=3), dict(act=-1), dict(x=None), dict(W=None),
                    dict(ws=None)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(x=ODD), dict(W=ODD), dict(ws=P + 16)):
            assert call(**bad) == MISALIGNED, bad
        assert call(M=1 << 25) == UNSUPPORTED
        assert call(M=300, nb=255) == SMALL
    assert fwd(y=None) == INVALID and fwd(y=ODD) == MISALIGNED
    assert bwd(dy=None) == INVALID and bwd(dx=None, dW=None) == INVALID and bwd(dW=ODD) == MISALIGNED
