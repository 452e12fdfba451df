"""The sequence-block operators in streams of calls: results of one call feed the
next without a pause between, directly and from a captured graph.  Every kernel is
launched while the one before it still runs, so a missing wait shows here as
other bits than those of calls made one at a time."""

import pytest

from tests import harness

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    harness.ensure_built()


def block(dtype, M, H, F):
    """A chain of the operators, [M, H] -> [M, H]; returns (step, outputs): step(sync)
    runs it, with a synchronisation after every call if asked."""
    import torch
    from layer_rnn_gb300 import binding
    ops = binding.Ops(dtype)
    dt = ops.tdtype
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: (torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5).to(dt)  # noqa: E731
    new = lambda *s, t=dt: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    x, W = rnd(M, H) * H ** 0.5, rnd(2 * F, H)
    q4 = [ops.w4_alloc(r, c, 32, zeros=True) for r, c in ((3 * H, F), (H, H))]
    src = [rnd(3 * H, F), rnd(H, H)]
    y, gx, h0, hy, s = new(M, F), new(M, 3 * H), new(1, 1, H, t=torch.float32), new(1, 1, H, t=torch.float32), new(M, H)
    dx, dW, out = new(M, H), new(2 * F, H), new(M, H)
    ws = new(ops.glu_workspace_bytes(M, H, F, backward=True), t=torch.uint8)
    sws = new(ops.scan_workspace_bytes(M, 1, H), t=torch.uint8)
    dgx, dh0 = new(M, 3 * H), new(1, 1, H, t=torch.float32)

    def step(sync=False, stream=None):
        calls = [
            lambda: ops.w4_quantize(src[0], q4[0][0], q4[0][1], 32, q4[0][2], stream=stream),
            lambda: ops.w4_quantize(src[1], q4[1][0], q4[1][1], 32, q4[1][2], stream=stream),
            lambda: ops.glu_forward(x, W, y, ws, stream=stream),
            lambda: ops.w4_matvec(y, q4[0][0], q4[0][1], gx, 32, q4[0][2], stream=stream),
            lambda: ops.scan_forward(gx.view(M, 1, 3 * H), h0, s.view(M, 1, H), hy, ws=sws, out_gate=True, stream=stream),
            lambda: ops.w4_matvec(s, q4[1][0], q4[1][1], out, 32, q4[1][2], stream=stream),
            lambda: ops.scan_backward(gx.view(M, 1, 3 * H), s.view(M, 1, H), hy, dgx.view(M, 1, 3 * H), dh0, sws,
                                      out_gate=True, stream=stream),
            lambda: ops.glu_backward(x, W, y, dx, dW, ws, stream=stream),
            lambda: ops.scan_step(dgx, state, state, s, out_gate=True, stream=stream),
        ]
        for c in calls:
            c()
            if sync:
                torch.cuda.synchronize()

    state = new(M, H, t=torch.float32)
    return step, dict(y=y, gx=gx, hy=hy, s=s, out=out, dgx=dgx, dh0=dh0, dx=dx, dW=dW, state=state), ops


def bits(outputs):
    return {k: v.detach().clone() for k, v in outputs.items()}


def reset(outputs):
    for v in outputs.values():
        v.zero_()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,H,F", [(1, 64, 96), (20, 136, 200), (100, 64, 72), (300, 328, 520), (90, 37, 51)])
def test_calls_in_a_row_and_in_a_graph_give_the_same_bits(M, H, F, dtype):
    import torch
    step, outputs, ops = block(dtype, M, H, F)
    reset(outputs)
    torch.cuda.synchronize()
    step(sync=True)
    want = bits(outputs)
    for _ in range(3):
        reset(outputs)
        step()
        torch.cuda.synchronize()
        got = bits(outputs)
        assert all(torch.equal(got[k], want[k]) for k in want), [k for k in want if not torch.equal(got[k], want[k])]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        reset(outputs)
        step()
    for _ in range(3):
        reset(outputs)
        g.replay()
        torch.cuda.synchronize()
        got = bits(outputs)
        assert all(torch.equal(got[k], want[k]) for k in want), [k for k in want if not torch.equal(got[k], want[k])]
    assert ops.check_status() == 0
