"""The gated linear recurrence on the GPU against its float64 form.

Bars (largest error over the largest value of the reference).  float32: a
step rounds a few times (2^-24 each, about 4) and the state forgets at the rate
1 - f, so errors of up to 1 / (1 - f) steps pile up; f <= 0.99 at these inputs
gives 4 * 100 * 2^-24 = 2.4e-5 at worst.  Gradients multiply two such
quantities: 5e-5.  bfloat16: one rounding of the result, 2^-9 of the value,
and the float32 error: 2^-8.
"""

import numpy as np
import pytest

from tests import harness
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
F32, GRAD, BF16 = 2.4e-5, 5e-5, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    harness.ensure_built()


def data(T, N, H, D, gate, dtype, seed):
    rng = np.random.default_rng(seed)
    G = 3 if gate else 2
    gx = rng.standard_normal((T, N, D, G, H))
    gx[:, :, :, 0] = np.clip(gx[:, :, :, 0] + 1.5, -4, 4)
    r = lambda a: harness.from_dev(harness.to_dev(a, dtype))  # noqa: E731  rounded to storage
    f = lambda *s: rng.standard_normal(s).astype(np.float32).astype(np.float64)  # noqa: E731
    return dict(gx=r(gx.reshape(T, N, D * G * H)), h0=f(D, N, H), dy=r(rng.standard_normal((T, N, D * H))),
                dhy=f(D, N, H))


def run_gpu(i, D, gate, dtype, lengths=None, state=True, poison=False, pad=0, stream=None):
    """Forward and backward through the binding; rows `pad` elements apart
    from dense where asked."""
    import torch
    from layer_rnn_gb300 import binding
    ops = binding.Ops(dtype)
    T, N, W = i["gx"].shape
    H = W // (D * (3 if gate else 2))
    gx, dy = harness.to_dev(i["gx"], dtype), harness.to_dev(i["dy"], dtype)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if poison:  # what lies past a sequence's length is never looked at
        for n, ln in enumerate(lengths):
            gx[max(0, ln):, n] = float("nan")
            dy[max(0, ln):, n] = float("inf")

    def strided(t):
        if not pad:
            return t
        w = torch.full((*t.shape[:-1], t.shape[-1] + pad), 7.0, dtype=t.dtype, device="cuda")
        w[..., :t.shape[-1]] = t
        return w[..., :t.shape[-1]]

    gx, dy = strided(gx), strided(dy)
    y, dgx = strided(torch.empty_like(dy.contiguous())), strided(torch.empty_like(gx.contiguous()))
    new = lambda: torch.empty((D, N, H), dtype=torch.float32, device="cuda")  # noqa: E731
    up = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda") if state else None  # noqa: E731
    h0, dhy, hy, dh0 = up(i["h0"]), up(i["dhy"]), new(), new()
    ws = torch.empty(ops.scan_workspace_bytes(T, N, H, D), dtype=torch.uint8, device="cuda")
    yi = torch.empty_like(y.contiguous())
    torch.cuda.synchronize()
    ops.scan_forward(gx, h0, y, hy, lengths=lens, ws=ws, out_gate=gate, stream=stream)
    ops.scan_forward(gx, h0, yi, hy, lengths=lens, out_gate=gate, stream=stream)
    ops.scan_backward(gx, dy, dhy, dgx, dh0, ws, lengths=lens, out_gate=gate, stream=stream)
    torch.cuda.synchronize()
    assert ops.check_status() == 0
    assert torch.equal(yi.view(torch.uint8), y.contiguous().view(torch.uint8)), "inference and training forwards agree bit for bit"
    if pad:
        for t in (y, dgx):
            assert (t._base[..., t.shape[-1]:] == 7.0).all(), "the gap between rows is untouched"
    return {k: harness.from_dev(v.contiguous()) for k, v in dict(y=y, hy=hy, dgx=dgx, dh0=dh0).items()}


def check(i, out, D, gate, dtype, lengths=None, state=True):
    h0, dhy = (i["h0"], i["dhy"]) if state else (None, None)
    y, hy, tape = ref.scan(i["gx"], h0, D, gate, lengths)
    dgx, dh0 = ref.scan_backward(i["gx"], tape, i["dy"], dhy, D, gate)
    bars = dict(y=F32, hy=F32, dgx=GRAD, dh0=GRAD)
    if dtype == "bf16":
        bars.update(y=BF16, dgx=BF16)
    for k, want in dict(y=y, hy=hy, dgx=dgx, dh0=dh0).items():
        assert harness.rel_err(out[k], want) <= bars[k], k


# lengths around the tile sizes and the saved states, channel counts around the
# groups, odd widths (one element a load), more sequences than lanes
SHAPES = [(1, 1, 1), (1, 3, 8), (2, 1, 64), (63, 2, 20), (64, 1, 16), (65, 3, 12), (127, 1, 68), (128, 2, 4),
          (129, 1, 7), (300, 5, 33), (1030, 1, 64), (1025, 2, 5), (2500, 1, 8), (40, 70, 24)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,gate", [(1, False), (1, True), (2, False), (2, True)])
@pytest.mark.parametrize("T,N,H", SHAPES)
def test_matches_the_definition(T, N, H, D, gate, dtype):
    i = data(T, N, H, D, gate, dtype, T + N + H)
    check(i, run_gpu(i, D, gate, dtype), D, gate, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("T,N,H,lengths", [
    (5, 4, 8, [0, 5, 1, 4]), (70, 3, 20, [0, 0, 0]), (130, 5, 9, [130, 0, 64, 129, 1]),
    (1030, 3, 16, [1024, 1030, 3]), (9, 2, 4, [-3, 40])])
def test_lengths(T, N, H, lengths, gate, dtype):
    """Padding is never read; a sequence of length 0 hands its state through."""
    i = data(T, N, H, 2, gate, dtype, T)
    clipped = [min(max(v, 0), T) for v in lengths]
    out = run_gpu(i, 2, gate, dtype, lengths, poison=True)
    check(i, out, 2, gate, dtype, lengths)
    for n, ln in enumerate(clipped):
        assert (out["y"][ln:, n] == 0).all() and (out["dgx"][ln:, n] == 0).all()
        if ln == 0:
            assert np.array_equal(out["hy"][:, n], i["h0"][:, n])
            assert np.array_equal(out["dh0"][:, n], i["dhy"][:, n])


@pytest.mark.parametrize("dtype,pad", [("f32", 4), ("bf16", 8), ("f32", 1), ("bf16", 3), ("bf16", 2)])
def test_row_pitch(dtype, pad):
    i = data(133, 3, 12, 2, True, dtype, pad)
    check(i, run_gpu(i, 2, True, dtype, pad=pad), 2, True, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_states(dtype):
    i = data(100, 2, 16, 1, True, dtype, 5)
    check(i, run_gpu(i, 1, True, dtype, state=False), 1, True, dtype, state=False)


def test_gradient_against_differences():
    """The GPU's own forward, differenced in a few directions: float32 outputs
    of size 1 at a step of 1e-2 leave rounding near 1e-7 * sqrt(size) / 1e-2 and
    a third-order term near 1e-4."""
    i = data(70, 2, 6, 2, True, "f32", 9)
    out = run_gpu(i, 2, True, "f32")
    rng = np.random.default_rng(1)

    def loss(j):
        o = run_gpu(j, 2, True, "f32")
        return (o["y"] * i["dy"]).sum() + (o["hy"] * i["dhy"]).sum()

    for _ in range(4):
        v, w = rng.standard_normal(i["gx"].shape), rng.standard_normal(i["h0"].shape)
        v, w = v / np.linalg.norm(v), w / np.linalg.norm(w)
        e = 1e-2
        hi = loss(dict(i, gx=i["gx"] + e * v, h0=i["h0"] + e * w))
        lo = loss(dict(i, gx=i["gx"] - e * v, h0=i["h0"] - e * w))
        want = (out["dgx"] * v).sum() + (out["dh0"] * w).sum()
        assert abs((hi - lo) / (2 * e) - want) < 2e-3 * max(1.0, abs(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_saturated_gates_and_infinities(dtype):
    """f is exactly 1 or next to 0 at the ends; NaN in one channel stays there."""
    i = data(70, 1, 8, 1, False, dtype, 2)
    g = i["gx"].reshape(70, 1, 2, 8)
    g[:, :, 0, 0], g[:, :, 0, 1] = np.inf, -np.inf
    g[:, :, 0, 2], g[:, :, 0, 3] = 200.0, -200.0
    out = run_gpu(i, 1, False, dtype)
    z = g[:, 0, 1]
    held = harness.from_dev(harness.to_dev(i["h0"], dtype))[0, 0]  # y is stored in dtype
    for c in (0, 2):
        assert np.array_equal(out["y"][:, 0, c], np.full(70, held[c]))
    for c in (1, 3):
        assert harness.rel_err(out["y"][:, 0, c], z[:, c]) < 1e-6
    g[5, 0, 1, 4] = np.nan
    out = run_gpu(i, 1, False, dtype)
    bad = np.isnan(out["y"][:, 0])
    assert bad[5:, 4].all() and not bad[:5].any() and not bad[:, [0, 1, 2, 3, 5, 6, 7]].any()


def test_same_bits_again_and_on_another_stream():
    import torch
    i = data(1100, 3, 24, 2, True, "bf16", 8)
    a, b = run_gpu(i, 2, True, "bf16"), run_gpu(i, 2, True, "bf16", stream=torch.cuda.Stream())
    assert all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,gate", [(1, 1, False), (3, 8, True), (128, 33, True), (5, 1024, False)])
def test_step_by_step_is_the_scan(N, H, gate, dtype):
    """Steps one by one, the state updated in place, against the definition."""
    import torch
    from layer_rnn_gb300 import binding
    T = 6
    i = data(T, N, H, 1, gate, dtype, N)
    ops = binding.Ops(dtype)
    state = torch.tensor(i["h0"][0], dtype=torch.float32, device="cuda")
    ys = []
    for t in range(T):
        ys.append(harness.empty((N, H), dtype))
        ops.scan_step(harness.to_dev(i["gx"][t], dtype), state, state, ys[-1], out_gate=gate)
    y = torch.stack(ys)
    want, hy, _ = ref.scan(i["gx"], i["h0"], 1, gate)
    assert harness.rel_err(harness.from_dev(y), want) <= (BF16 if dtype == "bf16" else F32)
    assert harness.rel_err(harness.from_dev(state), hy[0]) <= F32


@pytest.mark.parametrize("T,N,H", [(4096, 1, 1024), (512, 16, 256)])
def test_long(T, N, H):
    """Many tiles a cluster, against the same recurrence run in float64 by torch."""
    import torch
    from layer_rnn_gb300 import binding
    gen = torch.Generator(device="cuda").manual_seed(1)
    gx = torch.randn((T, N, 2, H), generator=gen, device="cuda")
    gx[:, :, 0] += 2
    h = torch.randn((1, N, H), generator=gen, device="cuda")
    y, hy = torch.empty((T, N, H), device="cuda"), torch.empty_like(h)
    binding.Ops("f32").scan_forward(gx.view(T, N, 2 * H), h, y, hy)
    s = h[0].double()
    f = torch.sigmoid(gx[:, :, 0].double())
    b = (1 - f) * gx[:, :, 1].double()
    worst = torch.zeros((), device="cuda", dtype=torch.float64)
    for t in range(T):
        s = f[t] * s + b[t]
        worst = torch.maximum(worst, (s - y[t]).abs().max())
    # f <= sigmoid(2 + 5) here: 4 * 1100 * 2^-24 of values of size about 1
    assert worst.item() < 2.7e-4
    assert (hy[0] - s).abs().max().item() < 2.7e-4
