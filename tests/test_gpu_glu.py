"""The gated feed-forward against its float64 form.

Bars (largest error over the largest result).  bfloat16 forward: float32 sums
and one rounding, 2^-9: 2^-8.  bfloat16 backward: dg and du are rounded too
(2^-9 each, in a sum): 2^-7.  float32: operands keep 22 bits (2^-22) or all,
sums of K terms in float32, the activation a few ulp: 4e-6; the backward chains
two such products: 1.2e-5.
"""

import numpy as np
import pytest

from tests import harness
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
BARS = {"f32": (4e-6, 1.2e-5), "bf16": (2.0 ** -8, 2.0 ** -7)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    harness.ensure_built()


def make(M, K, F, dtype, seed=0):
    rng = np.random.default_rng(seed + M * 7 + K * 3 + F)
    r = lambda a: harness.from_dev(harness.to_dev(a, dtype))  # noqa: E731
    return dict(x=r(rng.standard_normal((M, K))), W=r(rng.standard_normal((2 * F, K)) / np.sqrt(K)),
                dy=r(rng.standard_normal((M, F))))


def run(d, act, dtype, backward=True, dx=True, dW=True, stream=None):
    import torch
    from layer_rnn_gb300 import binding
    ops = binding.Ops(dtype)
    (M, K), F = d["x"].shape, d["W"].shape[0] // 2
    x, W, dy = (harness.to_dev(d[k], dtype) for k in ("x", "W", "dy"))
    out = dict(y=harness.empty((M, F), dtype))
    # the workspace holds garbage: nothing may be expected of it
    ws = torch.full((ops.glu_workspace_bytes(M, K, F, backward),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    ops.glu_forward(x, W, out["y"], ws, act=act, stream=stream)
    if backward:
        out["dx"] = harness.empty((M, K), dtype) if dx else None
        out["dW"] = harness.empty((2 * F, K), dtype) if dW else None
        ops.glu_backward(x, W, dy, out["dx"], out["dW"], ws, act=act, stream=stream)
    torch.cuda.synchronize()
    assert ops.check_status() == 0
    return {k: harness.from_dev(v) for k, v in out.items() if v is not None}


def check(d, out, act, dtype):
    fwd, grad = BARS[dtype]
    assert harness.rel_err(out["y"], ref.glu(d["x"], d["W"], act)) <= fwd
    if "dx" in out or "dW" in out:
        dx, dW = ref.glu_backward(d["x"], d["W"], d["dy"], act)
        if "dx" in out:
            assert harness.rel_err(out["dx"], dx) <= grad
        if "dW" in out:
            assert harness.rel_err(out["dW"], dW) <= grad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("M,K,F", [(1, 1, 1), (1, 64, 8), (2, 72, 9), (3, 65, 100), (8, 1000, 7), (9, 520, 40),
                                   (16, 8, 64), (17, 200, 33), (31, 1003, 16), (32, 64, 130)])
def test_few_rows(M, K, F, act, dtype):
    d = make(M, K, F, dtype)
    check(d, run(d, act, dtype), act, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("M,K,F", [(33, 64, 64), (65, 1, 1), (100, 72, 128), (128, 65, 129), (129, 200, 100),
                                   (256, 64, 256), (257, 130, 7), (300, 1003, 77), (600, 256, 264)])
def test_many_rows(M, K, F, act, dtype):
    d = make(M, K, F, dtype)
    check(d, run(d, act, dtype), act, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,F", [(20000, 64, 72), (256, 264, 8200), (9000, 520, 300), (40, 16, 20000)])
def test_long_contractions(M, K, F, dtype):
    """Few tiles, long sums: cut along the contraction, joined in order."""
    d = make(M, K, F, dtype)
    a = run(d, "silu", dtype)
    check(d, a, "silu", dtype)
    b = run(d, "silu", dtype)
    assert all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("M,K,F", [(4, 16384, 24), (32, 8192, 40), (20, 40000, 9)])
def test_few_rows_split_over_a_cluster(M, K, F):
    d = make(M, K, F, "bf16")
    check(d, run(d, "gelu", "bf16", backward=False), "gelu", "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_either_gradient_alone_and_another_stream(dtype):
    import torch
    d = make(300, 136, 200, dtype)
    both = run(d, "silu", dtype)
    s = torch.cuda.Stream()
    assert np.array_equal(run(d, "silu", dtype, dW=False, stream=s)["dx"], both["dx"])
    assert np.array_equal(run(d, "silu", dtype, dx=False, stream=s)["dW"], both["dW"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [5, 200])
def test_large_pre_activations(M, dtype):
    """Gates far into saturation, rows of zeros, and a row of large values."""
    d = make(M, 64, 40, dtype)
    d["x"][0] = 0
    d["x"][1] *= 100.0
    d["x"] = harness.from_dev(harness.to_dev(d["x"], dtype))
    for act in ("silu", "gelu", "sigmoid"):
        out = run(d, act, dtype)
        assert all(np.isfinite(v).all() for v in out.values())
        check(d, out, act, dtype)
        assert (out["y"][0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [6, 150])
def test_a_row_that_is_not_finite_spoils_itself_alone(M, dtype):
    if dtype == "f32" and M > 64:
        pytest.skip("one scale serves the whole operand there: documented")
    d = make(M, 72, 24, dtype)
    good = run(d, "silu", dtype, backward=False)["y"]
    d["x"][3, 5] = np.nan
    bad = run(d, "silu", dtype, backward=False)["y"]
    assert np.isnan(bad[3]).all()
    keep = np.arange(M) != 3
    assert np.array_equal(bad[keep], good[keep])


def test_gradient_against_differences():
    """float32, a few directions: y of size 1 at a step of 1e-2 leaves rounding
    near 1e-6 / 1e-2 of |y| |dy| and a third-order term near 1e-4."""
    d = make(70, 24, 40, "f32")
    out = run(d, "gelu", "f32")
    rng = np.random.default_rng(1)
    loss = lambda e: (run(e, "gelu", "f32", backward=False)["y"] * d["dy"]).sum()  # noqa: E731
    for _ in range(4):
        v, w = rng.standard_normal(d["x"].shape), rng.standard_normal(d["W"].shape)
        v, w = v / np.linalg.norm(v), w / np.linalg.norm(w)
        e = 1e-2
        diff = (loss(dict(d, x=d["x"] + e * v, W=d["W"] + e * w)) -
                loss(dict(d, x=d["x"] - e * v, W=d["W"] - e * w))) / (2 * e)
        want = (out["dx"] * v).sum() + (out["dW"] * w).sum()
        assert abs(diff - want) < 2e-2 * max(1.0, abs(want))


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,F", [(150, 72, 24), (300, 136, 200), (130, 37, 41)])
def test_many_rows_keep_a_value_that_is_not_finite_apart(M, K, F, dtype, value):
    """A token's rows of y and dx take its value that is not finite, no others do;
    a weight's feature likewise."""
    d = make(M, K, F, dtype)
    good = run(d, "silu", dtype)
    x, W = d["x"], d["W"]
    d["x"] = x.copy()
    d["x"][3, 5] = value
    bad = run(d, "silu", dtype)
    keep = np.arange(M) != 3
    # float32: without that value the operand's scale, and so its last bits, may be others
    same = lambda a, b: np.isfinite(a).all() and harness.rel_err(a, b) <= (1e-6 if dtype == "f32" else 0)  # noqa: E731
    assert not np.isfinite(bad["y"][3]).any()
    assert same(bad["y"][keep], good["y"][keep]) and same(bad["dx"][keep], good["dx"][keep])
    d["x"], d["W"] = x, W.copy()
    d["W"][7, 2] = value
    bad = run(d, "silu", dtype, backward=False)
    keep = np.arange(F) != 7
    assert same(bad["y"][:, keep], good["y"][:, keep])
