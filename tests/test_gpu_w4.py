"""Products with 4-bit weights against their float64 form.

Bars (largest error over the largest result).  float32: tokens keep 22 bits
(2^-22 of the largest value, per term of a sum of K random signs: no growth in
the ratio), sums in float32 of up to K / 16 terms in a row and of the warps'
parts: sqrt(K / 16) 2^-24 at random, held to 2e-6 for K up to 4 k and 6e-6
above.  bfloat16: one rounding, 2^-9, and that: 2^-8.
"""

import numpy as np
import pytest

from tests import harness
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    harness.ensure_built()


def bar(dtype, K):
    return 2.0 ** -8 if dtype == "bf16" else 2e-6 if K <= 4096 else 6e-6


def make(M, R, K, group, zeros, dtype, seed, pitch=None):
    rng = np.random.default_rng(seed)
    pitch = pitch or ((K + 1) // 2 + 15) // 16 * 16
    G = -(-K // group)
    rnd = lambda a: harness.from_dev(harness.to_dev(a, dtype))  # noqa: E731
    return dict(x=rnd(rng.standard_normal((M, K))), s=rnd(rng.uniform(0.5, 1.5, (R, G))),
                q=rng.integers(0, 256, (R, pitch)).astype(np.uint8),
                z=rng.integers(0, 16, (R, G)).astype(np.uint8) if zeros else None)


def run(d, group, dtype, stream=None):
    import torch
    from layer_rnn_gb300 import binding
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    y = harness.empty((d["x"].shape[0], d["q"].shape[0]), dtype)
    x, s = harness.to_dev(d["x"], dtype), harness.to_dev(d["s"], dtype)
    q, z = up(d["q"]), up(d["z"])
    torch.cuda.synchronize()
    binding.Ops(dtype).w4_matvec(x, q, s, y, group=group, zeros=z, stream=stream)
    torch.cuda.synchronize()
    return harness.from_dev(y)


def want(d, group):
    w = ref.w4_weights(d["q"], d["s"], d["z"], d["x"].shape[1], group)
    return d["x"] @ w.T


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,R,K", [
    (1, 1, 1), (1, 16, 31), (1, 17, 256), (2, 15, 257), (3, 100, 1000), (4, 33, 2049), (5, 64, 512),
    (8, 40, 777), (9, 31, 1280), (16, 50, 300), (17, 20, 640), (40, 16, 96), (1, 3000, 700)])
def test_matches_the_definition(M, R, K, group, zeros, dtype):
    d = make(M, R, K, group, zeros, dtype, M * R + K)
    assert harness.rel_err(run(d, group, dtype), want(d, group)) <= bar(dtype, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,R,K,group", [(1, 48, 16384, 64), (16, 33, 8200, 32), (8, 16, 20000, 128),
                                         (1, 20, 65536, 128), (16, 17, 40001, 32), (3, 5000, 4096, 128)])
def test_split_over_a_cluster(M, R, K, group, dtype):
    d = make(M, R, K, group, True, dtype, 7)
    assert harness.rel_err(run(d, group, dtype), want(d, group)) <= bar(dtype, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,R,K,group", [(12, 40001, 130, 32), (16, 100003, 97, 64), (9, 12001, 4100, 128),
                                         (6, 50001, 260, 32)])
def test_more_rows_than_the_card_holds_at_once(M, R, K, group, dtype):
    d = make(M, R, K, group, True, dtype, 11)
    assert harness.rel_err(run(d, group, dtype), want(d, group)) <= bar(dtype, K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wider_pitch_and_garbage_past_the_row(dtype):
    d = make(3, 40, 333, 64, True, dtype, 1, pitch=512)
    a = run(d, 64, dtype)
    d["q"][:, 167:] ^= 255
    d["q"][:, 166] ^= 0xF0  # the nibble after the last weight
    assert np.array_equal(a, run(d, 64, dtype))
    assert harness.rel_err(a, want(d, 64)) <= bar(dtype, 333)


def test_token_scales_and_values_that_are_not_finite():
    """float32 tokens of very different sizes keep their own precision; one that
    is not finite spoils its own row alone."""
    d = make(6, 50, 300, 32, False, "f32", 3)
    d["x"] = (d["x"] * np.array([1e-30, 1e30, 1.0, 0.0, 1.0, 1.0])[:, None]).astype(np.float32).astype(float)
    ref_y = want(d, 32)
    y = run(d, 32, "f32")
    for m in (0, 1, 2, 4, 5):
        assert harness.rel_err(y[m], ref_y[m]) <= bar("f32", 300)
    assert (y[3] == 0).all()
    d["x"][4, 7], d["x"][5, 9] = np.nan, np.inf
    z = run(d, 32, "f32")
    assert np.array_equal(z[:4], y[:4]) and np.isnan(z[4]).all() and not np.isfinite(z[5]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_again_and_on_another_stream(dtype):
    import torch
    d = make(5, 700, 9000, 64, True, dtype, 2)
    assert np.array_equal(run(d, 64, dtype), run(d, 64, dtype, stream=torch.cuda.Stream()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("R,K", [(1, 1), (7, 200), (33, 513)])
def test_quantised_weights_are_nearest(R, K, group, zeros, dtype):
    """Each weight lies within half a step (and, at the symmetric grid's upper
    end or by the rounding of the zero point, within one step), and the product
    with them is the product with what they stand for."""
    import torch
    from layer_rnn_gb300 import binding
    rng = np.random.default_rng(R)
    W = harness.from_dev(harness.to_dev(rng.standard_normal((R, K)), dtype))
    W[0, :min(K, group)] = 0  # a group of zeros
    ops = binding.Ops(dtype)
    q, s, z = ops.w4_alloc(R, K, group, zeros)
    ops.w4_quantize(harness.to_dev(W, dtype), q, s, group, z)
    torch.cuda.synchronize()
    w = ref.w4_weights(q.cpu().numpy(), harness.from_dev(s), None if z is None else z.cpu().numpy(), K, group)
    step = harness.from_dev(s)[:, np.arange(K) // group]
    assert (np.abs(w - W) <= step * (1.0 + 0.07)).all()
    assert (np.abs(w - W) <= step * 0.51).mean() > 0.9
    assert (q.cpu().numpy()[:, (K + 1) // 2:] == 0).all()
    x = rng.standard_normal((2, K)).astype(np.float32).astype(float)
    y = harness.empty((2, R), dtype)
    ops.w4_matvec(harness.to_dev(x, dtype), q, s, y, group, z)
    xr = harness.from_dev(harness.to_dev(x, dtype))
    assert harness.rel_err(harness.from_dev(y), xr @ w.T) <= bar(dtype, K)
