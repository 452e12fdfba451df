"""The operators together, as a model uses them: the example trains (its loss
falls from about log 32 to less than half) and, with 4-bit weights, generates far
better than the one in 32 of chance; its training gradient is the one that plain
torch operations give."""

import importlib.util
import os

import pytest

from tests import harness

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    harness.ensure_built()
    spec = importlib.util.spec_from_file_location("recurrent_lm",
                                                  os.path.join(harness.ROOT, "examples", "recurrent_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_trains_and_generates(lm, dtype, capsys):
    first, last, share = lm.main(["--dtype", dtype])
    assert last < 0.5 * first
    assert share > 4 / 32


def test_gradient_is_that_of_plain_operations(lm):
    """float64 recomputation by torch's own differentiation; float32 kernels through
    two layers of products of a few hundred terms: 1e-4 of the largest entry."""
    import torch
    from layer_rnn_gb300 import binding
    model = lm.Model(binding.Ops("f32"), vocab=16, width=40, H=24, F=36)
    gen = torch.Generator(device="cuda").manual_seed(3)
    tokens = lm.sequences(gen, 16, 70, 5)
    loss = torch.nn.functional.cross_entropy(model.logits(tokens[:-1]).reshape(-1, 16), tokens[1:].reshape(-1))
    loss.backward()

    def norm(h):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)

    copies = [p.detach().double().requires_grad_() for p in model.parameters()]
    it = iter(copies)
    embed = next(it)
    h = embed[tokens[:-1]]
    for _ in model.layers:
        gates, out, up, down = (next(it) for _ in range(4))
        p, z, q = (norm(h) @ gates.t()).split(24, -1)
        f, state, ys = torch.sigmoid(p), torch.zeros_like(p[0]), []
        for t in range(p.shape[0]):
            state = f[t] * state + (1 - f[t]) * z[t]
            ys.append(torch.sigmoid(q[t]) * state)
        h = h + torch.stack(ys) @ out.t()
        g, u = (norm(h) @ up.t()).split(36, -1)
        h = h + (g * torch.sigmoid(g) * u) @ down.t()
    want = torch.nn.functional.cross_entropy((norm(h) @ embed.t()).reshape(-1, 16), tokens[1:].reshape(-1))
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-5
    for a, b in zip(model.parameters(), copies):
        assert (a.grad - b.grad).abs().max() <= 1e-4 * b.grad.abs().max()
