"""The mixture-of-experts example: its gradients against plain fp64 torch, and its
training.

Tolerance: the reference follows the example's formulas in fp64 from the same
weights, with the example's own relu mask: a z that rounding moves across zero
changes a whole term of the gradients, which no bound on roundings covers.  The example rounds to bf16 (2^-8 each) the looked up rows and
targets, z, a, dy, dz, and W1 and W2 once: a gradient has at most 6 of these on its
path, so its Frobenius norm of error is within 6 * 2^-8 of its norm.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_training_step.py")
    spec = importlib.util.spec_from_file_location("moe_training_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("vocab,dim,hidden,experts,batch", [(300, 64, 128, 4, 700), (37, 128, 64, 8, 33)])
def test_gradients_match_plain_torch(example, vocab, dim, hidden, experts, batch):
    layer = example.MoeLayer(vocab, dim, hidden, experts, batch, seed=3)
    ids = torch.randint(0, vocab, (batch,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    loss = layer.gradients(ids)
    mask = torch.empty_like(layer.z, dtype=torch.bool)
    mask[layer.order.long()] = layer.z > 0              # in the batch's order
    w1, w2, emb = (t.double().requires_grad_() for t in (layer.w1, layer.w2, layer.emb))
    e = layer.expert_of[ids]
    x = emb[ids]
    z = torch.einsum("thd,td->th", w1[e], x)
    y = torch.einsum("tdh,th->td", w2[e], z * mask)
    want = (y - layer.targets.double()[ids]).square().mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 6 * 2 ** -8 * float(want.detach())
    for name, got, ref in (("W1", layer.dw1, w1.grad), ("W2", layer.dw2, w2.grad), ("E", layer.demb, emb.grad)):
        assert float((got.double() - ref).norm()) <= 6 * 2 ** -8 * float(ref.norm()), name


def test_training_lowers_the_loss(example):
    layer = example.MoeLayer(vocab=500, dim=128, hidden=256, experts=4, batch=2048)
    g = torch.Generator(device="cuda").manual_seed(5)
    losses = [float(layer.step(torch.randint(0, 500, (2048,), device="cuda", generator=g))) for _ in range(30)]
    assert losses[-1] < losses[0] / 4
    assert 0.0 < float(layer.norm[1]) <= 1.0
