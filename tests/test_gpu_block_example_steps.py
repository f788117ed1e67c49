"""Each step of the block example's gradients by itself: what it left in its buffer against plain fp64 torch on what the
steps before it left, so that no rounding but the step's own stands between the two.

Tolerance, of Frobenius norms: a bf16 buffer is rounded once, 2^-8 of each element.  A sum of n <= 1000 terms in fp32 is
within n 2^-24 of the sum of their magnitudes, which is up to sqrt(n) of the result's size where signs are mixed: 2^-9;
a norm's gradient is a difference of such.  So fp32 buffers within 2^-8 and bf16 ones within 2^-7.
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
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "block_training_step.py")
    spec = importlib.util.spec_from_file_location("block_training_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def near(got, want, what):
    bound = 2.0 ** -7 if got.dtype == torch.bfloat16 else 2.0 ** -8
    off = float((got.double().reshape(want.shape) - want).norm())
    assert off <= bound * float(want.norm()), (what, off / float(want.norm()))


def rms(x, w):
    return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w


@pytest.mark.parametrize("vocab,dim,hidden,batch", [(300, 64, 128, 700), (1000, 256, 96, 333)])
def test_each_step_from_the_one_before(mfsdp, example, vocab, dim, hidden, batch):
    model = example.BlockModel(vocab, dim, hidden, batch, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    for v in model.vectors.values():
        v.add_(torch.randn(dim, generator=g, device="cuda") * 0.2)
    ids, targets = (torch.randint(0, vocab, (batch,), device="cuda", generator=g) for _ in range(2))
    targets[::7] = -100
    loss = model.gradients(ids, targets)
    d = {k: t.double() for k, t in vars(model).items() if torch.is_tensor(t)}
    vec, dvec = {k: t.double() for k, t in model.vectors.items()}, model.dvectors
    w1, w2, head = (t[0].double() for t in (model.w1, model.w2, model.head_bf16))

    # there
    assert torch.equal(model.h, model.emb_bf16[ids].float())
    near(model.x, rms(d["h"], vec["first_weight"]), "x")
    near(model.z, d["x"] @ w1.t(), "z")
    assert torch.equal(model.a, model.z.relu())
    near(model.y, d["a"] @ w2.t(), "y")
    h, y = (d[k].clone().requires_grad_() for k in "hy")
    leaf = {k: vec[k].clone().requires_grad_() for k in ("post_weight", "gate", "head_weight")}
    out = h + leaf["gate"] * rms(y, leaf["post_weight"])
    normed = rms(out, leaf["head_weight"])
    near(model.out, out.detach(), "out")
    near(model.normed, normed.detach(), "normed")
    # the logits went to their gradient's place: made again, by the same call
    logits = torch.empty_like(model.logits)
    mfsdp.expert_matmul(model.normed, model.head_bf16, model.starts, logits, model.head_ws)
    near(logits, d["normed"] @ head.t(), "logits")
    x = logits.double().requires_grad_()
    logp = torch.log_softmax(x, 1)
    live = (targets >= 0)[:, None]
    mine = torch.where(live, logp.gather(1, torch.where(live, targets[:, None], 0)), 0.0)[:, 0]
    entropy = -(logp.exp() * logp).sum(1)
    want = -(mine.mean() + model.entropy_bonus * entropy.mean())
    near(model.logprob, mine.detach(), "logprob")
    near(model.entropy, entropy.detach(), "entropy")
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -8 * abs(float(want.detach()))

    # and back
    want.backward()
    near(model.logits, x.grad, "dlogits")
    dlogits = d["logits"]
    near(model.dhead, dlogits.t() @ d["normed"], "dhead")
    near(model.dnormed, dlogits @ head, "dnormed")
    normed.backward(d["dnormed"])
    near(model.dy, y.grad, "dy")
    for k, t in leaf.items():
        near(dvec[k], t.grad, k)
    near(model.dw2, d["dy"].t() @ d["a"], "dw2")
    near(model.dz, (d["dy"] @ w2) * (model.z > 0), "dz")
    near(model.dw1, d["dz"].t() @ d["x"], "dw1")
    near(model.dx, d["dz"] @ w1, "dx")
    first, h0 = vec["first_weight"].clone().requires_grad_(), d["h"].clone().requires_grad_()
    rms(h0, first).backward(d["dx"])
    near(dvec["first_weight"], first.grad, "first_weight")
    near(model.dout, h.grad + h0.grad, "dout")
    near(model.demb, torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids, d["dout"]), "demb")
