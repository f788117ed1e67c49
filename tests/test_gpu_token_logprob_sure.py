"""Log-probabilities of sure tokens, whose target has nearly all of the probability, and their gradient, against
softmax in 64 bits.

u = 2^-24.  A sure token's logprob is -log1p(r), with r the others' sum over the target's term, and its
entropy log1p(r) + sum e d / (1 + r): sums of terms of one sign, so that they are right in relation to themselves, however
small.  A term e of r is (3 d + 4)u off (its difference d to the largest, the coefficient, the product; exp2); on
its way it is rescaled at most 40 times (batches of a thread, 5 shuffles, 15 warps, 15 CTAs), 5u each, and
added at most 80 times.  d <= 35 here: 105 + 4 + 200 + 80 = 389u of r, log1p one more: 400u.  The entropy's terms have
a factor d of 2u and the division beside it: 410u; taken as 500u.

lse is the rounded product of the largest logit and the scale, and log1p(r), rounded once more.  The gradient takes
p = exp(z - lse) with the same rounded product: a target whose others are below 2^-60 has z = lse, and p = 1 but for
exp2's 4u and a rounding or two, whatever the logit's size.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# one row over a cluster, a warp, CTAs of 128 threads, teams of 8, 4 and 1 warps
LAYOUTS = [(1, 32000, 20), (1, 32000, 0), (1, 131073, 4), (1, 512, 0), (500, 2000, 5), (700, 515, 0), (8000, 700, 0),
           (29500, 600, 0)]


def half_step(x):
    return torch.exp2(torch.frexp(x.double().abs()).exponent.double() - 25.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("offset", [100.0, 1000.0])
@pytest.mark.parametrize("n,vocab", [(1, 512), (1, 40000), (1300, 515)])
def test_gradient_where_one_logit_has_it_all(mfsdp, n, vocab, offset, scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + vocab)
    x = torch.randn(n, vocab, generator=g, device="cuda") + offset
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    x.scatter_(1, y[:, None], offset + 120.0 + 20.0 * torch.rand(n, 1, generator=g, device="cuda"))
    x = x.to(dtype)
    top = x.gather(1, y[:, None])[:, 0].double() * float(torch.tensor(scale, dtype=torch.float32))
    lse, ent = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    mfsdp.token_logprob(x, y, lse=lse, entropy=ent, scale=scale)
    off = half_step(top) if scale != 1.0 else torch.zeros_like(top)
    assert bool(((lse.double() - top).abs() <= off).all())
    assert float(ent.abs().max()) <= 2.0 ** -60
    for dlp, dent in ((1.0, None), (None, 1.0), (-0.5, 0.75)):
        dx = torch.full_like(x, 7.0)
        mfsdp.token_logprob_grad(x, y, lse, dx, dlogprob=torch.full((n,), dlp, device="cuda") if dlp else None,
                                 entropy=ent if dent else None,
                                 dentropy=torch.full((n,), dent, device="cuda") if dent else None, scale=scale)
        mine = dx.gather(1, y[:, None])[:, 0].double().abs()
        assert float(mine.max()) <= scale * (abs(dlp or 0.0) + abs(dent or 0.0)) * 8 * U * (1 + 2.0 ** -7)
        dx.scatter_(1, y[:, None], 0.0)
        assert float(dx.abs().max()) <= 2.0 ** -60


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0.0, 100.0])
@pytest.mark.parametrize("n,vocab,k", LAYOUTS)
def test_log_probabilities_near_zero(mfsdp, n, vocab, k, offset, dtype):
    """The others have from 0.15 (bf16: some more) down to some 1e-6 of the target's term."""
    g = torch.Generator(device="cuda").manual_seed(vocab + k)
    for seed in range(8 if n == 1 else 1):
        x = torch.randn(n, vocab, generator=g, device="cuda") + offset
        y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        r = torch.exp(torch.empty(n, 1, device="cuda").uniform_(math.log(1e-6), math.log(0.15), generator=g))
        x.scatter_(1, y[:, None], x.logsumexp(1, keepdim=True) - r.log())
        x = x.to(dtype)
        z = x.double()
        d = z - z.gather(1, y[:, None])
        e = d.exp().scatter_(1, y[:, None], 0.0)
        assert float(d[e > 0].abs().max()) <= 35.0
        rest = e.sum(1)
        want, entropy = -torch.log1p(rest), torch.log1p(rest) - (e * d).sum(1) / (1.0 + rest)
        logp, lse, ent = (torch.full((n,), 7.0, device="cuda") for _ in range(3))
        top = torch.full((n, k), 7.0, device="cuda") if k else None
        mfsdp.token_logprob(x, y, logp, lse=lse, entropy=ent, top_logprob=top)
        assert bool(((logp.double() - want).abs() <= 400 * U * want.abs()).all())
        assert bool(((ent.double() - entropy).abs() <= 500 * U * entropy).all())
        true = z.gather(1, y[:, None])[:, 0] - want
        assert bool(((lse.double() - true).abs() <= half_step(true) + 400 * U * want.abs()).all())       # (scale 1)
        if k:
            assert torch.equal(top[:, 0], logp)
        alone = torch.full((n,), 7.0, device="cuda")
        mfsdp.token_logprob(x, y, alone)
        assert bool(((alone.double() - want).abs() <= 400 * U * want.abs()).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,k", LAYOUTS)
def test_largest_logit_at_the_border(mfsdp, n, vocab, k, dtype):
    """-2^100 is the lowest live logit: alone it has all the probability, twice half of it each."""
    x = torch.full((n, vocab), -math.inf, dtype=dtype, device="cuda")
    y = torch.full((n,), vocab // 3, device="cuda")
    x[:, vocab // 3] = -2.0 ** 100
    logp, lse, ent = (torch.full((n,), 7.0, device="cuda") for _ in range(3))
    top = torch.full((n, k), 7.0, device="cuda") if k else None
    for copies in (1, 2):
        for entropy in (ent, None):
            mfsdp.token_logprob(x, y, logp, lse=lse, entropy=entropy, top_logprob=top)
            assert float((logp + math.log(copies)).abs().max()) <= 4 * U and (lse == -2.0 ** 100).all()
            assert float((ent - math.log(copies)).abs().max()) <= 4 * U
            if k:
                assert torch.equal(top[:, 0], logp) and torch.isneginf(top[:, copies:]).all()
        x[:, vocab - 1] = -2.0 ** 100
