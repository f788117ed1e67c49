"""The gradient of sure tokens, whose target has all of the probability, at logits far from zero.

u = 2^-24.  lse is one rounding, half a step of fp32, of the largest logit's product with the scale; where that is
representable (scale 1) the half step is 0.  The gradient takes p = exp(z - lse): the others are below
2^-60 here, so p = 1 but for lse's half step, exp2's 4u and a rounding or two.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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
        assert bool((mine <= scale * (abs(dlp or 0.0) + abs(dent or 0.0)) * (off + 8 * U) * (1 + 2.0 ** -7)).all())
        dx.scatter_(1, y[:, None], 0.0)
        assert float(dx.abs().max()) <= 2.0 ** -60
