"""The gradient of the logits in place of the logits, where rows share their first and last lines: bit by bit what it is
apart from them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,pad,offset", [(20000, 1, 0, 0), (20000, 3, 0, 1), (20000, 7, 1, 0), (9999, 33, 0, 3),
                                                (5000, 129, 0, 1), (300, 4099, 2, 5), (3, 70001, 0, 1)])
def test_in_place_is_apart(mfsdp, n, vocab, pad, offset, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    flat = (torch.randn(n * (vocab + pad) + offset, generator=g, device="cuda") * 2.5).to(dtype)
    x = flat[offset:].view(n, vocab + pad)[:, :vocab]
    y = torch.randint(-1, vocab, (n,), generator=g, device="cuda")
    lse, ent = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    mfsdp.token_logprob(x, y, lse=lse, entropy=ent)
    kw = dict(dlogprob=torch.randn(n, generator=g, device="cuda"), entropy=ent,
              dentropy=torch.randn(n, generator=g, device="cuda"))
    apart = torch.empty(n, vocab + pad + 1, dtype=dtype, device="cuda")[:, :vocab]
    mfsdp.token_logprob_grad(x, y, lse, apart, **kw)
    for _ in range(5):
        again = flat.clone()
        same = again[offset:].view(n, vocab + pad)[:, :vocab]
        mfsdp.token_logprob_grad(same, y, lse, same, **kw)
        assert torch.equal(same, apart)
        left = torch.ones_like(again, dtype=torch.bool)
        left[offset:].view(n, vocab + pad)[:, :vocab] = False
        assert torch.equal(again[left], flat[left])
