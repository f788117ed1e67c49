"""Log-probabilities and their gradient against softmax in 64 bits, within bounds that come from differences of
logits and so do not grow with the logits themselves.

Bounds, u = 2^-24, first order.  M is a row's largest live logit, d_j = scale (M - x_j), p the probabilities,
h = sum p d, m2 = sum p d^2.
  A term exp(-d) is (3 d + 4)u off: the difference, the coefficient and their product u each; exp2's 2^-22.  On its way
  it is rescaled at most 42 times (7 batches of a thread, 5 shuffles, 15 warps, 15 CTAs), 5u each, and added at most 72 times.
  S is then within (3 h + 4 + 210 + 72 = 286)u of itself, taken as 3 h + 290, and log S has that and 2u of its value.
  logprob = (x_y - M) scale - log S: 2 d_y u beside it:  L = (2 d_y + 3 h + 300 + 2 log S)u.
  lse = M scale + log S, the product and the sum rounded: (|M scale| + |lse| + 3 h + 300 + 2 log S)u.
  entropy = log S + h: h's weights are off by (3 d + 290)u each, its divisor by (3 h + 290)u, its factors by 3u and
  some: (3 m2 + 3 h^2 + 600 h)u beside log S's.
  Gradient: log p = z - lse has lse's error and the product's, u |z|, u of itself, 2u more on the way to exp2 and exp2's 4u, so
  p is that of lse and (|z| + 3 |log p| + 4)u of itself off; log p + entropy the sum of its summands' absolute errors; four
  roundings more.
A bf16 output is rounded once more, by 2^-8 of its value at most.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
CASES = [(1, 1, 0), (3, 2, 0), (5, 7, 1), (33, 2000, 3), (2, 4097, 0), (700, 515, 0), (1, 32000, 0), (7, 31999, 2),
         (1, 131073, 0), (400, 9000, 8)]


def logits(n, vocab, pad, dtype, offset, masked, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, vocab + pad, generator=g, device="cuda") * 2.5 + offset).to(dtype)[:, :vocab]
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    if masked:
        gone = torch.rand(n, vocab, generator=g, device="cuda") < 0.7
        x[gone] = torch.finfo(dtype).min if masked == "lowest" else -math.inf
        x[:, vocab // 2] = offset                    # one is live
    if vocab > 600:
        x[:, 500:580] = float(offset + 4.0)           # equal ones
    y[::5] = -100
    return x, y


def definition(x, y, scale):
    scale = float(torch.tensor(scale, dtype=torch.float32))
    z = torch.where(x.double() < -2.0 ** 100, -math.inf, x.double()) * scale
    top = z.amax(1, keepdim=True)
    d = top - z
    e = torch.exp(-d)
    s = e.sum(1, keepdim=True)
    p = e / s
    d0 = torch.where(p > 0, d, 0.0)
    h, m2 = (p * d0).sum(1), (p * d0 * d0).sum(1)
    log_s = torch.log(s)[:, 0]
    logp = -d - log_s[:, None]
    live = (y >= 0) & (y < x.shape[1])
    at = torch.where(live, y, 0)[:, None]
    mine, dy = logp.gather(1, at)[:, 0], d.gather(1, at)[:, 0]
    base = 3 * h + 300 + 2 * log_s
    b = {"logp": torch.where(torch.isfinite(dy) & live, 2 * dy + base, 0.0) * U, "lse": (top[:, 0].abs() + (top[:, 0] + log_s).abs() + base) * U,
         "entropy": (base + 3 * m2 + 3 * h * h + 600 * h) * U}
    return dict(z=torch.where(p > 0, z, 0.0), logp=torch.where(live, mine, 0.0), lse=top[:, 0] + log_s, entropy=log_s + h, all=logp, p=p, at=at, live=live,
                b=b, base=base)


def check(got, want, bound, what):
    got, want = got.double(), want.double()
    inf = ~torch.isfinite(want)
    assert torch.equal(got[inf], want[inf]), what
    off = ((got - want).abs() - bound.expand(want.shape))[~inf]
    assert not off.numel() or float(off.max()) <= 0.0, (what, float(off.max()))


@pytest.mark.parametrize("masked", [None, "-inf", "lowest"])
@pytest.mark.parametrize("dtype,offset", [(torch.float32, 0.0), (torch.float32, 1000.0), (torch.bfloat16, 0.0),
                                          (torch.bfloat16, -100.0)])
@pytest.mark.parametrize("n,vocab,pad", CASES)
def test_values_and_gradient(mfsdp, n, vocab, pad, dtype, offset, masked):
    for scale, k in ((1.0, 0), (0.7, min(vocab, 5)), (1.0, min(vocab, 32))):
        x, y = logits(n, vocab, pad, dtype, offset, masked, seed=vocab + k)
        w = definition(x, y, scale)
        out = {name: torch.full((n,), 7.0, device="cuda") for name in ("logp", "lse", "entropy")}
        ids = torch.full((n, k), -7, dtype=torch.int32, device="cuda") if k else None
        top = torch.full((n, k), 7.0, device="cuda") if k else None
        mfsdp.token_logprob(x, y, out["logp"], lse=out["lse"], entropy=out["entropy"], top_ids=ids, top_logprob=top,
                            scale=scale)
        for name, got in out.items():
            check(got, w[name], w["b"][name], name)
        if k:
            want_ids = torch.sort(x.float().cpu(), dim=1, descending=True, stable=True).indices[:, :k].cuda()
            assert torch.equal(ids.long(), want_ids)
            theirs = w["all"].gather(1, want_ids)
            away = torch.where(torch.isfinite(theirs), -theirs, 0.0)
            check(top, theirs, (2 * away + w["base"][:, None]) * U, "top")
        g = torch.Generator(device="cuda").manual_seed(1)
        dlp, dent = (torch.randn(n, generator=g, device="cuda") for _ in range(2))
        logp, p, s = w["all"], w["p"], float(torch.tensor(scale, dtype=torch.float32))
        lp = torch.where(p > 0, logp, 0.0)
        for use_dlp, use_dent in ((True, False), (False, True), (True, True)):
            dx = torch.full_like(x, 7.0)
            mfsdp.token_logprob_grad(x, y if use_dlp else None, out["lse"], dx, dlogprob=dlp if use_dlp else None,
                                     entropy=out["entropy"] if use_dent else None, dentropy=dent if use_dent else None,
                                     scale=scale)
            a = torch.where(w["live"], dlp.double(), 0.0)[:, None] * use_dlp
            c = dent.double()[:, None] * use_dent
            one = torch.zeros_like(p).scatter_(1, w["at"], 1.0)
            factor = lp + w["entropy"][:, None]
            want = s * (a * (one - p) - c * p * factor)
            rel = w["b"]["lse"][:, None] + (w["z"].abs() + 3 * lp.abs() + 4) * U
            slack = s * p * (a.abs() * (rel + 6 * U)
                             + c.abs() * (factor.abs() * (rel + 8 * U)
                                          + w["b"]["lse"][:, None] + U * (w["z"].abs() + lp.abs()) + w["b"]["entropy"][:, None]))
            slack = slack + (4 * U + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)) * want.abs() + 2.0 ** -100
            check(dx, want, slack, ("gradient", use_dlp, use_dent))
