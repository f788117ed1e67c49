"""GPU parity of the operators next to the owner step with the fp64 oracle, at
the sizes, layouts and masks where they can go wrong.

Tolerances, from the arithmetic (u = 2^-24, an fp32 rounding; h = 2^-8, a bf16 one: 8 significant bits):
  norm        fp32 sums of 8 then 8 squares (11 roundings of S at most, halved
              by the root), one rounding of the root: 7 u
  clipped     the coefficient's rounding and the norm's, the product's: 9 u (+ h)
  lookup      the scale's rounding and the product's: 2 u (+ h)
  embedding gradient   a sum of m terms in any order: (m + 2) u times the sum of
              their magnitudes, then scale and accumulate: 3 u more (+ h of the result)
  products    a sum of K products: max(K, 32) u times the sum of their
              magnitudes.  Any order of fp32 additions stays inside it; a tensor
              core adds 16 products at a time and may truncate (2 u each of
              K / 16 + 1 additions).  (+ h of the result for bf16, u for fp32)
"""
import numpy as np
import pytest

from oracle.ops import (embedding_grad_ref, embedding_lookup_ref, expert_matmul_ref, expert_weight_grad_ref,
                        grad_clip_ref, sort_ids_ref)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(a, dtype="f32"):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda().to(DT[dtype])


def host(t):
    return t.double().cpu().numpy()


def rnd(dtype):
    return H if dtype == "bf16" else U


def scratch(n):
    return torch.full((max(int(n), 1),), 0xFF, dtype=torch.uint8, device="cuda")     # never relied on to be zero


def close(got, want, bound, what=""):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, error {err[bad][0]:.3e}"


# ------------------------------------------------------------ norm, clipping
def clip(m, srcs, dsts=None, **kw):
    s = m.grad_set(srcs, dsts)
    out = torch.full((2,), -7.0, device="cuda")
    m.grad_clip(s, out, scratch(m.grad_clip_workspace_bytes(s)), **kw)
    return [float(v) for v in out.double().cpu()]


def check_clip(m, srcs, dsts, max_norm, eps=1e-6):
    before = [host(s) for s in srcs]
    norm, coef, want = grad_clip_ref(before, max_norm, eps)
    got_norm, got_coef = clip(m, srcs, dsts, max_norm=max_norm, eps=eps)
    assert abs(got_norm - norm) <= 7 * U * norm and abs(got_coef - coef) <= 8 * U * coef
    for s, d, w in zip(srcs, dsts or srcs, want):
        close(host(d), w, (9 * U + rnd("bf16" if d.dtype == torch.bfloat16 else "f32")) * np.abs(w), "clipped")


@pytest.mark.parametrize("src,dst", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("sizes,gap", [([1], 0), ([7, 1, 8, 9], 1), ([16384, 16385, 3, 100_003], 3), ([131072, 4096], 0),
                                       ([500_000], 5)])
def test_clip(mfsdp, src, dst, sizes, gap):
    rng = np.random.default_rng(sum(sizes) + gap)
    total = sum(sizes) + gap * (len(sizes) + 1)
    flat = dev(rng.standard_normal(total), src)
    out = torch.full((total + 1,), 77.0, device="cuda").to(DT[dst])
    at, srcs, dsts, owned = gap, [], [], np.zeros(total + 1, bool)
    for n in sizes:
        srcs.append(flat[at:at + n])
        dsts.append(out[at + 1:at + 1 + n])          # another alignment than the source's
        owned[at + 1:at + 1 + n] = True
        at += n + gap
    check_clip(mfsdp, srcs, dsts, 0.5)
    assert np.all(host(out)[~owned] == 77.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_in_place_and_unclipped(mfsdp, dtype):
    rng = np.random.default_rng(5)
    flat = dev(rng.standard_normal(70_001) * 1e-3, dtype)
    keep = flat.clone()
    parts = [flat[1:30_000], flat[30_000:70_000]]
    norm, coef = clip(mfsdp, parts, max_norm=100.0)
    assert coef == 1.0 and torch.equal(flat, keep)               # below the limit: not a bit changes
    check_clip(mfsdp, parts, None, norm / 3)
    assert flat[0] == keep[0] and flat[70_000] == keep[70_000]
    norm2, _ = clip(mfsdp, parts, max_norm=float("inf"))
    assert abs(norm2 - norm / 3) <= (H + 20 * U) * norm / 3


def test_clip_many_tensors(mfsdp):
    """More tensors than one launch's table, with empty ones among them."""
    rng = np.random.default_rng(6)
    sizes = rng.integers(0, 200, 1300)
    flat = dev(rng.standard_normal(int(sizes.sum())))
    ends = np.cumsum(sizes)
    srcs = [flat[e - n:e] for n, e in zip(sizes, ends)]
    out = torch.zeros_like(flat)
    check_clip(mfsdp, srcs, [out[e - n:e] for n, e in zip(sizes, ends)], 3.0)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-44])
def test_norm_outside_the_range_of_fp32_squares(mfsdp, value):
    x = torch.full((40_000,), value, device="cuda")
    x[::3] = 0.0
    v = float(x[1].double())
    want = v * np.sqrt(40_000 - 13_334)
    norm, coef = clip(mfsdp, [x.clone()], max_norm=v, eps=0.0)
    if want > 3.4028235e38:
        assert norm == float("inf")
    else:
        assert abs(norm - want) <= max(7 * U * want, 2.0 ** -149)
    assert abs(coef - v / want) <= 9 * U * v / want               # right although the square overflows fp32


def test_clip_special_values(mfsdp):
    ones = torch.ones(5000, device="cuda")
    assert clip(mfsdp, [torch.zeros(100, device="cuda")], max_norm=1.0) == [0.0, 1.0]
    assert clip(mfsdp, [torch.zeros(100, device="cuda")], max_norm=0.0, eps=0.0) == [0.0, 1.0]
    assert clip(mfsdp, [], max_norm=1.0) == [0.0, 1.0]
    assert clip(mfsdp, [ones[:0]], max_norm=1.0) == [0.0, 1.0]
    assert clip(mfsdp, [ones.clone()], max_norm=0.0)[1] == 0.0
    for bad, norm, coef in ((float("inf"), np.inf, 0.0), (float("nan"), np.nan, np.nan)):
        for at in (0, 4999):
            x = ones.clone()
            x[at] = bad
            got = clip(mfsdp, [ones.clone(), x], [torch.empty_like(ones), torch.empty_like(ones)], max_norm=1.0)
            assert np.array_equal(got, [norm, coef], equal_nan=True)


def test_norm_alone_and_repeatable(mfsdp):
    x = dev(np.random.default_rng(7).standard_normal(3_000_001))
    s = mfsdp.grad_set([x, x[5:]])
    out, ws = torch.zeros(2, device="cuda"), scratch(mfsdp.grad_clip_workspace_bytes(s))
    mfsdp.grad_norm(s, out, ws)
    first = out.clone()
    want = np.sqrt(np.sum(host(x) ** 2) + np.sum(host(x)[5:] ** 2))
    assert abs(float(out[0]) - want) <= 7 * U * want and float(out[1]) == 1.0
    for _ in range(3):
        mfsdp.grad_norm(s, out, ws)
        assert torch.equal(out, first)


# ------------------------------------------------------------------- id sort
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,keys", [(0, 5), (1, 1), (31, 3), (2048, 128), (2049, 255), (2049, 256), (5000, 70_000),
                                    (300_001, 32_000), (70_000, 1 << 20)])
def test_sort_ids(mfsdp, idt, n, keys):
    rng = np.random.default_rng(n + keys)
    ids = rng.integers(-2, keys + 2, n)
    ids[: n // 3] = keys // 2                       # one heavy id
    order = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    starts = torch.full((keys + 1,), -1, dtype=torch.int32, device="cuda")
    mfsdp.sort_ids(torch.from_numpy(ids).to(idt).cuda(), keys, order, starts,
                   scratch(mfsdp.sort_ids_workspace_bytes(n, keys)))
    want_order, want_starts = sort_ids_ref(ids, keys)
    assert np.array_equal(order.cpu().numpy(), want_order) and np.array_equal(starts.cpu().numpy(), want_starts)


def test_sort_ids_far_outside(mfsdp):
    ids = torch.tensor([1 << 40, -(1 << 62), 1, (1 << 32) + 1, 0, 2 ** 31], device="cuda")
    order, starts = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    mfsdp.sort_ids(ids, 2, order, starts, scratch(mfsdp.sort_ids_workspace_bytes(6, 2)))
    assert order.tolist() == [4, 2, 0, 1, 3, 5] and starts.tolist() == [0, 1, 2]


# ----------------------------------------------------------------- embedding
EMB = [  # n, vocab, dim, ids
    (1, 50, 64, "uniform"), (3, 7, 1, "uniform"), (129, 33, 127, "uniform"), (257, 2000, 768, "zipf"),
    (1000, 11, 2056, "uniform"), (4000, 300, 96, "one"), (700, 40, 2500, "zipf"), (5, 9, 40, "masked"),
    (20_000, 50, 72, "zipf"),
]


def emb_ids(kind, n, vocab, rng):
    if kind == "uniform":
        return rng.integers(-1, vocab + 1, n)                 # some masked
    if kind == "zipf":
        return np.minimum(rng.zipf(1.3, n) - 1, vocab - 1)
    return np.full(n, vocab - 1 if kind == "one" else -100)


def padded(rows, width, dtype, extra, fill):
    """A rows x width view with leading dimension width + extra, and its buffer."""
    buf = torch.full((rows, width + extra), fill, device="cuda").to(DT[dtype])
    return buf[:, :width], buf


@pytest.mark.parametrize("w,out", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,vocab,dim,kind", EMB)
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_lookup(mfsdp, w, out, n, vocab, dim, kind, extra):
    rng = np.random.default_rng(n + dim)
    ids = emb_ids(kind, n, vocab, rng)
    wt, _ = padded(vocab, dim, w, extra, 5.0)
    wt.copy_(dev(rng.standard_normal((vocab, dim)), w))
    o, buf = padded(n, dim, out, extra, 7.0)
    idt = torch.int64 if n % 2 else torch.int32
    mfsdp.embedding_lookup(wt, torch.from_numpy(ids).to(idt).cuda(), o, scale=1.7)
    want = embedding_lookup_ref(host(wt), ids, 1.7)
    close(host(o), want, (2 * U + rnd(out)) * np.abs(want), "lookup")
    assert np.all(host(buf)[:, dim:] == 7.0)


@pytest.mark.parametrize("dout,grad", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("n,vocab,dim,kind", EMB)
@pytest.mark.parametrize("extra,accumulate", [(0, False), (8, True), (3, False), (5, True)])
def test_embedding_grad(mfsdp, dout, grad, n, vocab, dim, kind, extra, accumulate):
    rng = np.random.default_rng(n + dim + 1)
    ids = emb_ids(kind, n, vocab, rng)
    d, _ = padded(n, dim, dout, extra, 1e6)
    d.copy_(dev(rng.standard_normal((n, dim)), dout))
    g, buf = padded(vocab, dim, grad, extra, 7.0)
    g.copy_(dev(rng.standard_normal((vocab, dim)), grad))
    g0 = host(g)
    mfsdp.embedding_grad(d, torch.from_numpy(ids).cuda(), g, scratch(mfsdp.embedding_grad_workspace_bytes(n, vocab, dim)),
                         scale=0.6, accumulate=accumulate)
    hd = host(d)
    want = embedding_grad_ref(hd, ids, vocab, 0.6, g0 if accumulate else None)
    mag = embedding_grad_ref(np.abs(hd), ids, vocab, 0.6, np.abs(g0) if accumulate else None)
    cnt = np.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)[:, None]
    close(host(g), want, (cnt + 5) * U * mag + rnd(grad) * np.abs(want), "embedding gradient")
    if accumulate:
        assert np.array_equal(host(g)[cnt[:, 0] == 0], g0[cnt[:, 0] == 0])
    else:
        assert np.all(host(g)[cnt[:, 0] == 0] == 0.0)
    assert np.all(host(buf)[:, dim:] == 7.0)


@pytest.mark.parametrize("dout,grad", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,vocab,dim,kind", [(512, 3, 300, "one"), (513, 900, 264, "zipf"), (480, 5, 520, "uniform"),
                                              (200, 1_500_000, 8, "uniform"), (65_537, 30_000, 48, "zipf"),
                                              (90_000, 70_000, 17, "uniform"), (600, 1_300_000, 8, "uniform"),
                                              (6000, 4000, 1100, "uniform"), (2500, 9, 2048, "zipf"),
                                              (1024, 3, 264, "one"), (1025, 700, 264, "zipf"), (1000, 1, 8, "one")])
@pytest.mark.parametrize("extra,accumulate", [(0, False), (0, True), (3, True)])
def test_embedding_grad_lengths(mfsdp, dout, grad, n, vocab, dim, kind, extra, accumulate):
    """Few ids and many, few rows and many, on both sides of where the launches change."""
    test_embedding_grad(mfsdp, dout, grad, n, vocab, dim, kind, extra, accumulate)


def test_embedding_grad_masked_values_do_not_leak(mfsdp):
    """NaN and Inf in rows whose id is masked stay out of every sum."""
    d = torch.full((40, 48), float("nan"), device="cuda")
    d[::2] = 1.0
    d[1] = float("inf")
    ids = torch.tensor([3 if t % 2 == 0 else (-1, 9)[t % 4 == 1] for t in range(40)], device="cuda")
    g = torch.full((9, 48), float("nan"), device="cuda")
    mfsdp.embedding_grad(d, ids, g, scratch(mfsdp.embedding_grad_workspace_bytes(40, 9, 48)))
    want = torch.zeros_like(g)
    want[3] = 20.0
    assert torch.equal(g, want)
    g.fill_(2.0)
    mfsdp.embedding_grad(d[:0], ids[:0], g, scratch(mfsdp.embedding_grad_workspace_bytes(0, 9, 48)))
    assert torch.equal(g, torch.zeros_like(g))


def test_embedding_gradient_is_the_lookups_adjoint(mfsdp):
    """<c, lookup(w)> = <grad(c), w>, each side within its own bound."""
    rng = np.random.default_rng(8)
    n, vocab, dim = 3000, 500, 160
    ids = torch.from_numpy(emb_ids("uniform", n, vocab, rng)).cuda()
    w, c = dev(rng.standard_normal((vocab, dim))), dev(rng.standard_normal((n, dim)))
    o, g = torch.empty_like(c), torch.empty_like(w)
    mfsdp.embedding_lookup(w, ids, o, scale=2.0)
    mfsdp.embedding_grad(c, ids, g, scratch(mfsdp.embedding_grad_workspace_bytes(n, vocab, dim)), scale=2.0)
    a, b = np.sum(host(c) * host(o)), np.sum(host(g) * host(w))
    cnt = int(torch.bincount(ids.clamp(0, vocab - 1)).max())
    assert abs(a - b) <= (cnt + 8) * U * np.sum(np.abs(host(c) * host(o)))


# ------------------------------------------------------- products by expert
EXP = [  # rows of each expert, rows, cols
    ([1], 8, 8), ([1], 64, 64), ([3, 0, 5], 1, 1), ([0, 0, 7, 0], 72, 40), ([130, 1, 0, 16], 200, 136),
    ([300], 256, 128), ([64, 257, 15, 0, 33], 331, 515), ([17, 0, 129], 128, 1000), ([2] * 40, 24, 48),
    ([0, 0], 16, 16), ([513, 255], 384, 264),
]


def expert_case(counts, rows, cols, extra, tail, seed):
    rng = np.random.default_rng(seed + rows + cols)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(starts[-1]) + tail
    x, _ = padded(n, cols, "bf16", extra, 1e4)
    dy, _ = padded(n, rows, "bf16", extra, 1e4)
    x.copy_(dev(rng.standard_normal((n, cols)), "bf16"))
    dy.copy_(dev(rng.standard_normal((n, rows)), "bf16"))
    w = torch.full((len(counts), rows * cols + extra), 1e4, device="cuda").to(torch.bfloat16)
    w = w[:, :rows * cols].unflatten(1, (rows, cols))
    w.copy_(dev(rng.standard_normal(tuple(w.shape)), "bf16"))
    return n, starts, torch.from_numpy(starts).cuda(), x, dy, w


def expert_ws(m, w, n, x, dy):
    e, rows, cols = w.shape
    ld = lambda t, width: t.stride(0) if t.shape[0] > 1 else width
    return scratch(m.expert_workspace_bytes(e, rows, cols, n, w_stride=w.stride(0) if e > 1 else None,
                                            rows_ld=ld(dy, rows), cols_ld=ld(x, cols)))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,rows,cols", EXP)
@pytest.mark.parametrize("extra,tail", [(0, 0), (8, 2), (3, 0)])
@pytest.mark.parametrize("input_grad", [False, True])
def test_expert_matmul(mfsdp, out, counts, rows, cols, extra, tail, input_grad):
    n, starts, dstarts, x, dy, w = expert_case(counts, rows, cols, extra, tail, 1)
    a, width, k = (dy, cols, rows) if input_grad else (x, rows, cols)
    y, buf = padded(n, width, out, extra, 7.0)
    mfsdp.expert_matmul(a, w, dstarts, y, expert_ws(mfsdp, w, n, x if not input_grad else y, y if not input_grad else dy),
                        input_grad=input_grad)
    want = expert_matmul_ref(host(a), host(w), starts, input_grad)
    mag = expert_matmul_ref(np.abs(host(a)), np.abs(host(w)), starts, input_grad)
    close(host(y), want, max(k, 32) * U * mag + rnd(out) * np.abs(want), "expert product")
    assert np.all(host(y)[starts[-1]:] == 0.0)
    assert np.all(host(buf)[:, width:] == 7.0)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,rows,cols", [([1] * 16, 100, 1096), ([16], 37, 2056), ([5, 0, 11], 64, 300), ([4] * 4, 9, 8),
                                              ([0, 1, 0], 1408, 2048), ([17], 65, 1000), ([3, 1, 0, 2] * 2, 33, 4099)])
@pytest.mark.parametrize("extra,tail", [(0, 0), (8, 3), (3, 1)])
def test_expert_matmul_few_tokens(mfsdp, out, counts, rows, cols, extra, tail):
    test_expert_matmul(mfsdp, out, counts, rows, cols, extra, tail, False)


@pytest.mark.parametrize("out,accumulate", [("bf16", False), ("f32", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("counts,rows,cols", EXP)
@pytest.mark.parametrize("extra,tail", [(0, 0), (8, 2), (3, 0)])
def test_expert_weight_grad(mfsdp, out, accumulate, counts, rows, cols, extra, tail):
    n, starts, dstarts, x, dy, w = expert_case(counts, rows, cols, extra, tail, 2)
    if tail:
        x[-tail:] = float("nan")                       # rows of no expert
        dy[-tail:] = float("inf")
    rng = np.random.default_rng(3)
    flat = torch.full((len(counts), rows * cols + extra), 7.0, device="cuda").to(DT[out])
    dw = flat[:, :rows * cols].unflatten(1, (rows, cols))
    dw.copy_(dev(rng.standard_normal(tuple(dw.shape)), out))
    dw0 = host(dw)
    mfsdp.expert_weight_grad(dy, x, dstarts, dw, expert_ws(mfsdp, w, n, x, dy), accumulate=accumulate)
    hx, hdy = host(x), host(dy)
    want = expert_weight_grad_ref(hdy, hx, starts, dw0 if accumulate else None)
    mag = expert_weight_grad_ref(np.abs(hdy), np.abs(hx), starts, np.abs(dw0) if accumulate else None)
    k = np.maximum(np.asarray(counts), 32)[:, None, None] + 1
    close(host(dw), want, k * U * mag + rnd(out) * np.abs(want), "weight gradient")
    assert np.all(host(flat)[:, rows * cols:] == 7.0)


@pytest.mark.parametrize("out,accumulate", [("bf16", False), ("f32", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("counts,rows,cols", [([4096], 64, 72), ([11_003], 300, 260), ([4096, 0, 1, 700], 130, 264),
                                              ([0, 9000], 1000, 500), ([2048, 2049, 2047, 2040], 33, 21)])
@pytest.mark.parametrize("extra,tail", [(0, 0), (3, 5)])
def test_expert_weight_grad_long_groups(mfsdp, out, accumulate, counts, rows, cols, extra, tail):
    """Few tiles and many tokens: the contraction is cut, and its parts added."""
    test_expert_weight_grad(mfsdp, out, accumulate, counts, rows, cols, extra, tail)


def test_expert_weight_grad_starts_that_fall(mfsdp):
    """Starts outside the rows are clamped, and a group that ends before it starts
    is empty: the experts beside it still get theirs, and nothing else is written."""
    n, rows, cols = 6000, 64, 40
    rng = np.random.default_rng(8)
    dy, x = dev(rng.standard_normal((n, rows)), "bf16"), dev(rng.standard_normal((n, cols)), "bf16")
    starts = torch.tensor([0, 5000, 200, 90_000, -4], dtype=torch.int32, device="cuda")
    flat = torch.full((4 * rows * cols + 64,), 7.0, device="cuda")
    dw = flat[:4 * rows * cols].view(4, rows, cols)
    ws = scratch(mfsdp.expert_workspace_bytes(4, rows, cols, n))
    mfsdp.expert_weight_grad(dy, x, starts, dw, ws)
    assert mfsdp.op_device_status(ws)[0] == 0
    hx, hdy, got = host(x), host(dy), host(dw)
    for e, (lo, hi) in enumerate([(0, 5000), (0, 0), (200, 6000), (0, 0)]):
        want, mag = hdy[lo:hi].T @ hx[lo:hi], np.abs(hdy[lo:hi]).T @ np.abs(hx[lo:hi])
        close(got[e], want, (max(hi - lo, 32) + 1) * U * mag + U * np.abs(want), f"expert {e}")
    assert torch.all(flat[4 * rows * cols:] == 7.0)


def test_expert_neighbours_do_not_leak(mfsdp):
    """NaN and Inf in one expert's rows or matrix stay inside that expert."""
    counts, rows, cols = [19, 45, 8, 37], 96, 72
    n, starts, dstarts, x, dy, w = expert_case(counts, rows, cols, 0, 0, 4)
    x[19:64], dy[19:64], w[1] = float("nan"), float("inf"), float("nan")
    ws = expert_ws(mfsdp, w, n, x, dy)
    y, dx = torch.empty(n, rows, device="cuda"), torch.empty(n, cols, device="cuda")
    dw = torch.empty(4, rows, cols, device="cuda")
    mfsdp.expert_matmul(x, w, dstarts, y, ws)
    mfsdp.expert_matmul(dy, w, dstarts, dx, ws, input_grad=True)
    mfsdp.expert_weight_grad(dy, x, dstarts, dw, ws)
    for t in (y, dx):
        assert torch.isfinite(t[:19]).all() and torch.isfinite(t[64:]).all() and not torch.isfinite(t[19:64]).any()
    assert torch.isfinite(dw[[0, 2, 3]]).all() and not torch.isfinite(dw[1]).any()


@pytest.mark.parametrize("experts,n", [(128, 8), (1024, 16), (300, 13)])
def test_expert_matmul_few_tokens_of_many_experts(mfsdp, experts, n):
    """Experts that different warps look at, on every SM: all rows of all tokens are there."""
    rng = np.random.default_rng(experts)
    counts = np.zeros(experts, np.int64)
    np.add.at(counts, rng.integers(0, experts, n), 1)
    for _ in range(5):
        test_expert_matmul(mfsdp, "f32", list(counts), 700, 264, 0, 0, False)


@pytest.mark.parametrize("counts,rows,cols", [([40, 0, 300], 72, 5000), ([17, 33], 4100, 2049), ([7000], 2100, 1304),
                                              ([2100, 5001], 1100, 1299)])
@pytest.mark.parametrize("extra,accumulate", [(0, False), (3, True)])
def test_expert_long_contractions(mfsdp, counts, rows, cols, extra, accumulate):
    """Contractions past what one accumulator takes, in each of the products."""
    for grad in (False, True):
        test_expert_matmul(mfsdp, "f32", counts, rows, cols, extra, 0, grad)
    test_expert_weight_grad(mfsdp, "f32", accumulate, counts, rows, cols, extra, 0)


@pytest.mark.parametrize("k", [2048, 16_384, 70_000])
def test_expert_fp32_outputs_keep_their_bits(mfsdp, k):
    """Positive operands, so no partial sum is larger than the result: 2048 / 16 + 1
    additions on a tensor core, each cutting off 2 u of it at most, and k / 2048 + 1
    rounded ones."""
    rng = np.random.default_rng(k)
    bound = (2 * 129 + k / 2048 + 1) * U
    x, w = dev(np.abs(rng.standard_normal((64, k))), "bf16"), dev(np.abs(rng.standard_normal((1, 96, k))), "bf16")
    starts = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    y = torch.empty(64, 96, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, scratch(mfsdp.expert_workspace_bytes(1, 96, k, 64)))
    want = host(x) @ host(w)[0].T
    close(host(y), want, bound * want, "forward")
    starts[1] = k
    dy, xs = x.T.contiguous(), w[0].T.contiguous()
    dy, xs = torch.cat([dy] * 40, 1), torch.cat([xs] * 10, 1)                     # 2560 x 960: not cut for the GPU's sake
    dw = torch.empty(1, 2560, 960, device="cuda")
    mfsdp.expert_weight_grad(dy, xs, starts, dw, scratch(mfsdp.expert_workspace_bytes(1, 2560, 960, k)))
    got = host(dw)[0].reshape(40, 64, 10, 96)
    close(got, np.broadcast_to(want[None, :, None, :], got.shape), bound * want[None, :, None, :], "weight gradient")
    wt = w.transpose(1, 2).contiguous()                                           # k rows: the input gradient's contraction
    dxx = torch.empty(64, 96, device="cuda")
    starts[1] = 64
    mfsdp.expert_matmul(x, wt, starts, dxx, scratch(mfsdp.expert_workspace_bytes(1, k, 96, 64)), input_grad=True)
    close(host(dxx), want, bound * want, "input gradient")


@pytest.mark.parametrize("n,rows,cols", [(70, 37, 301), (9, 45, 29), (300, 131, 1021)])
def test_expert_padding_is_neither_read_nor_written(mfsdp, n, rows, cols):
    """Rows that end inside 16 bytes, with NaN between them."""
    up = lambda v: -(-v // 8) * 8
    rng = np.random.default_rng(n)
    nan = float("nan")
    starts = torch.tensor([0, n // 3, n], dtype=torch.int32, device="cuda")
    x, _ = padded(n, cols, "bf16", up(cols) - cols, nan)
    dy, _ = padded(n, rows, "bf16", up(rows) - rows, nan)
    x.copy_(dev(rng.standard_normal((n, cols)), "bf16"))
    dy.copy_(dev(rng.standard_normal((n, rows)), "bf16"))
    w = dev(rng.standard_normal((2, rows, cols)), "bf16")
    ws = scratch(mfsdp.expert_workspace_bytes(2, rows, cols, n, rows_ld=up(rows), cols_ld=up(cols)))
    y, ybuf = padded(n, rows, "f32", up(rows) - rows, 7.0)
    dx, dxbuf = padded(n, cols, "bf16", up(cols) - cols, 7.0)
    dw = torch.empty(2, rows, cols, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, ws)
    mfsdp.expert_matmul(dy, w, starts, dx, ws, input_grad=True)
    mfsdp.expert_weight_grad(dy, x, starts, dw, ws)
    hs, hx, hdy, hw = starts.cpu().numpy(), host(x), host(dy), host(w)
    for got, a, grad, k, h in ((y, hx, False, cols, U), (dx, hdy, True, rows, H)):
        want, mag = expert_matmul_ref(a, hw, hs, grad), expert_matmul_ref(np.abs(a), np.abs(hw), hs, grad)
        close(host(got), want, max(k, 32) * U * mag + h * np.abs(want), "product")
    want = expert_weight_grad_ref(hdy, hx, hs, None)
    mag = expert_weight_grad_ref(np.abs(hdy), np.abs(hx), hs, None)
    close(host(dw), want, (n + 33) * U * mag + U * np.abs(want), "weight gradient")
    assert torch.all(ybuf[:, rows:] == 7.0) and torch.all(dxbuf[:, cols:] == 7.0)


def test_expert_gradients_are_adjoints(mfsdp):
    """<c, y(x, w)> = <dx(c), x> = <dw(c), w>, within the products' own bounds."""
    counts, rows, cols = [70, 0, 33, 128], 136, 264
    n, starts, dstarts, x, c, w = expert_case(counts, rows, cols, 0, 0, 5)
    ws = expert_ws(mfsdp, w, n, x, c)
    y, dx = torch.empty(n, rows, device="cuda"), torch.empty(n, cols, device="cuda")
    dw = torch.empty(4, rows, cols, device="cuda")
    mfsdp.expert_matmul(x, w, dstarts, y, ws)
    mfsdp.expert_matmul(c, w, dstarts, dx, ws, input_grad=True)
    mfsdp.expert_weight_grad(c, x, dstarts, dw, ws)
    a, b, d = np.sum(host(c) * host(y)), np.sum(host(dx) * host(x)), np.sum(host(dw) * host(w))
    mag = np.sum(np.abs(host(c)) * expert_matmul_ref(np.abs(host(x)), np.abs(host(w)), starts))
    assert abs(a - b) <= 2 * cols * U * mag and abs(a - d) <= 2 * cols * U * mag


# -------------------------------------------------------- streams and graphs
def test_operators_on_another_stream_and_in_a_graph(mfsdp):
    """The whole chain queued on a side stream, then captured and replayed:
    the same bits as on the default stream."""
    rng = np.random.default_rng(9)
    vocab, dim, n, e, rows = 90, 64, 300, 5, 48
    table = dev(rng.standard_normal((vocab, dim)))
    w = dev(rng.standard_normal((e, rows, dim)), "bf16")
    ids, expert = torch.from_numpy(rng.integers(0, vocab, n)).cuda(), torch.from_numpy(rng.integers(0, e, n)).cuda()
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")

    class Bufs:
        def __init__(self):
            self.order, self.starts = z(n, d=torch.int32), z(e + 1, d=torch.int32)
            self.h, self.hs, self.y = z(n, dim, d=torch.bfloat16), z(n, dim, d=torch.bfloat16), z(n, rows, d=torch.bfloat16)
            self.dx, self.dw, self.dtab = z(n, dim), z(e, rows, dim), z(vocab, dim)
            self.norm = z(2)
            self.set = mfsdp.grad_set([self.dw, self.dtab])
            self.ws = [scratch(k) for k in (mfsdp.sort_ids_workspace_bytes(n, e),
                                            mfsdp.expert_workspace_bytes(e, rows, dim, n),
                                            mfsdp.embedding_grad_workspace_bytes(n, vocab, dim),
                                            mfsdp.grad_clip_workspace_bytes(self.set))]

        def run(self):
            mfsdp.embedding_lookup(table, ids, self.h)
            mfsdp.sort_ids(expert, e, self.order, self.starts, self.ws[0])
            mfsdp.embedding_lookup(self.h, self.order, self.hs)
            mfsdp.expert_matmul(self.hs, w, self.starts, self.y, self.ws[1])
            mfsdp.expert_matmul(self.y, w, self.starts, self.dx, self.ws[1], input_grad=True)
            mfsdp.expert_weight_grad(self.y, self.hs, self.starts, self.dw, self.ws[1])
            mfsdp.embedding_grad(self.dx, ids, self.dtab, self.ws[2])
            mfsdp.grad_clip(self.set, self.norm, self.ws[3], max_norm=1.0)

        def results(self):
            return [self.order, self.starts, self.y, self.dx, self.dw, self.dtab, self.norm]

    ref = Bufs()
    ref.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = Bufs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref.results(), b.results()))
    c = Bufs()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref.results(), c.results()))
