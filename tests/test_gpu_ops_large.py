"""The operators on tensors of more than 2^31 elements, checked on rows at their
ends and at random in fp64.  (Tolerances as in test_gpu_ops.py.)
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
ROWS, DIM = 280_000, 8192                      # 2.3e9 elements


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    yield
    torch.cuda.empty_cache()


def scratch(n):
    return torch.full((int(n),), 0xFF, dtype=torch.uint8, device="cuda")


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), f"{what}: {float(err.max()):.3e}"


def table(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def test_embedding(mfsdp):
    w = table(ROWS, DIM, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, ROWS, (ROWS,), generator=g, device="cuda")
    ids[:3], ids[-3:] = torch.tensor([ROWS - 1, 0, ROWS - 1]), torch.tensor([ROWS - 1, 1, ROWS - 2])
    out = torch.empty_like(w)
    mfsdp.embedding_lookup(w, ids, out, scale=0.5)
    pick = torch.cat([torch.tensor([0, 1, 2, ROWS - 3, ROWS - 2, ROWS - 1], device="cuda"),
                      torch.randint(0, ROWS, (500,), generator=g, device="cuda")])
    assert torch.equal(out[pick], (w[ids[pick]].float() * 0.5).bfloat16())        # a power of two: exact
    grad = w                                                                      # (written over)
    ws = scratch(mfsdp.embedding_grad_workspace_bytes(ROWS, ROWS, DIM))
    mfsdp.embedding_grad(out, ids, grad, ws, scale=0.5)
    assert mfsdp.op_device_status(ws)[0] == 0
    for v in [0, 1, ROWS - 2, ROWS - 1] + [int(i) for i in ids[pick[6:60]]] + list(range(1000, 1050)):
        rows = out[(ids == v).nonzero()[:, 0]].double()
        want, mag = 0.5 * rows.sum(0), 0.5 * rows.abs().sum(0)
        within(grad[v], want, (len(rows) + 5) * U * mag + H * want.abs(), f"row {v}")


@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_of_the_widest_rows(mfsdp, accumulate):
    dim = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(9)
    ids = torch.tensor([1, 4, 1], device="cuda")
    w, dout = torch.randn(5, dim, generator=g, device="cuda"), torch.randn(3, dim, generator=g, device="cuda")
    out = torch.empty(3, dim, device="cuda")
    mfsdp.embedding_lookup(w, ids, out)
    assert torch.equal(out, w[ids])
    ws = scratch(mfsdp.embedding_grad_workspace_bytes(3, 5, dim))
    want = (w.double() if accumulate else torch.zeros_like(w, dtype=torch.float64)).index_add(0, ids, dout.double())
    mag = (w.abs().double() if accumulate else torch.zeros_like(w, dtype=torch.float64)).index_add(0, ids, dout.abs().double())
    mfsdp.embedding_grad(dout, ids, w, ws, accumulate=accumulate)
    within(w, want, 6 * U * mag, "gradient")


def test_clip(mfsdp):
    n = ROWS * DIM + 5
    flat = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    total = sum(float(c.double().square().sum()) for c in flat.split(1 << 26))
    s = mfsdp.grad_set([flat[:7], flat[7:]])
    keep = torch.cat([flat[:4096], flat[-4096:]]).double()
    out = torch.empty(2, device="cuda")
    ws = scratch(mfsdp.grad_clip_workspace_bytes(s))
    mfsdp.grad_clip(s, out, ws, max_norm=1.0)
    norm = total ** 0.5
    assert abs(float(out[0]) - norm) <= 7 * U * norm
    want = keep / (norm + 1e-6)
    within(torch.cat([flat[:4096], flat[-4096:]]), want, (9 * U + H) * want.abs(), "clipped")
    after = sum(float(c.double().square().sum()) for c in flat.split(1 << 26)) ** 0.5
    assert abs(after - 1.0) <= H + 9 * U


def test_expert_stack(mfsdp):
    """A stack of matrices, and its gradient, of 2.4e9 elements."""
    e, rows, cols, n = 560, 2048, 2100, 1120
    w = table(e * rows, cols, 4).view(e, rows, cols)
    x, dy = table(n, cols, 5), table(n, rows, 6)
    starts = torch.arange(0, n + 1, 2, dtype=torch.int32, device="cuda")
    ws = scratch(mfsdp.expert_workspace_bytes(e, rows, cols, n))
    y, dx = torch.empty(n, rows, device="cuda"), torch.empty(n, cols, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, ws)
    mfsdp.expert_matmul(dy, w, starts, dx, ws, input_grad=True)
    assert mfsdp.op_device_status(ws)[0] == 0
    for i in (0, 1, 300, 498, 499, 500, 558, 559):
        m, a, d = w[i].double(), x[2 * i:2 * i + 2].double(), dy[2 * i:2 * i + 2].double()
        within(y[2 * i:2 * i + 2], a @ m.T, cols * U * (a.abs() @ m.abs().T) + U * (a @ m.T).abs(), f"y of {i}")
        within(dx[2 * i:2 * i + 2], d @ m, rows * U * (d.abs() @ m.abs()) + U * (d @ m).abs(), f"dx of {i}")
    mfsdp.expert_weight_grad(dy, x, starts, w, ws)                                # (written over)
    assert mfsdp.op_device_status(ws)[0] == 0
    for i in (0, 1, 300, 498, 499, 500, 558, 559):
        a, d = x[2 * i:2 * i + 2].double(), dy[2 * i:2 * i + 2].double()
        within(w[i], d.T @ a, 33 * U * (d.abs().T @ a.abs()) + H * (d.T @ a).abs(), f"dw of {i}")


def test_expert_activations(mfsdp):
    """Activations of 2.3e9 elements, for two experts."""
    n, cols, rows = 560_000, 4096, 64
    x, w, dy = table(n, cols, 7), table(2 * rows, cols, 8).view(2, rows, cols), table(n, rows, 9)
    starts = torch.tensor([0, 30_001, n - 3], dtype=torch.int32, device="cuda")
    ws = scratch(mfsdp.expert_workspace_bytes(2, rows, cols, n))
    y = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(2, rows, cols, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, ws)
    mfsdp.expert_weight_grad(dy, x, starts, dw, ws)
    pick = torch.tensor([0, 30_000, 30_001, 524_287, 524_288, 524_289, n - 4], device="cuda")
    for t in pick.tolist():
        m, a = w[0 if t < 30_001 else 1].double(), x[t].double()
        want = m @ a
        within(y[t], want, cols * U * (m.abs() @ a.abs()) + H * want.abs(), f"token {t}")
    assert not y[n - 3:].any()
    for e, (lo, hi) in enumerate([(0, 30_001), (30_001, n - 3)]):
        want, mag = (torch.zeros(rows, cols, dtype=torch.float64, device="cuda") for _ in range(2))
        for at in range(lo, hi, 1 << 16):
            a, d = x[at:min(hi, at + (1 << 16))].double(), dy[at:min(hi, at + (1 << 16))].double()
            want += d.T @ a
            mag += d.abs().T @ a.abs()
        within(dw[e], want, (hi - lo + 1) * U * mag + U * want.abs(), f"dw of {e}")
    x2 = x
    mfsdp.expert_matmul(dy, w, starts, x2, ws, input_grad=True)                   # (written over)
    for t in pick.tolist():
        m, d = w[0 if t < 30_001 else 1].double(), dy[t].double()
        want = d @ m
        within(x2[t], want, rows * U * (d.abs() @ m.abs()) + H * want.abs(), f"dx of {t}")
    assert not x2[n - 3:].any()
    assert mfsdp.op_device_status(ws)[0] == 0
