"""GPU cases of the operators next to the owner step that earlier tests leave out.
(Helpers and the derivation of the tolerances: test_gpu_ops.py.)
"""
import threading

import numpy as np
import pytest

from oracle.ops import grad_clip_ref
from tests.test_gpu_ops import U, scratch, test_embedding_grad as check_embedding_grad, \
    test_expert_matmul as check_matmul, test_expert_weight_grad as check_weight_grad, test_sort_ids as check_sort

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# ------------------------------------------------------------ norm, clipping
@pytest.mark.parametrize("limit", [float("inf"), 1.0, 0.0])
@pytest.mark.parametrize("bad,at", [("nan", 0), ("nan", 69_999), ("inf", 1), ("-inf", 40_000)])
def test_norm_that_is_no_number(mfsdp, limit, bad, at):
    """A NaN reaches both outputs at any limit, so that a caller who looks at the
    coefficient alone sees it; an infinite norm is clipped to nothing by a finite limit
    and by an infinite one not at all."""
    x = torch.ones(70_000, device="cuda")
    x[at] = float(bad)
    want = list(grad_clip_ref([x.double().cpu().numpy()], limit, 1e-6)[:2])
    assert np.array_equal(want, [np.nan, np.nan] if bad == "nan" else [np.inf, float(limit == np.inf)], equal_nan=True)
    s, out = mfsdp.grad_set([x], [torch.empty_like(x)]), torch.full((2,), 7.0, device="cuda")
    ws = scratch(mfsdp.grad_clip_workspace_bytes(s))
    mfsdp.grad_norm(s, out, ws, max_norm=limit)
    assert np.array_equal(out.tolist(), want, equal_nan=True)
    out.fill_(7.0)
    mfsdp.grad_clip(s, out, ws, max_norm=limit)
    assert np.array_equal(out.tolist(), want, equal_nan=True)
    if bad == "nan":
        assert torch.isnan(s.dsts[0]).all()


# ------------------------------------------------------- products by expert
def positive(*shape, seed):
    """Magnitudes of normal bf16 values: no sum of their products is larger than the whole."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(generator=g).abs_().bfloat16()


def rounded_once(got, want, k, what):
    """A bf16 output is the rounding of a value whose error comes from the sums alone: an accumulator
    takes 32768 of the contraction at most, 2048 additions of 16 products that cut off 2 u
    each, then a rounded addition for each accumulator.  Rounding is monotone, so the output
    lies between the rounded ends of that interval."""
    sums = (2 * 2048 + k / 32768 + 2) * U
    low, high = ((want * (1 + s)).bfloat16() for s in (-sums, sums))
    bad = (got < low) | (got > high)
    rel = (got.double() - want) / want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, mean error {float(rel.mean()):.3e}"


@pytest.mark.parametrize("rows,cols", [(96, 960), (93, 955)])
def test_bf16_outputs_of_a_million_long_contraction(mfsdp, rows, cols):
    """(93 and 955: no row of an output starts on a 16-byte boundary.)"""
    k = 1 << 20
    x, w = positive(64, k, seed=1), positive(1, rows, k, seed=2)
    starts = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    want = x.double() @ w[0].double().T
    y = torch.empty(64, rows, dtype=torch.bfloat16, device="cuda")
    ws = scratch(mfsdp.expert_workspace_bytes(1, rows, k, 64))
    mfsdp.expert_matmul(x, w, starts, y, ws)
    rounded_once(y, want, k, "forward")
    wt = w.transpose(1, 2).contiguous()                                # the input gradient contracts over rows
    ws = scratch(mfsdp.expert_workspace_bytes(1, k, rows, 64))
    mfsdp.expert_matmul(x, wt, starts, y, ws, input_grad=True)
    rounded_once(y, want, k, "input gradient")
    del w, wt, want
    # 2560 x 960: tiles for every SM, so that the contraction is not cut for theirs
    base = positive(k, 80, seed=3)
    xs = base.repeat(1, 12)[:, :cols].contiguous()
    dy = x.T.contiguous().repeat(1, 40)
    want = (x.double() @ base.double()).repeat(40, 12)[:, :cols]
    starts[1] = k
    ws = scratch(mfsdp.expert_workspace_bytes(1, 2560, cols, k))
    dw = torch.empty(1, 2560, cols, dtype=torch.bfloat16, device="cuda")
    mfsdp.expert_weight_grad(dy, xs, starts, dw, ws)
    rounded_once(dw[0], want, k, "weight gradient")
    before = dw.clone()
    mfsdp.expert_weight_grad(dy, xs, starts, dw, ws, accumulate=True)
    rounded_once(dw[0], want + before[0].double(), k, "weight gradient added")
    assert mfsdp.op_device_status(ws)[0] == 0


@pytest.mark.parametrize("counts,k", [([40, 300], 32_768), ([17, 0, 33], 32_769), ([260], 65_537), ([33, 5], 100_008)])
@pytest.mark.parametrize("extra", [0, 3])
def test_bf16_outputs_over_several_accumulators(mfsdp, counts, k, extra):
    """On both sides of one accumulator's contraction, groups beside each other, and tiles of one
    and of two chunks of columns."""
    check_matmul(mfsdp, "bf16", counts, 72, k, extra, 2, False)
    check_matmul(mfsdp, "bf16", counts, k, 40, extra, 2, True)


@pytest.mark.parametrize("counts", [[32_768, 70], [40_001, 5, 65_700, 1030]])
@pytest.mark.parametrize("extra,accumulate", [(0, False), (0, True), (3, False), (3, True)])
def test_bf16_weight_gradients_over_several_accumulators(mfsdp, counts, extra, accumulate):
    """Tiles of one accumulator among tiles of several; 300 x 1800 in tiles of 256 x 256, 16 of them, so
    that groups are not cut for the GPU's sake."""
    check_weight_grad(mfsdp, "bf16", accumulate, counts, 300, 1800, extra, 0)


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("k", [1025, 2048, 16_384, 70_000])
def test_fp32_outputs_in_the_2_norm(mfsdp, k):
    """Normal operands.  A turn of 1024 is 64 additions of 16 products; each cuts off up to a unit of
    the partial sum p, half a unit in the mean, which is 0.72 u |p| (u = 2^-24; the mean of
    a unit over p's place between two powers of two), always towards zero.  The partial sums
    of N terms that are independent add up to N / sqrt(3) of the last one: 0.72 * 64 / sqrt(3) =
    26.6 u of the turn's result, and 27 with the cuts' spread about their mean.  The
    turns' errors are independent of each other, so they are 27 u of the whole; the T rounded
    additions that join them are off by 0.42 u of the sums so far, 0.3 sqrt(T) u.  (Turns of 2048
    would be 53 u by this count, and were measured at 35.)"""
    g = torch.Generator(device="cuda").manual_seed(k)
    normal = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g).bfloat16()
    bound = (27 + 0.3 * (k / 1024 + 1) ** 0.5) * U
    x, w = normal(64, k), normal(1, 96, k)
    want = x.double() @ w[0].double().T
    starts = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    y = torch.empty(64, 96, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, scratch(mfsdp.expert_workspace_bytes(1, 96, k, 64)))
    assert relative(y, want) <= bound, "forward"
    wt = w.transpose(1, 2).contiguous()                               # k rows: the input gradient's contraction
    mfsdp.expert_matmul(x, wt, starts, y, scratch(mfsdp.expert_workspace_bytes(1, k, 96, 64)), input_grad=True)
    assert relative(y, want) <= bound, "input gradient"
    # few tokens: a lane adds k / 32 products one after the other, rounded, 0.42 u each of a sum that
    # grows like their root: 0.3 sqrt(k / 32) u; a third more, and the lanes' five
    starts[1] = 16
    mfsdp.expert_matmul(x[:16], w, starts, y[:16], scratch(mfsdp.expert_workspace_bytes(1, 96, k, 16)))
    assert relative(y[:16], want[:16]) <= (0.4 * (k / 32) ** 0.5 + 5) * U, "few tokens"
    starts[1] = k
    dy, xs = x.T.contiguous(), wt[0]
    for rows, cols in ((64, 96), (2560, 960)):                        # cut for the GPU's sake, and not
        a, b = dy.repeat(1, rows // 64), xs.repeat(1, cols // 96)
        dw = torch.empty(1, rows, cols, device="cuda")
        mfsdp.expert_weight_grad(a, b, starts, dw, scratch(mfsdp.expert_workspace_bytes(1, rows, cols, k)))
        assert relative(dw[0], want.repeat(rows // 64, cols // 96)) <= bound, f"weight gradient {rows} x {cols}"


@pytest.mark.parametrize("k", [1025, 2048, 16_384, 70_000])
def test_fp32_outputs_element_by_element(mfsdp, k):
    """Magnitudes: no partial sum is larger than the result.  A turn is 64 additions, and one more to
    start with, which cut off 2 u each at most; joining T turns is T + 1 rounded additions."""
    bound = (2 * 65 + k / 1024 + 2) * U
    x, w = positive(64, k, seed=k), positive(1, 96, k, seed=k + 1)
    want = x.double() @ w[0].double().T
    starts = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    y = torch.empty(64, 96, device="cuda")
    mfsdp.expert_matmul(x, w, starts, y, scratch(mfsdp.expert_workspace_bytes(1, 96, k, 64)))
    assert float(((y.double() - want) / want).abs().max()) <= bound, "forward"
    wt = w.transpose(1, 2).contiguous()
    mfsdp.expert_matmul(x, wt, starts, y, scratch(mfsdp.expert_workspace_bytes(1, k, 96, 64)), input_grad=True)
    assert float(((y.double() - want) / want).abs().max()) <= bound, "input gradient"
    starts[1] = k
    a, b = x.T.repeat(1, 40).contiguous(), wt[0].repeat(1, 10)
    dw = torch.empty(1, 2560, 960, device="cuda")
    mfsdp.expert_weight_grad(a, b, starts, dw, scratch(mfsdp.expert_workspace_bytes(1, 2560, 960, k)))
    want = want.repeat(40, 10)
    assert float(((dw[0].double() - want) / want).abs().max()) <= bound, "weight gradient"


# ----------------------------------------------------------------- embedding
@pytest.mark.parametrize("n,vocab,dim,grad,accumulate,sorts", [
    (512, 32_000, 2048, "f32", False, False), (513, 32_000, 2048, "f32", False, True),
    (1024, 32_000, 1024, "f32", False, True), (1024, 32_000, 1024, "f32", True, False),
    (1024, 32_000, 256, "f32", False, False), (1024, 32_768, 264, "f32", False, True),
    (1024, 32_768, 264, "bf16", False, False), (1025, 1000, 64, "bf16", True, True),
    (512, 32_000, 375, "f32", False, False), (257, 13_000, 1365, "f32", False, True),
    (256, 13_000, 1365, "f32", False, False),
    (512, 32_000, 1365, "f32", True, False), (513, 100, 9, "f32", True, False), (1025, 100, 9, "f32", True, True),
    (1024, 5000, 1365, "f32", False, False), (1024, 6500, 1365, "f32", False, True),
    (0, 40_000, 2048, "f32", False, False),
])
def test_embedding_grad_of_few_ids_beside_many_rows(mfsdp, n, vocab, dim, grad, accumulate, sorts):
    """On both sides of where few ids go through the sort: which way a call took shows in its
    workspace, where the sort leaves its keys."""
    check_embedding_grad(mfsdp, "bf16", grad, max(n, 1), vocab, dim, "zipf", 0, accumulate)
    ids = torch.arange(n, device="cuda") % vocab
    dout = torch.zeros(n, dim, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(vocab, dim, device="cuda").to({"f32": torch.float32, "bf16": torch.bfloat16}[grad])
    ws = scratch(mfsdp.embedding_grad_workspace_bytes(n, vocab, dim))
    mfsdp.embedding_grad(dout, ids, g, ws, accumulate=accumulate)
    assert mfsdp.op_device_status(ws)[0] == 0 or (n == 0 and accumulate)
    assert bool((ws[256:256 + 4 * n] != 0xFF).any()) == sorts


# ------------------------------------------------------------------- id sort
@pytest.mark.parametrize("n", [20_001, 32_768, 40_000, 65_535, 65_536, 65_537])
@pytest.mark.parametrize("keys", [3, 128, 32_000, 70_000])
def test_sort_of_as_many_ids_as_a_cluster_holds(mfsdp, n, keys):
    """Three to eight pairs a thread, and on both sides of the last length that one cluster sorts."""
    check_sort(mfsdp, torch.int64, n, keys)


# ------------------------------------------- streams, graphs, threads, repeats
class Chain:
    """Every operator once, at sizes that take the ways of several launches: a sort in a
    cluster, slabs that cut rows, fp32 products in turns, a weight gradient that is cut and one that
    adds, and clipping of more than one chunk a tensor.  dim 1101: no row starts on a 16-byte boundary."""

    def __init__(self, m, dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.m, vocab, n, e, rows = m, 3000, 6000, 2, 320

        def normal(*shape, dtype=torch.float32):
            return torch.empty(shape, device="cuda").normal_(generator=g).to(dtype)

        def new(*shape, dtype=torch.float32):
            return torch.full(shape, 7, dtype=dtype, device="cuda")

        rng = np.random.default_rng(seed)
        self.table, self.w = normal(vocab, dim), normal(e, rows, dim, dtype=torch.bfloat16)
        self.ids = torch.from_numpy(np.minimum(rng.zipf(1.3, n) - 1, vocab)).cuda()      # some masked
        self.expert = torch.from_numpy(rng.integers(0, e, n)).cuda()
        self.order, self.starts = new(n, dtype=torch.int32), new(e + 1, dtype=torch.int32)
        self.h, self.hs = new(n, dim, dtype=torch.bfloat16), new(n, dim, dtype=torch.bfloat16)
        self.y, self.yb = new(n, rows), new(n, rows, dtype=torch.bfloat16)
        self.dx, self.dw, self.dwb = new(n, dim), new(e, rows, dim), new(e, rows, dim, dtype=torch.bfloat16)
        self.dtab, self.norm = new(vocab, dim), new(2)
        self.clipped = [new(*t.shape) for t in (self.dw, self.dtab)]
        self.set = m.grad_set([self.dw, self.dtab], self.clipped)
        self.ws = [scratch(k) for k in (m.sort_ids_workspace_bytes(n, e), m.expert_workspace_bytes(e, rows, dim, n),
                                        m.embedding_grad_workspace_bytes(n, vocab, dim),
                                        m.grad_clip_workspace_bytes(self.set))]
        plain = m.expert_workspace_bytes(e, rows, dim, 4095)
        assert self.ws[1].numel() > plain + 4 * self.dw.numel()                  # the weight gradient is cut
        torch.cuda.synchronize()

    def run(self):
        m = self.m
        m.embedding_lookup(self.table, self.ids, self.h)
        m.sort_ids(self.expert, 2, self.order, self.starts, self.ws[0])
        m.embedding_lookup(self.h, self.order, self.hs)
        m.expert_matmul(self.hs, self.w, self.starts, self.y, self.ws[1])
        self.yb.copy_(self.y)
        m.expert_matmul(self.yb, self.w, self.starts, self.dx, self.ws[1], input_grad=True)
        m.expert_weight_grad(self.yb, self.hs, self.starts, self.dw, self.ws[1])
        self.dwb.fill_(1.0)
        m.expert_weight_grad(self.yb, self.hs, self.starts, self.dwb, self.ws[1], accumulate=True)
        m.embedding_grad(self.dx, self.ids, self.dtab, self.ws[2])
        m.embedding_grad(self.dx, self.ids, self.dtab, self.ws[2], accumulate=True)
        m.grad_clip(self.set, self.norm, self.ws[3], max_norm=1.0)

    def results(self):
        return [self.order, self.starts, self.hs, self.y, self.dx, self.dw, self.dwb, self.dtab, self.norm,
                *self.clipped]

    def keep(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.results()]


def same(chain, want):
    torch.cuda.synchronize()
    assert chain.m.op_device_status(chain.ws[1])[0] == chain.m.op_device_status(chain.ws[2])[0] == 0
    for k, (a, b) in enumerate(zip(chain.results(), want)):
        assert torch.equal(a, b), f"result {k}"
        assert torch.isfinite(a.float()).all()


@pytest.mark.parametrize("dim", [1104, 1101])
def test_chain_repeats_bit_for_bit(mfsdp, dim):
    """On one workspace, eagerly and replayed: no sum's order depends on timing."""
    c = Chain(mfsdp, dim)
    c.run()
    want = c.keep()
    for _ in range(5):
        c.run()
        same(c, want)
    d = Chain(mfsdp, dim)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run()
    for _ in range(5):
        graph.replay()
        same(d, want)


@pytest.mark.parametrize("dim", [1104, 1101])
def test_two_chains_on_two_streams_at_once(mfsdp, dim):
    chains = [Chain(mfsdp, dim, seed) for seed in (0, 1)]
    want = []
    for c in chains:
        c.run()
        want.append(c.keep())
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(10):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run()
    for c, w in zip(chains, want):
        same(c, w)


def test_two_host_threads(mfsdp):
    """Calls from two threads, each on its own stream and workspaces."""
    chains = [Chain(mfsdp, 1104, seed) for seed in (2, 3)]
    want, errors = [], []
    for c in chains:
        c.run()
        want.append(c.keep())

    def work(c):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    c.run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                # noqa: BLE001 (a thread's exceptions are lost)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, w in zip(chains, want):
        same(c, w)
