"""The operators around the owner-local optimizer step, as measured cases.

Five operators that a training program runs next to the owner step: the global
gradient norm with clipping over a rank's tensors, the embedding lookup with
scaling, its gradient by sorted tokens, the matrix products grouped by expert
(forward and input gradient), and the grouped weight gradient.  Each is given
in its plain form (elementary torch operations in fp32, rounded once at the
end) and as the calls of this package's binding (`own` true); `exact` is the
definition in 64 bits.

Sizes come from the package's own workloads: the tiny and GPT-2-block sets, an
8B-shaped rank, a 32000 x 2048 embedding, and a mixture-of-experts layer of 128
experts, 1408 x 2048 up and 2048 x 1408 down, of which 13 are unrouted.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6          # added to the norm before it divides the limit
_F = {"f32": torch.float32, "bf16": torch.bfloat16}
_B = {"f32": 4, "bf16": 2}


def _binding():
    from matrix_optimizers_under_gb300 import binding
    return binding


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest owner set (one 256 x 512 matrix and its tail), fp32: a latency-bound clip
        dict(name="clip_tiny", op="clip", sizes="131072,4096", dtypes="f32,f32", gap=0, std=1e-2, max_norm=1.0),
        # one GPT-2 block: four bf16 matrices and the packed fp32 tail
        dict(name="clip_gpt2_block", op="clip", sizes="1769472,589824,2359296,2359296,9984",
             dtypes="bf16,bf16,bf16,bf16,f32", gap=0, std=1e-3, max_norm=1.0),
        # an 8B-shaped rank's owned matrices (872 M bf16 elements, 28 matrices) and its norm vectors
        dict(name="clip_8b_rank", op="clip",
             sizes=",".join(["58720256"] * 12 + ["16777216"] * 8 + ["4194304"] * 8 + ["32768"]),
             dtypes=",".join(["bf16"] * 28 + ["f32"]), gap=0, std=1e-3, max_norm=1.0),
        # one new token of one sequence: a single row
        dict(name="lookup_one_token", op="lookup", n=1, vocab=32000, dim=2048, w="f32", out="bf16", ids="i64"),
        # a training batch of 16 sequences of 2048 tokens
        dict(name="lookup_batch", op="lookup", n=32768, vocab=32000, dim=2048, w="f32", out="bf16", ids="i64"),
        # a short odd sequence on a small vocabulary
        dict(name="embed_grad_short", op="embed_grad", n=257, vocab=2000, dim=768, dout="f32", grad="f32", ids="i64",
             accumulate=False),
        # the training batch's gradient, into the fp32 tail that AdamW reads
        dict(name="embed_grad_batch", op="embed_grad", n=32768, vocab=32000, dim=2048, dout="bf16", grad="f32",
             ids="i64", accumulate=False),
        # one token routed to 8 experts: bound by the 8 experts' weights and by latency
        dict(name="expert_one_token", op="expert", n=8, experts=128, active=8, rows=1408, cols=2048, y="bf16",
             input_grad=False),
        # a training batch through the up projection, 13 of 128 experts unrouted
        dict(name="expert_forward", op="expert", n=32768, experts=128, active=115, rows=1408, cols=2048, y="bf16",
             input_grad=False),
        # the input gradient through the down projection at half that batch, odd row count
        dict(name="expert_input_grad", op="expert", n=16383, experts=128, active=115, rows=2048, cols=1408, y="bf16",
             input_grad=True),
        # a small layer with odd sizes (no row of it starts on a 16-byte boundary), fp32 gradients
        dict(name="expert_weight_grad_odd", op="expert_wgrad", n=1501, experts=9, active=7, rows=331, cols=515,
             dw="f32", accumulate=False),
        # the training batch's weight gradients of all 128 up projections, into the bf16 gradient buffer
        dict(name="expert_weight_grad", op="expert_wgrad", n=32768, experts=128, active=115, rows=1408, cols=2048,
             dw="bf16", accumulate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    """A width: a multiple of 64 or of 8 as models have, or any number."""
    d = _log(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, d // step * step)


def draw(rng):
    op = rng.choice(["clip", "lookup", "embed_grad", "expert", "expert", "expert_wgrad"])
    if op == "clip":
        n = _log(rng, 1, 300)
        total = _log(rng, 1000, 200_000_000)
        sizes = [max(1, min(_log(rng, 1, 2 * total // n + 2), total)) for _ in range(n)]
        dtypes = [rng.choice(["bf16", "bf16", "f32"]) for _ in range(n)]
        return dict(op=op, sizes=",".join(map(str, sizes)), dtypes=",".join(dtypes), gap=rng.choice([0, 0, 1, 3]),
                    std=rng.choice([1e-4, 1e-3, 1e-2]), max_norm=rng.choice([0.01, 1.0, 1000.0]))
    if op == "lookup":
        vocab, dim = _log(rng, 500, 64000), _dim(rng, 64, 4096)
        return dict(op=op, n=_log(rng, 1, 65536), vocab=vocab, dim=dim, w=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["bf16", "f32"]), ids=rng.choice(["i64", "i32"]))
    if op == "embed_grad":
        vocab, dim = _log(rng, 500, 50000), _dim(rng, 64, 2048)
        return dict(op=op, n=_log(rng, 1, 65536), vocab=vocab, dim=dim, dout=rng.choice(["bf16", "f32"]),
                    grad=rng.choice(["f32", "bf16"]), ids=rng.choice(["i64", "i32"]),
                    accumulate=rng.choice([False, True]))
    experts = rng.choice([1, 4, 8, 16, 64, 128])
    rows, cols = _dim(rng, 64, 2048), _dim(rng, 64, 2048)
    n = _log(rng, 1, 32768)
    active = min(n, rng.randint(max(1, experts // 2), experts))
    if op == "expert":
        return dict(op=op, n=n, experts=experts, active=active, rows=rows, cols=cols, y=rng.choice(["bf16", "f32"]),
                    input_grad=rng.choice([False, True]))
    return dict(op=op, n=n, experts=experts, active=active, rows=rows, cols=cols, dw=rng.choice(["bf16", "f32"]),
                accumulate=rng.choice([False, True]))


# ----------------------------------------------------------------- the inputs
def _zipf(vocab):
    """Frequencies of a vocabulary as text has them: rank ** -1 over shuffled ids."""
    p = 1.0 / np.arange(1, vocab + 1, dtype=np.float64)
    return p / p.sum()


def _ids(case, seed):
    rng = np.random.default_rng([seed, 1])
    p = _zipf(case["vocab"])
    perm = rng.permutation(case["vocab"])
    ids = perm[np.minimum(np.searchsorted(np.cumsum(p), rng.random(case["n"])), case["vocab"] - 1)]
    return torch.from_numpy(ids.astype(np.int64 if case["ids"] == "i64" else np.int32)).cuda()


def _counts(case, seed):
    """Rows of each expert: `active` experts share the rows unevenly (every one
    of them has one at least), the others have none."""
    rng = np.random.default_rng([seed, 2])
    live = np.sort(rng.permutation(case["experts"])[:case["active"]])
    share = rng.gamma(2.0, size=case["active"])
    extra = rng.multinomial(case["n"] - case["active"], share / share.sum())
    counts = np.zeros(case["experts"], np.int64)
    counts[live] = 1 + extra
    return counts


def _randn(shape, dtype, std, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "clip":
        sizes = [int(s) for s in case["sizes"].split(",")]
        dtypes = [_F[d] for d in case["dtypes"].split(",")]
        # the tensors lie in one flat buffer a dtype, `gap` elements apart, and
        # so do the clipped ones (the buffers are the outputs; gaps stay zero)
        flat, at = {}, {}
        for d in sorted(set(dtypes), key=str):
            total = sum(s + case["gap"] for s, t in zip(sizes, dtypes) if t == d)
            flat[d] = _randn((total,), d, case["std"], gen)
            at[d] = 0
        out = {d: torch.zeros_like(f) for d, f in flat.items()}
        st["out"] = list(out.values())
        st["src"], st["dst"] = [], []
        for s, d in zip(sizes, dtypes):
            st["src"].append(flat[d][at[d]:at[d] + s])
            st["dst"].append(out[d][at[d]:at[d] + s])
            at[d] += s + case["gap"]
        if own:
            m = _binding()
            st["set"] = m.grad_set(st["src"], st["dst"])
            st["norm"] = torch.zeros(2, device="cuda")
            st["ws"] = torch.empty(m.grad_clip_workspace_bytes(st["set"]), dtype=torch.uint8, device="cuda")
        return st
    if op == "lookup":
        st["w"] = _randn((case["vocab"], case["dim"]), _F[case["w"]], 0.02, gen)
        st["ids"] = _ids(case, seed)
        if own:
            st["out"] = torch.empty((case["n"], case["dim"]), dtype=_F[case["out"]], device="cuda")
        return st
    if op == "embed_grad":
        st["dout"] = _randn((case["n"], case["dim"]), _F[case["dout"]], 1e-3, gen)
        st["ids"] = _ids(case, seed)
        if case["accumulate"]:
            st["grad0"] = _randn((case["vocab"], case["dim"]), _F[case["grad"]], 1e-3, gen)
        if own:
            m = _binding()
            st["grad"] = torch.empty((case["vocab"], case["dim"]), dtype=_F[case["grad"]], device="cuda")
            st["ws"] = torch.empty(m.embedding_grad_workspace_bytes(case["n"], case["vocab"], case["dim"]),
                                   dtype=torch.uint8, device="cuda")
        return st
    counts = _counts(case, seed)
    st["counts"] = counts.tolist()
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    st["starts"] = torch.from_numpy(starts).cuda()
    e, n, rows, cols = case["experts"], case["n"], case["rows"], case["cols"]
    if op == "expert":
        st["w"] = _randn((e, rows, cols), torch.bfloat16, cols ** -0.5, gen)
        st["x"] = _randn((n, rows if case["input_grad"] else cols), torch.bfloat16, 1.0, gen)
        if own:
            st["y"] = torch.empty((n, cols if case["input_grad"] else rows), dtype=_F[case["y"]], device="cuda")
    else:
        st["dy"] = _randn((n, rows), torch.bfloat16, 1e-3, gen)
        st["x"] = _randn((n, cols), torch.bfloat16, 1.0, gen)
        if case["accumulate"]:
            st["dw0"] = _randn((e, rows, cols), _F[case["dw"]], 1e-3, gen)
        if own:
            st["dw"] = torch.empty((e, rows, cols), dtype=_F[case["dw"]], device="cuda")
    if own:
        st["ws"] = torch.empty(_binding().expert_workspace_bytes(e, rows, cols, n), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------- one pass
def _scale(case):
    return math.sqrt(case["dim"])       # the lookup's scale: rows of unit size from weights of size dim ** -0.5


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    m, case = _binding(), st["case"]
    op = case["op"]
    if op == "clip":
        m.grad_clip(st["set"], st["norm"], st["ws"], max_norm=case["max_norm"], eps=EPS)
        return [st["norm"][0]] + st["out"]
    if op == "lookup":
        m.embedding_lookup(st["w"], st["ids"], st["out"], scale=_scale(case))
        return st["out"]
    if op == "embed_grad":
        if case["accumulate"]:
            st["grad"].copy_(st["grad0"])
        m.embedding_grad(st["dout"], st["ids"], st["grad"], st["ws"], scale=_scale(case),
                         accumulate=case["accumulate"])
        return st["grad"]
    if op == "expert":
        m.expert_matmul(st["x"], st["w"], st["starts"], st["y"], st["ws"], input_grad=case["input_grad"])
        return st["y"]
    if case["accumulate"]:
        st["dw"].copy_(st["dw0"])
    m.expert_weight_grad(st["dy"], st["x"], st["starts"], st["dw"], st["ws"], accumulate=case["accumulate"])
    return st["dw"]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), device="cuda")
        for g in st["src"]:
            g = g.float()
            total = total + (g * g).sum()
        norm = torch.sqrt(total)
        coef = torch.clamp(case["max_norm"] / (norm + EPS), max=1.0)
        for g, d in zip(st["src"], st["dst"]):
            d.copy_(g.float() * coef)
        return [norm] + st["out"]
    if op == "lookup":
        return (st["w"][st["ids"]].float() * _scale(case)).to(_F[case["out"]])
    if op == "embed_grad":
        grad = torch.zeros((case["vocab"], case["dim"]), device="cuda")
        grad.index_add_(0, st["ids"], st["dout"].float() * _scale(case))
        if case["accumulate"]:
            grad += st["grad0"].float()
        return grad.to(_F[case["grad"]])
    n, rows, cols = case["n"], case["rows"], case["cols"]
    if op == "expert":
        y = torch.zeros((n, cols if case["input_grad"] else rows), dtype=_F[case["y"]], device="cuda")
        at = 0
        for e, c in enumerate(st["counts"]):
            if c:
                w = st["w"][e].float()
                y[at:at + c] = (st["x"][at:at + c].float() @ (w if case["input_grad"] else w.t())).to(y.dtype)
            at += c
        return y
    dw = torch.zeros((case["experts"], rows, cols), dtype=_F[case["dw"]], device="cuda")
    at = 0
    for e, c in enumerate(st["counts"]):
        prod = st["dy"][at:at + c].float().t() @ st["x"][at:at + c].float()
        dw[e] = (prod + st["dw0"][e].float() if case["accumulate"] else prod).to(dw.dtype)
        at += c
    return dw


# ------------------------------------------------------------------- the work
def _distinct(case):
    """Expected number of different ids among the n drawn."""
    return float(np.sum(-np.expm1(case["n"] * np.log1p(-np.minimum(_zipf(case["vocab"]), 1 - 1e-12)))))


def work(case):
    op = case["op"]
    if op == "clip":
        sizes = [int(s) for s in case["sizes"].split(",")]
        nb = [_B[d] for d in case["dtypes"].split(",")]
        return {"bytes": sum(2 * s * b for s, b in zip(sizes, nb)) + 4, "flops": 3 * sum(sizes)}
    if op in ("lookup", "embed_grad"):
        idb = 8 if case["ids"] == "i64" else 4
        n, dim = case["n"], case["dim"]
        if op == "lookup":
            return {"bytes": int(_distinct(case) * dim * _B[case["w"]]) + n * idb + n * dim * _B[case["out"]],
                    "flops": n * dim}
        out = case["vocab"] * dim * _B[case["grad"]] * (2 if case["accumulate"] else 1)
        return {"bytes": n * dim * _B[case["dout"]] + n * idb + out, "flops": 2 * n * dim}
    n, e, rows, cols = case["n"], case["experts"], case["rows"], case["cols"]
    flops = 2 * n * rows * cols
    if op == "expert":
        a, b = (rows, cols) if case["input_grad"] else (cols, rows)
        return {"bytes": n * a * 2 + case["active"] * rows * cols * 2 + n * b * _B[case["y"]] + 4 * (e + 1),
                "flops": flops}
    out = e * rows * cols * _B[case["dw"]] * (2 if case["accumulate"] else 1)
    return {"bytes": n * (rows + cols) * 2 + out + 4 * (e + 1), "flops": flops}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    global own
    keep, own = own, False          # the inputs alone, without this package's calls
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op = case["op"]
    if op == "clip":
        parts = [torch.linalg.vector_norm(c.double()) for g in st["src"] for c in g.split(1 << 24)]
        norm = torch.linalg.vector_norm(torch.stack(parts))
        limit = case["max_norm"] / (norm.item() + EPS)
        flat = {o.dtype: torch.zeros_like(o, dtype=torch.float64) for o in st["out"]}
        at = {d: 0 for d in flat}
        for g in st["src"]:
            flat[g.dtype][at[g.dtype]:at[g.dtype] + g.numel()] = g.double() * min(1.0, limit)
            at[g.dtype] += g.numel() + case["gap"]
        return [norm] + list(flat.values())
    if op == "lookup":
        return torch.index_select(st["w"], 0, st["ids"].long()).double().mul_(_scale(case))
    if op == "embed_grad":
        order = torch.argsort(st["ids"].long(), stable=True)
        ids, seg = torch.unique_consecutive(st["ids"].long()[order], return_counts=True)
        out = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        ends = torch.cumsum(seg, 0).tolist()
        run_ = torch.cumsum(st["dout"].double()[order], 0)
        last = run_[torch.tensor(ends, device="cuda") - 1]
        last[1:] -= last[:-1].clone()
        out[ids] = last * _scale(case)
        return out + st["grad0"].double() if case["accumulate"] else out
    n = case["n"]
    expert = torch.repeat_interleave(torch.arange(case["experts"]), torch.tensor(st["counts"]))
    if op == "expert":
        width = case["cols"] if case["input_grad"] else case["rows"]
        out = torch.zeros((n, width), dtype=torch.float64, device="cuda")
        for e in torch.unique(expert).tolist():
            idx = torch.nonzero(expert == e).flatten().cuda()
            x, w = st["x"][idx].double(), st["w"][e].double()
            out[idx] = torch.einsum("tr,rc->tc", x, w) if case["input_grad"] else torch.einsum("tc,rc->tr", x, w)
        return out
    out = torch.zeros((case["experts"], case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(expert).tolist():
        idx = torch.nonzero(expert == e).flatten().cuda()
        out[e] = torch.einsum("tr,tc->rc", st["dy"][idx].double(), st["x"][idx].double())
    return out + st["dw0"].double() if case["accumulate"] else out
