"""GPU cases of the operators next to the owner step that earlier tests leave out.
(Helpers and the derivation of the tolerances: test_gpu_ops.py.)
"""
import numpy as np
import pytest

from oracle.ops import grad_clip_ref
from tests.test_gpu_ops import scratch

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
