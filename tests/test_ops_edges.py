"""Edges of the operators next to the owner step that need no GPU: the oracle's
special values, and calls that the host turns away."""
import numpy as np

from oracle.ops import grad_clip_ref


def test_clip_oracle_at_an_infinite_limit():
    norm, coef, out = grad_clip_ref([[1.0, np.nan], [2.0]], np.inf, 1e-6)
    assert np.isnan(norm) and np.isnan(coef) and np.isnan(np.concatenate(out)).all()
    assert grad_clip_ref([[np.inf, 1.0]], np.inf, 1e-6)[:2] == (np.inf, 1.0)
    assert grad_clip_ref([[3.0, 4.0]], np.inf, 1e-6)[:2] == (5.0, 1.0)


def test_scales_that_fp32_does_not_hold_are_refused(mfsdp):
    """The kernels multiply in fp32: a scale that is infinite there would make every
    zero a NaN."""
    lib = mfsdp.raw_lib()
    a, b, c, ws = 0x10000000, 0x20000000, 0x30000000, 0x50000000      # fake, aligned, far apart
    wsb = lib.mfsdp_embedding_grad_workspace_bytes(10, 100, 64)

    def lookup(scale, out=c):
        return lib.mfsdp_embedding_lookup(a, 0, 100, 64, 64, b, mfsdp.ID_I32, 10, scale, out, 0, 64, None)

    def grad(scale, g=c):
        return lib.mfsdp_embedding_grad(a, 0, 64, b, mfsdp.ID_I32, 10, scale, g, 0, 100, 64, 64, 0, ws, wsb, None)
    for scale in (1e300, -1e300, 3.5e38, float("inf"), float("nan")):
        assert lookup(scale) == grad(scale) == mfsdp.ERR_INVALID_ARG, scale
    for scale in (3.4e38, 0.0, -1e-60):                                # turned away later, for the output's alignment
        assert lookup(scale, c + 4) == grad(scale, c + 4) == mfsdp.ERR_MISALIGNED, scale
