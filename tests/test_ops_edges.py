"""Edges of the operators next to the owner step that need no GPU: the oracle's
special values, and calls that the host turns away."""
import numpy as np

from oracle.ops import grad_clip_ref


def test_clip_oracle_at_an_infinite_limit():
    norm, coef, out = grad_clip_ref([[1.0, np.nan], [2.0]], np.inf, 1e-6)
    assert np.isnan(norm) and np.isnan(coef) and np.isnan(np.concatenate(out)).all()
    assert grad_clip_ref([[np.inf, 1.0]], np.inf, 1e-6)[:2] == (np.inf, 1.0)
    assert grad_clip_ref([[3.0, 4.0]], np.inf, 1e-6)[:2] == (5.0, 1.0)
