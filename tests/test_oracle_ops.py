"""Pins of the oracle of the operators next to the owner step: closed forms,
and every gradient against differences of its forward product (CPU)."""
import numpy as np
import pytest

from oracle.ops import (embedding_grad_ref, embedding_lookup_ref, expert_matmul_ref, expert_weight_grad_ref,
                        grad_clip_ref, sort_ids_ref)


def test_clip_closed_forms():
    norm, coef, out = grad_clip_ref([[3.0], [4.0]], 1.0, 0.0)
    assert norm == 5.0 and coef == 0.2 and np.allclose(np.concatenate(out), [0.6, 0.8])
    assert grad_clip_ref([[3.0, 4.0]], 10.0, 0.0)[1] == 1.0
    assert grad_clip_ref([[0.0]], 0.0, 0.0)[:2] == (0.0, 1.0)
    assert grad_clip_ref([], 1.0, 1e-6)[:2] == (0.0, 1.0)
    assert grad_clip_ref([[1.0]], np.inf, 1e-6)[1] == 1.0
    assert np.isnan(grad_clip_ref([[np.nan]], 1.0, 0.0)[1]) and grad_clip_ref([[np.inf]], 1.0, 0.0)[1] == 0.0
    a = np.random.default_rng(0).standard_normal(100)
    got = np.concatenate(grad_clip_ref([a[:7], a[7:]], 2.0, 0.0)[2])
    assert np.isclose(np.linalg.norm(got), 2.0)


def test_sort_ids_small():
    order, starts = sort_ids_ref([2, 0, 5, 2, -1, 0], 3)
    assert order.tolist() == [1, 5, 0, 3, 2, 4] and starts.tolist() == [0, 2, 2, 4]
    ids = np.random.default_rng(1).integers(-2, 5003, 4000)
    order, starts = sort_ids_ref(ids, 5000)
    for k in (0, 17, 4999):
        assert order[starts[k]:starts[k + 1]].tolist() == np.flatnonzero(ids == k).tolist()


def _diff(f, a, at, h):
    p, m = a.copy(), a.copy()
    p[at] += h
    m[at] -= h
    return (f(p) - f(m)) / (2 * h)


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(2)
    w, ids = rng.standard_normal((7, 5)), [3, 0, 3, 9, -1, 3, 6]
    c = rng.standard_normal((7, 5))
    g = embedding_grad_ref(c, ids, 7, 1.5)
    for at in np.ndindex(w.shape):
        assert np.isclose(_diff(lambda x: np.sum(c * embedding_lookup_ref(x, ids, 1.5)), w, at, 0.5), g[at])
    assert np.all(g[[1, 2, 4, 5]] == 0.0)
    assert np.allclose(embedding_grad_ref(c, ids, 7, 1.5, w), w + g)


@pytest.mark.parametrize("starts", [[0, 3, 3, 8], [0, 0, 6, 6]])
def test_expert_gradients_against_differences(starts):
    rng = np.random.default_rng(3)
    x, w, c = rng.standard_normal((8, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((8, 5))
    dx, dw = expert_matmul_ref(c, w, starts, True), expert_weight_grad_ref(c, x, starts)
    for at in np.ndindex(x.shape):
        assert np.isclose(_diff(lambda a: np.sum(c * expert_matmul_ref(a, w, starts)), x, at, 0.5), dx[at])
    for at in np.ndindex(w.shape):
        assert np.isclose(_diff(lambda a: np.sum(c * expert_matmul_ref(x, a, starts)), w, at, 0.5), dw[at])
    assert np.all(expert_matmul_ref(x, w, starts)[starts[-1]:] == 0.0)
