"""Pins of the float64 oracle of the steps around a projection."""
import numpy as np
import pytest

from oracle import step


def test_rmsnorm_by_hand():
    got = step.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(got, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)


def test_activation_by_hand():
    assert step.activation([0.0], "sigmoid")[0] == 0.5
    assert step.activation([0.0], "silu")[0] == 0.0
    assert step.activation([2.5], None)[0] == 2.5
    assert step.activation([-1000.0], "sigmoid")[0] == 0.0


def test_norm_residual_without_norm_and_gate_is_an_add():
    y, r = np.array([[1.0, -2.0]]), np.array([[0.5, 0.5]])
    r2, x, _ = step.norm_residual(y, r, None, None, None, None, 0.0, 2.0, post=False)
    assert np.array_equal(r2, [[2.5, -3.5]])
    assert np.allclose((x * x).mean(), 1.0)


def test_lora_equals_dense_update():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((3, 8)), rng.standard_normal((3, 5))
    A, B = rng.standard_normal((2, 4, 8)), rng.standard_normal((2, 5, 4))
    got, _ = step.lora(x, A, B, [1, -1, 0], [4, 2], [1.0, 0.5], y)
    assert np.allclose(got[0], y[0] + 0.5 * (B[1, :, :2] @ A[1, :2]) @ x[0])
    assert np.array_equal(got[1], y[1])
    assert np.allclose(got[2], y[2] + (B[0] @ A[0]) @ x[2])


def test_verify_by_hand():
    # V = 2: p = (0.75, 0.25) at temperature 1
    l = np.log(np.array([[3.0, 1.0], [3.0, 1.0]]))
    e = np.array([[1.0, 1.0]])
    q = np.array([[0.9, 0.1], [0.5, 0.5]])
    # 0.5 * 0.9 < 0.75: kept; then argmax p / e = 0
    acc, tok, _ = step.verify(l, [0, 2], [0, 0], q, [0.5, 0.0], e, [1.0])
    assert acc[0] == 1 and list(tok) == [0, 0]
    # 0.9 * 0.9 >= 0.75: refused; residual (0, 0.15) draws 1
    acc, tok, _ = step.verify(l, [0, 2], [0, 0], q, [0.9, 0.0], e, [1.0])
    assert acc[0] == 0 and list(tok) == [1, -1]
    # a certain drafter, refused: its own token is out
    acc, tok, _ = step.verify(l, [0, 2], [0, 0], None, [0.8, 0.0], e, [1.0])
    assert acc[0] == 0 and list(tok) == [1, -1]
    # greedy
    acc, tok, _ = step.verify(l, [0, 2], [0, 7], None, [0.0, 0.0], e, [0.0])
    assert acc[0] == 1 and list(tok) == [0, 0]
    # nothing allowed
    acc, tok, _ = step.verify(np.full((1, 3), -np.inf), [0, 1], [0], None, [0.0], np.ones((1, 3)),
                              [1.0])
    assert acc[0] == 0 and tok[0] == -1


@pytest.mark.parametrize("certain", [False, True])
def test_verify_draws_from_the_target(certain):
    # the first token of a sequence follows p whatever the drafter proposes
    rng = np.random.default_rng(3)
    n, V = 4000, 5
    l = np.repeat(rng.standard_normal((1, V)) * 1.5, 2 * n, axis=0)
    p = np.exp(l[0]) / np.exp(l[0]).sum()
    q0 = rng.dirichlet(np.ones(V))
    drafts = np.full(2 * n, 2) if certain else rng.choice(V, 2 * n, p=q0)
    acc, tok, _ = step.verify(l, np.arange(0, 2 * n + 1, 2), drafts,
                              None if certain else np.repeat(q0[None], 2 * n, axis=0),
                              rng.random(2 * n), rng.exponential(size=(n, V)), np.ones(n))
    got = np.bincount(tok[::2], minlength=V)
    chi2 = ((got - n * p) ** 2 / (n * p)).sum()
    assert chi2 < 33.4          # 4 degrees of freedom: probability 1e-6
