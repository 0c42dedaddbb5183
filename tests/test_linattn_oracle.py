"""The oracle of linear attention and of the norms around a block against closed forms and other ways of computing them."""
import numpy as np
import pytest

from oracle import kda_oracle as O


def _inputs(T, H, H_k, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((H, dk, dv)), r.standard_normal((T, H_k, dk)), r.standard_normal((T, H_k, dk)), r.standard_normal((T, H, dv)),
            -r.exponential(0.3, (T, H)))


def test_one_token_by_hand():
    # S = e^-ln2 * 6 + 3 * 5 = 18, o = 0.5 * 2 * 18
    o, states = O.linattn_recurrent(np.array([[[6.0]]]), np.array([[[2.0]]]), np.array([[[3.0]]]), np.array([[[5.0]]]),
                                    np.array([[-np.log(2.0)]]), 0.5)
    assert states[1].item() == pytest.approx(18.0, rel=1e-15) and o.item() == pytest.approx(18.0, rel=1e-15)


@pytest.mark.parametrize("H,H_k", [(2, 2), (6, 2), (3, 1)])
def test_recurrence_is_the_masked_product_with_decays(H, H_k):
    S0, q, k, v, g = _inputs(9, H, H_k, 4, 3)
    o, states = O.linattn_recurrent(S0, q, k, v, g, 0.7)
    for h in range(H):
        hk = h * H_k // H
        b = np.cumsum(g[:, h])
        w = np.exp(np.tril(b[:, None] - b[None, :])) * np.tril(np.ones((9, 9)))
        ref = ((q[:, hk] @ k[:, hk].T) * w) @ v[:, h] + np.exp(b)[:, None] * (q[:, hk] @ S0[h])
        assert np.allclose(o[:, h], 0.7 * ref, rtol=1e-12, atol=1e-12)
        end = np.exp(b[-1]) * S0[h] + (k[:, hk] * np.exp(b[-1] - b)[:, None]).T @ v[:, h]
        assert np.allclose(states[-1][h], end, rtol=1e-12, atol=1e-12)


def test_closed_forms():
    S0, q, k, v, _ = _inputs(5, 2, 2, 4, 3)
    _, states = O.linattn_recurrent(S0, q, k, v, np.zeros(2))
    assert np.allclose(states[-1], S0 + np.einsum("thi,thj->hij", k, v))         # nothing decays: a sum
    _, states = O.linattn_recurrent(S0, q, k, v, np.full(2, -np.inf))
    assert np.allclose(states[-1], k[-1][:, :, None] * v[-1][:, None, :])        # everything decays: the last token
    _, states = O.linattn_recurrent(S0, q, 0 * k, v, np.array([-1.0, -2.0]))
    assert np.allclose(states[-1], np.exp([-5.0, -10.0])[:, None, None] * S0)    # no key: pure decay


def test_bounds_are_of_absolute_values():
    S0, q, k, v, g = _inputs(6, 2, 1, 3, 3)
    o, states = O.linattn_recurrent(S0, q, k, v, g, -1.0)
    ob, sb = O.linattn_recurrent(S0, q, k, v, g, -1.0, bound=True)
    assert np.all(ob >= np.abs(o)) and all(np.all(b >= np.abs(s)) for b, s in zip(sb, states))
    o1, _ = O.linattn_recurrent(*(np.abs(x) for x in (S0, q, k, v)), g, 1.0)
    assert np.allclose(o1, ob)


def test_norms():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(O.rms(x, 0.0), x / np.sqrt(12.5))
    assert np.allclose(O.rms(1e3 * x, 0.0), O.rms(x, 0.0)) and np.allclose(O.rms(0 * x, 1e-6), 0)
    z = np.array([[0.0, 0.0]])
    assert np.allclose(O.gate_of(z, "sigmoid"), 0.5) and np.allclose(O.gate_of(z, "silu"), 0) and np.allclose(O.gate_of(x, "none"), x)
    assert O.gate_of(np.array([2.0]), "silu")[0] == pytest.approx(2 / (1 + np.exp(-2)))
    y = O.gated_norm(x[None], np.array([2.0, 1.0]), z[None], eps=0.0)
    assert np.allclose(y, 0.5 * x / np.sqrt(12.5) * [2.0, 1.0])
    # a gate that is the same for the whole head drops out when it comes before the norm
    assert np.allclose(O.gated_norm(x[None], np.ones(2), z[None] + 1, eps=0.0, gate_first=True), O.rms(x, 0.0)[None])
    h, out = O.residual_norm(np.array([[1.0, 1.0]]), x, np.array([1.0, 3.0]), post_weight=np.ones(2), gate=z, channel_scale=np.array([2.0, 0.0]),
                             res_scale=10.0, eps=0.0)
    assert np.allclose(h, [[1 + 10 * 3 / np.sqrt(12.5), 1.0]]) and np.allclose(out, O.rms(h, 0.0) * [1.0, 3.0])
    assert np.allclose(O.residual_norm(x, x, np.ones(2))[0], 2 * x)
