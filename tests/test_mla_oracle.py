"""The oracle of the latent page cache against closed forms and another way of computing it."""
import numpy as np
import pytest

from oracle import kda_oracle as O


def test_rotation_preserves_length_and_composes():
    rng = np.random.default_rng(0)
    table = O.rope_table(50, 16)
    for inter in (False, True):
        x, y = rng.standard_normal(16), rng.standard_normal(16)
        rx = O.rope_rotate(x, table[7], inter)
        assert np.linalg.norm(rx) == pytest.approx(np.linalg.norm(x), rel=1e-14)
        # the product of two rotated vectors depends on the distance of their positions alone
        a = O.rope_rotate(x, table[7], inter) @ O.rope_rotate(y, table[3], inter)
        b = O.rope_rotate(x, table[44], inter) @ O.rope_rotate(y, table[40], inter)
        assert a == pytest.approx(b, rel=1e-12)
        assert np.allclose(O.rope_rotate(x, table[0], inter), x)


def test_rotation_of_a_unit_pair():
    table = O.rope_table(4, 2)
    assert np.allclose(O.rope_rotate(np.array([1.0, 0.0]), table[1]), [np.cos(1.0), np.sin(1.0)])
    # interleaved pairs are neighbours, half pairs are half a head apart
    table = O.rope_table(4, 4)
    x = np.array([1.0, 0.0, 0.0, 0.0])
    assert np.nonzero(O.rope_rotate(x, table[1], True))[0].tolist() == [0, 1]
    assert np.nonzero(O.rope_rotate(x, table[1], False))[0].tolist() == [0, 2]


def test_append_places_rows_and_normalises():
    rng = np.random.default_rng(1)
    pages = np.zeros((3, 16 * 132 + 5))
    c, k = rng.standard_normal((4, 128)), rng.standard_normal((4, 4))
    w = np.ones(128)
    out, q = O.mla_append(pages, 16, [17, -1, 0, 99999], [0, 0, 0, 0], O.rope_table(1, 4), c, k, norm_weight=w, eps=0.0)
    assert q is None and np.count_nonzero(out) == 2 * 132
    row = out[1, 132:264]
    assert np.mean(row[:128] ** 2) == pytest.approx(1.0) and np.allclose(row[128:], k[0])
    assert np.allclose(row[:128] * np.sqrt(np.mean(c[0] ** 2)), c[0])
    assert np.allclose(out[0, 128:132], k[2])


def test_decode_against_dense_attention():
    """The paged form equals one softmax over the gathered rows; equal keys give the mean value."""
    rng = np.random.default_rng(2)
    pages = rng.standard_normal((6, 16 * 20 + 3))
    table = np.array([[4, 1], [0, -1]])
    q, qp = rng.standard_normal((2, 2, 3, 16)), rng.standard_normal((2, 2, 3, 4))
    o, lse, _ = O.mla_decode(q, qp, pages, 16, table, [21, 1], 0.3, prefix_pages=[5], prefix_len=9)
    rows = pages[:, :320].reshape(6, 16, 20)
    keys = np.concatenate([rows[5, :9], rows[4], rows[1, :4]])          # query 0 of sequence 0 sees one token less
    x = 0.3 * (np.concatenate([q[0, 0], qp[0, 0]], -1) @ keys.T)
    w = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
    assert np.allclose(o[0, 0], w @ keys[:, :16]) and np.allclose(lse[0, 0], np.log(np.exp(x).sum(-1)))
    keys = rows[5, :9]                                                  # query 0 of sequence 1: the prefix alone
    x = 0.3 * (np.concatenate([q[1, 0], qp[1, 0]], -1) @ keys.T)
    assert np.allclose(lse[1, 0], np.log(np.exp(x).sum(-1)))
    o, lse, _ = O.mla_decode(0 * q, 0 * qp, pages, 16, table, [21, -1], 0.3)
    assert np.allclose(o[0, 1], np.concatenate([rows[4], rows[1, :5]])[:, :16].mean(0)) and np.allclose(lse[0, 1], np.log(21))
    assert np.all(o[1] == 0) and np.all(np.isneginf(lse[1]))
