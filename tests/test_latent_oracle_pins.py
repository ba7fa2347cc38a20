"""The fp64 latent-attention oracle against values worked out by hand (CPU)."""
import numpy as np
import pytest

from oracle import latent_oracle as lo


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_turn_of_each_pair(interleaved):
    f = np.zeros(32)
    f[0] = np.pi / 2                                   # a quarter turn a position for pair 0, none for the others
    x = np.arange(64.0) + 1
    y = lo.rotate(x, 1, f, interleaved)
    i, j = (0, 1) if interleaved else (0, 32)
    assert np.allclose([y[i], y[j]], [-x[j], x[i]])
    rest = [k for k in range(64) if k not in (i, j)]
    assert np.allclose(y[rest], x[rest])
    assert np.allclose(lo.rotate(x, 4, f, interleaved), x)      # four quarter turns
    f = np.random.default_rng(0).random(32)
    a, b = lo.rotate(x, 7, f, interleaved), lo.rotate(x[::-1].copy(), 3, f, interleaved)
    c, d = lo.rotate(x, 4, f, interleaved), lo.rotate(x[::-1].copy(), 0, f, interleaved)
    assert np.isclose(a @ b, c @ d)                    # scores depend on the distance alone


def test_attend_by_hand():
    # scores ln 1, ln 2, ln 5: weights 1/8, 2/8, 5/8, lse ln 8
    k = np.log([[1.0], [2.0], [5.0]])
    v = np.array([[8.0, 0.0], [0.0, 8.0], [8.0, 16.0]])
    out, lse = lo.attend(np.array([2.0]), k, v, 0.5)
    assert np.allclose(out, [1 + 5, 2 + 10]) and np.isclose(lse, np.log(8))
    out, lse = lo.attend(np.array([2.0]), k[:0], v[:0], 0.5)
    assert np.all(out == 0) and lse == -np.inf


def test_decode_and_prefill_masks():
    g = np.random.default_rng(1)
    rows = [g.standard_normal((n, 576)) for n in (5, 1, 0)]
    q = g.standard_normal((6, 2, 576))
    out, lse = lo.decode(q, rows, 0.1, tokens=2)
    assert np.allclose(out[0, 1], lo.attend(q[0, 1], rows[0][:4], rows[0][:4, :512], 0.1)[0])
    assert np.allclose(out[1, 0], lo.attend(q[1, 0], rows[0], rows[0][:, :512], 0.1)[0])
    assert lse[2, 0] == -np.inf and np.allclose(out[3, 0], rows[1][0, :512])    # one row: all the weight
    assert np.all(lse[4:] == -np.inf) and np.all(out[4:] == 0)
    k, v, r = g.standard_normal((7, 2, 128)), g.standard_normal((7, 2, 128)), g.standard_normal((7, 64))
    q = g.standard_normal((5, 2, 192))
    out, lse = lo.prefill(q, k, v, r, 0.1, [0, 2, 5], [0, 5, 7])                 # 2 queries of 5 keys, 3 of 2
    kk = np.concatenate([k[:4, 1], r[:4]], axis=1)
    assert np.allclose(out[0, 1], lo.attend(q[0, 1], kk, v[:4, 1], 0.1)[0])
    assert np.all(out[2] == 0) and np.all(lse[2] == -np.inf) and np.allclose(out[3], v[5])


def test_absorbed_and_expanded_forms_are_one():
    """Keys and values up-projected from the latent, or the query and the output instead: the same result."""
    g = np.random.default_rng(2)
    L, c = 9, g.standard_normal((9, 512))
    r, w_k, w_v = g.standard_normal((L, 64)), g.standard_normal((512, 128)), g.standard_normal((512, 128))
    q = g.standard_normal(192)
    expanded, l1 = lo.attend(q, np.concatenate([c @ w_k, r], 1), c @ w_v, 0.01)
    lat, l2 = lo.attend(np.concatenate([w_k @ q[:128], q[128:]]), np.concatenate([c, r], 1), c, 0.01)
    assert np.allclose(expanded, lat @ w_v) and np.isclose(l1, l2)
