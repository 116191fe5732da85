"""Pins of the filtered-distribution oracle: hand-worked rows, brute force over
the prefixes of the order, and the output law of the filtered verify."""
import numpy as np
import pytest
from scipy import stats
from scipy.special import softmax

from oracle import filtered as F


def test_hand_worked_rows():
    z = np.log(np.array([0.4, 0.1, 0.3, 0.2]))
    assert F.filter_row(z, 1.0, 2).probs == pytest.approx([4 / 7, 0, 3 / 7, 0])
    # before: 0, .4, .7, .9
    assert F.filter_row(z, 1.0, 0, 0.69).probs == pytest.approx([4 / 7, 0, 3 / 7, 0])
    assert F.filter_row(z, 1.0, 0, 0.71).n_kept == 3
    # top-p over the top-k's mass: shares 4/7, 3/7
    assert F.filter_row(z, 1.0, 2, 0.5).n_kept == 1
    assert F.filter_row(z, 1.0, 2, 0.58).n_kept == 2
    assert F.filter_row(z, 1.0, 0, 1.0, 0.49).probs == pytest.approx([4 / 9, 0, 3 / 9, 2 / 9])
    assert F.filter_row(z, 1.0, 0, 1.0, 1.0).n_kept == 1
    r = F.filter_row(z, 0.5)
    assert r.probs == pytest.approx(softmax(z / 0.5), rel=1e-13)
    assert (r.min_kept, r.last, r.n_kept) == (-np.inf, 3, 4)


def test_ties_go_to_the_lowest_index():
    z = np.array([1.0, 2.0, 2.0, -0.0, 0.0, 2.0])
    r = F.filter_row(z, 1.0, 2)
    assert np.nonzero(r.probs)[0].tolist() == [1, 2] and r.last == 2 and r.min_kept == 2.0
    r = F.filter_row(z, 1.0, 5)
    assert np.nonzero(r.probs)[0].tolist() == [0, 1, 2, 3, 5] and r.last == 3
    assert F.filter_row(z, 0.0).last == 1


def test_masked_rows():
    inf = np.inf
    r = F.filter_row([-inf, 3.0, np.nan, -inf], 1.0, 3)
    assert r.probs.tolist() == [0, 1, 0, 0] and r.n_kept == 1
    r = F.filter_row([-inf, np.nan], 1.0, 3)
    assert r.n_kept == 0 and r.last == -1 and not r.probs.any() and r.min_kept == inf
    r = F.filter_row([inf, 0.0, inf], 1.0, 3, 0.9)
    assert r.probs.tolist() == [0.5, 0, 0.5]


@pytest.mark.parametrize("seed", range(20))
def test_every_filter_is_the_shortest_or_longest_prefix(seed):
    rng = np.random.default_rng(seed)
    V = int(rng.integers(2, 12))
    z = np.round(rng.normal(size=V) * 2, 1)
    T = float(np.float32(rng.uniform(0.3, 2)))
    k, p, mp = int(rng.integers(1, V + 1)), float(np.float32(rng.uniform(0.05, 0.99))), \
        float(np.float32(rng.uniform(0.01, 0.9)))
    order = sorted(range(V), key=lambda i: (-z[i], i))
    pr = softmax(z / T)
    n = k
    share = [pr[order[i]] / sum(pr[j] for j in order[:k]) for i in range(k)]
    n = min(n, next(i for i in range(1, k + 1) if sum(share[:i]) >= p or i == k))
    while pr[order[n - 1]] < mp * pr.max():
        n -= 1
    r = F.filter_row(z, T, k, p, mp)
    assert sorted(np.nonzero(r.probs)[0]) == sorted(order[:n])
    assert r.n_kept == n and r.last == order[n - 1] and r.min_kept == z[order[n - 1]]
    assert r.probs.sum() == pytest.approx(1.0)
    assert r.inv_sum == pytest.approx(1 / np.exp((z[order[:n]] - z.max()) / T).sum())


def test_draw_is_the_inverse_cdf():
    w = np.array([0.0, 0.5, 0.0, 0.25, 0.25])
    assert [F.draw(w, u)[0] for u in (0.0, 0.49, 0.5, 0.74, 0.75, 0.999)] == [1, 1, 3, 3, 4, 4]
    assert F.draw(w * 3, 0.6)[1] == pytest.approx(0.1)
    assert F.draw(np.zeros(3), 0.5)[0] == 0


def test_verify_emits_the_filtered_target():
    """Whatever q the drafts come from, the first emitted token follows the
    filtered target."""
    rng = np.random.default_rng(5)
    V, N = 8, 40000
    zt = rng.normal(size=(2, V)) * 1.5
    rows = [F.filter_row(z, 0.8, 5, 0.9, 0.05) for z in zt]
    q = F.filter_row(rng.normal(size=V) * 1.5, 1.0, 6).probs
    seen = np.zeros(V)
    for _ in range(N):
        u = rng.random(3)
        d = F.draw(q, u[2])[0]
        a, c, _, _ = F.verify_seq(rows, q[None], [d], u[[0, 1]], 0.8)
        seen[d if a else c] += 1
    want = rows[0].probs
    assert not seen[want == 0].any()
    keep = want > 0
    assert stats.chisquare(seen[keep], N * want[keep]).pvalue > 1e-4


def test_verify_greedy_and_bad_drafts():
    rows = [F.filter_row(z, 0.0) for z in ([0.0, 2.0, 1.0], [5.0, 0.0, 5.0], [0.0, 0.0, 1.0])]
    q = np.full((2, 3), 1 / 3)
    assert F.verify_seq(rows, q, [1, 0], [0.9, 0.9, 0.9], 0.0)[:2] == (2, 2)
    assert F.verify_seq(rows, q, [1, 2], [0.0, 0.0, 0.9], 0.0)[:2] == (1, 0)
    assert F.verify_seq(rows, q, [-1, 2], [0.0, 0.0, 0.9], 0.0)[:2] == (0, 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 10))
    f = np.array([1.0, 0.3, 0.01])
    pos = [0, 7, 123456789]
    y = F.rotate(x, pos, f, interleaved, 1.25)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    i0 = [0, 2, 4] if interleaved else [0, 1, 2]
    i1 = [1, 3, 5] if interleaved else [3, 4, 5]
    z = (x[..., i0] + 1j * x[..., i1]) * 1.25 * np.exp(1j * np.outer(pos, f))[:, None]
    assert np.allclose(y[..., i0], z.real) and np.allclose(y[..., i1], z.imag)
