"""Pins of the eviction oracle (CPU): identities and brute force."""
import numpy as np
import pytest

import workload as W
from oracle import eviction as E
from oracle import mla as O


def draws(seed=0, lens=(5, 9, 2), nq=2, H=3, d_c=16, d_rope=8, page=4):
    g = np.random.default_rng(seed)
    table, pages = W.make_page_table(np.array(lens), page, seed, True, spare_pages=1)
    pool = g.standard_normal((pages, page, d_c + d_rope))
    q = g.standard_normal((len(lens), nq, H, d_c + d_rope))
    return pool, table, np.array(lens), q, d_c, d_rope


def lse_of(pool, table, lens, q, scale):
    B, nq, H, _ = q.shape
    out = np.empty((B, nq, H))
    for b in range(B):
        rows = O.gather_cache(pool, table[b], int(lens[b]))
        for i in range(nq):
            s = scale * rows[: lens[b] - nq + i + 1] @ q[b, i].T
            out[b, i] = np.log(np.exp(s).sum(axis=0))
    return out


def test_mass_of_a_step_sums_to_its_rows():
    # every query row's weights sum to one: the mass of a sequence is nq * H
    pool, table, lens, q, _, _ = draws()
    lse = lse_of(pool, table, lens, q, 0.3)
    m = E.attention_mass(q, pool, table, lens, lse, 0.3, np.zeros((3, 12)))
    assert np.allclose(m.sum(axis=1), q.shape[1] * q.shape[2], atol=1e-12)
    for b, n in enumerate(lens):
        assert (m[b, n:] == 0).all()


def test_mass_zero_queries_are_uniform():
    pool, table, lens, q, _, _ = draws(nq=1, lens=(5, 8, 1))
    lse = lse_of(pool, table, lens, 0 * q, 0.3)
    m = E.attention_mass(0 * q, pool, table, lens, lse, 0.3, np.full((3, 8), 2.0), decay=0.5)
    for b, n in enumerate(lens):
        # earlier tokens fade and gain H / n; the new token starts from nothing
        assert np.allclose(m[b, : n - 1], 1.0 + 3 / n) and np.isclose(m[b, n - 1], 3 / n)
        assert (m[b, n:] == 2.0).all()


def test_mass_weights_are_those_of_the_attention():
    # sum_n w_n c_n over one query and head is the attention's latent output
    pool, table, lens, q, d_c, _ = draws(nq=1)
    for b, n in enumerate(lens):
        rows = O.gather_cache(pool, table[b], int(n))
        o, l = O.attend_latent(q[b, 0, :1], rows[:, :d_c], rows[:, d_c:], 0.3)
        m = E.attention_mass(q[b : b + 1, :, :1], pool, table[b : b + 1], lens[b : b + 1], np.reshape(l, (1, 1, 1)), 0.3,
                             np.zeros((1, 12)))
        assert np.allclose(m[0, :n] @ rows[:, :d_c], np.reshape(o, (-1,)), atol=1e-12)


def test_mass_of_a_row_that_saw_nothing():
    pool, table, lens, q, _, _ = draws()
    lse = np.full(q.shape[:3], -np.inf)
    assert (E.attention_mass(q, pool, table, lens, lse, 0.3, np.zeros((3, 12))) == 0).all()


def test_mass_lens_says_what_the_old_mass_is():
    pool, table, lens, q, _, _ = draws(nq=1)
    lse = np.full(q.shape[:3], np.inf)          # no weight at all: only the old mass is left
    old = np.ones((3, 12))
    m = E.attention_mass(q, pool, table, lens, lse, 0.3, old, mass_lens=[0, 4, 9])
    assert (m[0, :5] == 0).all() and (m[1, :9] == [1] * 4 + [0] * 5).all() and (m[2, :2] == 1).all()


@pytest.mark.parametrize("budget,sink,recent,want", [
    (4, 0, 0, [1, 2, 4, 6]),        # 9, 5, 5 (index 2), then the first of the threes
    (4, 2, 1, [0, 1, 4, 7]),
    (3, 2, 9, [0, 1, 7]),           # the recent ones get what the sinks leave
    (1, 2, 2, [0]),
    (0, 2, 2, []),
    (8, 1, 1, list(range(8))),
    (99, 0, 0, list(range(8))),
])
def test_select_by_hand(budget, sink, recent, want):
    mass = np.array([[0.0, 5.0, 5.0, 3.0, 9.0, 0.0, 3.0 + 1e-9, 3.0]])
    assert E.select(mass, [8], [budget], sink, recent)[0].tolist() == want


def test_select_nan_and_ties():
    mass = np.array([[1.0, np.nan, np.inf, 1.0, -np.inf, -0.0, 0.0]])
    pick = lambda k: E.select(mass, [7], [k], 0, 0)[0].tolist()
    assert pick(1) == [1] and pick(2) == [1, 2] and pick(3) == [0, 1, 2] and pick(4) == [0, 1, 2, 3]
    assert pick(5) == [0, 1, 2, 3, 5] and pick(6) == [0, 1, 2, 3, 5, 6]


def test_compact_keeps_relative_positions():
    # the score of a query at a position p with a key at n depends on p - n: after a
    # move by n - j of both the query and the key it is the same
    pool, table, lens, q, d_c, _ = draws(nq=1)
    kept = [np.array([0, 2, 4]), np.array([3, 7, 8]), np.array([1])]
    after, _ = E.compact(pool, table, kept, d_c)
    for b, idx in enumerate(kept):
        rows, moved = O.gather_cache(pool, table[b], int(lens[b])), O.gather_cache(after, table[b], len(idx))
        for j, n in enumerate(idx):
            assert np.allclose(moved[j, :d_c], rows[n, :d_c], atol=0)
            k = rows[n, d_c:]
            assert np.isclose(O.rope(q[b, 0, 0, d_c:], 30) @ k, O.rope(q[b, 0, 0, d_c:], 30 + j - n) @ moved[j, d_c:])


def test_compact_bits_and_the_rest():
    pool, table, lens, q, d_c, _ = draws()
    kept = [np.array([0, 1, 4]), np.array([], dtype=int), np.array([0, 1])]
    mass = np.arange(36.0).reshape(3, 12)
    after, m = E.compact(pool, table, kept, d_c, mass=mass, rerotate=False)
    moved = np.zeros(pool.shape[:2], dtype=bool)
    moved[table[0][0], 2] = True                # only row 2 of sequence 0 changes
    assert (after[~moved] == pool[~moved]).all()
    assert (after[table[0][0], 2] == pool[table[0][1], 0]).all()
    assert m[0, :3].tolist() == [0, 1, 4] and (m[0, 3:] == mass[0, 3:]).all() and (m[1:] == mass[1:]).all()
