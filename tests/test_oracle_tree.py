"""Pins oracle/tree.py: block attention under a draft tree's visibility, page plans, commits."""
import numpy as np
import pytest

from oracle import attention, cache, tree


def _rot(h, seed=0):
    g = np.random.default_rng(seed)
    return np.stack([np.linalg.qr(g.normal(size=(128, 128)))[0] for _ in range(h)])


def test_chain_is_causal_attention():
    g = np.random.default_rng(1)
    q, k, v = g.normal(size=(5, 4, 128)), g.normal(size=(12, 2, 128)), g.normal(size=(12, 2, 128))
    eye = np.stack([np.eye(128)] * 2)
    o, _, _ = tree.block_attention(q, k, v, eye, 2, tree.visible(5, 12))
    np.testing.assert_allclose(o, attention.causal_attention(q, k, v, 2), rtol=1e-12, atol=1e-13)


def test_tree_path_is_decoding_that_path():
    g = np.random.default_rng(2)
    parents = [-1, 0, 0, 1, 2, 3, -1, 4]
    n, base = len(parents), 9
    q, k, v = g.normal(size=(n, 2, 128)), g.normal(size=(base + n, 1, 128)), g.normal(size=(base + n, 1, 128))
    r = _rot(1)
    o, _, _ = tree.block_attention(q, k, v, r, 2, tree.visible(n, base + n, parents))
    for i in range(n):
        path, j = [], i
        while j >= 0:
            path.append(base + j)
            j = parents[j]
        rows = list(range(base)) + path[::-1]
        np.testing.assert_allclose(o[i], attention.decode_attention(q[i], k[rows], v[rows], r, 2), rtol=1e-12, atol=1e-13)


def test_rows_that_see_nothing_are_zero():
    o, _, _ = tree.block_attention(np.ones((2, 1, 128)), np.zeros((0, 1, 128)), np.zeros((0, 1, 128)), _rot(1), 1)
    assert np.all(o == 0)


def test_plans_conserve_pages_and_read_back():
    g = np.random.default_rng(3)
    page, nb, n, mb = 8, 60, 6, 12
    table, ring = np.zeros((n, mb), np.int64), g.permutation(nb)
    lens, head, tail = np.zeros(n, np.int64), 7 * nb + 11, 8 * nb + 11
    for step in range(30):
        new = np.clip(lens + g.integers(-30, 31, n), 0, 60)
        t2, r2, h2, l2, cu, slots = tree.plan_pages(page, nb, lens, new, table, ring, head, tail, 400)
        if h2 == head and l2 == tail and np.any(-(-new // page) != -(-lens // page)):
            continue  # refused: too few pages
        table, ring, head, tail = t2, r2, h2, l2
        for b in range(n):
            for t in range(cu[b], cu[b + 1]):
                pos = lens[b] + t - cu[b]
                assert slots[t] == table[b, pos // page] * page + pos % page
        assert np.all(slots[cu[-1]:] == -1)
        lens = new
        held = [x for b in range(n) for x in table[b, :-(-lens[b] // page)]]
        free = [ring[i % nb] for i in range(head, tail)]
        assert sorted(held + free) == list(range(nb))


def test_refused_plan_changes_nothing():
    table, ring = np.zeros((1, 4), np.int64), np.arange(4)
    for old, new, head, tail, most in (([0], [33], 0, 4, 99), ([0], [9], 0, 1, 99), ([0], [9], 0, 4, 8),
                                       ([-1], [3], 0, 4, 9), ([0], [3], 3, 2, 9), ([8], [0], 0, 4, 9)):
        t, r, h, l, cu, slots = tree.plan_pages(8, 4, old, new, table, ring, head, tail, most)
        assert (h, l) == (head, tail) and np.all(cu == 0) and np.all(slots == -1)
        assert np.array_equal(t, table) and np.array_equal(r, ring)


@pytest.mark.parametrize("page", [8, 16])
def test_commit_is_writing_the_accepted_tokens(page):
    g = np.random.default_rng(4)
    hkv, base, n = 2, 13, 9
    r = _rot(hkv)
    k, v = g.normal(size=(base + n, hkv, 128)), g.normal(size=(base + n, hkv, 128))
    table = g.permutation(6)
    path = [1, 2, 5, 8]
    enc = lambda rows: cache.encode_tokens(k[rows], v[rows], r, r, None, 1.0, 1.0)  # noqa: E731
    pool = np.zeros(cache.pool_bytes(6, hkv, page), np.uint8)
    cache.write_tokens(pool, hkv, page, table, 0, enc(list(range(base + n))))
    slots = [table[(base + i) // page] * page + (base + i) % page for i in range(n)]
    got, new = tree.commit(pool, hkv, page, [0, n], [path], [4], slots, [base + n])
    assert new.tolist() == [base + 4]
    want = np.zeros_like(pool)
    cache.write_tokens(want, hkv, page, table, 0, enc(list(range(base)) + [base + i for i in path]))
    a = cache.read_sequence(got, hkv, page, table, base + 4)
    b = cache.read_sequence(want, hkv, page, table, base + 4)
    for key in a:
        assert np.array_equal(a[key], b[key])
