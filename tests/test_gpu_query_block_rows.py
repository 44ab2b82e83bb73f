"""Tree, chunk and cross attention: one query row does not change another, whatever its size.

Bounds as in test_gpu_query_block (they are a row's own)."""
import numpy as np
import pytest

import gpu_util as gu
from test_gpu_query_block import REL, Block, random_tree

pytestmark = pytest.mark.gpu


def check_rows(blk, got, bad, cross=False):
    """Every (query, head) outside `bad` is within its own bound."""
    import oracle
    for b, (n, length) in enumerate(zip(blk.ns, blk.lens)):
        c0 = blk.cu[b]
        kh, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), blk.hkv, blk.page, blk.table[b], length)
        see = None if cross else oracle.tree.visible(n, length, None if blk.parents is None else blk.parents[c0:c0 + n])
        q = blk.q[c0:c0 + n].astype(np.float64)
        keep = np.ones((n, blk.hq), bool)
        for i, j in bad:
            if c0 <= i < c0 + n:
                keep[i - c0, j] = False
        q[~keep] = 0.0
        ref, mag, size = oracle.tree.block_attention(q, kh, vh, blk.r, blk.hq // blk.hkv, see)
        bound = REL * (1 + size) * np.sqrt((mag ** 2).mean(-1))
        err = np.abs(got[c0:c0 + n] - ref).max(-1)
        assert np.all(err[keep] <= bound[keep]), (b, float((err / bound)[keep].max()))


@pytest.mark.parametrize("size", [1e9, 1e12, 1e20, 1e36])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,n", [(2, 5), (8, 3), (8, 30)])  # 10, 24 and 240 rows a KV head: each size of row tile
def test_a_huge_finite_row_leaves_the_others_alone(hq, n, dtype, size):
    blk = Block(51, hq, 1, 16, [700, 90], [n, n], "dense", dtype, random_tree)
    bad = [(1, 0), (n + 2, hq - 1)]
    for i, j in bad:
        blk.q[i, j] *= np.float32(size)
    if dtype == "bf16":
        from int2_kv_cache_gb300 import workloads as W
        blk.q = W.round_bf16(blk.q)
    check_rows(blk, blk.run(), bad)


@pytest.mark.parametrize("rot", ["identity", "signed_hadamard", "dense"])
def test_one_unscaled_head_of_a_group(rot):
    """A query head 10^10 times the others of its KV head, in a causal chunk of several row tiles and in cross attention."""
    for cross in (False, True):
        blk = Block(52, 8, 2, 8, [300, 77], [40, 20], rot, "f32")
        blk.q[:, 5] *= np.float32(1e10)
        check_rows(blk, blk.run(cross), [(i, 5) for i in range(60)], cross)


def test_tiny_rows_beside_normal_ones():
    """Rows from 10^-30 to 1 in one tile: each within its own bound, its mean over the values among them."""
    blk = Block(53, 4, 1, 16, [400], [16], "dense", "f32", random_tree)
    blk.q *= (10.0 ** np.linspace(-30, 0, 16)).astype(np.float32)[:, None, None]
    blk.check(blk.run())


@pytest.mark.parametrize("size", [2e34, 1e36, 2e37])
def test_a_tile_of_huge_rows_is_finite(size):
    """Rows whose logits are within fp32: a softmax of one token, however large (the scores' own rounding decides ties
    of such logits, so the key that wins is far ahead of the others)."""
    blk = Block(54, 2, 1, 16, [40], [4], "identity", "f32")
    blk.q[:] = np.float32(size)
    pos = 17
    for p in range(40):
        s, z = (0.0, 0.5) if p == pos else (0.0, -0.25)
        at = (p // 16, p % 16)
        rec = blk.pool[blk.table[0, at[0]], 0]
        rec[32 * at[1]:32 * at[1] + 32] = 0
        rec[64 * 16 + 4 * at[1]:64 * 16 + 4 * at[1] + 4] = np.array([s, z], np.float16).view(np.uint8)
    got = blk.run()
    import oracle
    _, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), 1, 16, blk.table[0], 40)
    want = np.broadcast_to(vh[pos, 0], got.shape)
    np.testing.assert_allclose(got, want, rtol=0, atol=2.0 ** -18 * np.abs(vh[pos]).max())


@pytest.mark.parametrize("hq,n", [(1, 9), (8, 8)])
def test_rows_of_very_different_size_over_many_units(hq, n):
    """Units with and without rows far apart follow one another in the same buffers."""
    rng = np.random.default_rng(3)
    ns = rng.integers(1, n + 1, 200).tolist()
    lens = [int(x + rng.integers(0, 400)) for x in ns]
    blk = Block(55, 2 * hq, 2, 16, lens, ns, "signed_hadamard", "f32", random_tree)
    bad = []
    for b in range(0, 200, 3):
        i, j = int(blk.cu[b]), int(rng.integers(0, 2 * hq))
        blk.q[i, j] *= np.float32(1e14)
        bad.append((i, j))
    check_rows(blk, blk.run(), bad)
