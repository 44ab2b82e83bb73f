"""Tree, chunk and cross attention: records with scale 0, many units a CTA for every size of row tile, and more rows than
the dense rotation has blocks."""
import numpy as np
import pytest

from test_gpu_query_block import Block, random_tree, set_meta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k_scale,v_scale", [(1.0, 1.0), (1e-6, 1e-6)])
@pytest.mark.parametrize("hq,n", [(2, 6), (4, 12)])
def test_records_with_scale_zero(hq, n, k_scale, v_scale):
    """A quarter of the records with scale 0 and codes 0, as the append writes a constant group, zero points down to
    fp16's smallest, in keys and in values."""
    blk = Block(61, hq, 1, 16, [500], [n], "dense", "f32", random_tree, k_scale=k_scale, v_scale=v_scale)
    rng = np.random.default_rng(6)
    for role, size in ((0, k_scale), (1, v_scale)):
        for pos in np.flatnonzero(rng.random(500) < 0.25):
            block, slot = blk.table[0, pos // 16], pos % 16
            at = 32 * 16 * role + 32 * slot
            blk.pool[block, 0, at:at + 32] = 0
            set_meta(blk.pool, 16, role, block, slot, 0.0, [size, -size, 2.0 ** -24, -3 * 2.0 ** -24, 0.0][pos % 5])
    blk.check(blk.run())


def test_only_constant_values():
    blk = Block(62, 4, 2, 8, [200, 7], [5, 7], "signed_hadamard", "bf16", random_tree)
    blk.pool[:, :, 32 * 8:64 * 8] = 0
    for b, length in enumerate(blk.lens):
        for pos in range(length):
            for h in range(2):
                at = 68 * 8 + 4 * (pos % 8)
                blk.pool[blk.table[b, pos // 8], h, at:at + 4] = np.array([0, 2.0 ** -24 * (1 + pos % 3)], np.float16).view(np.uint8)
    blk.check(blk.run())


@pytest.mark.parametrize("hq,hkv,most", [(8, 8, 16), (32, 4, 12)])  # row tiles of 16 and of 64 (one or two a sequence)
@pytest.mark.parametrize("n", [128, 300])                           # both ways of listing the work
@pytest.mark.parametrize("kind", ["tree", "chain", "cross"])
def test_many_units_a_block(hq, hkv, most, n, kind):
    """Five to ten units a CTA, most of them of several tiles: rings, buffers and barriers come round again."""
    rng = np.random.default_rng([n, hq])
    ns = rng.integers(5 if most == 12 else 0, most + 1, n).tolist()
    ns[n // 2] = most
    lens = [int(x + rng.integers(0, 400)) for x in ns]
    if kind == "cross":
        lens = [int(x) for x in rng.integers(0, 400, n)]
    blk = Block(63, hq, hkv, 16, lens, ns, "signed_hadamard", "bf16", random_tree if kind == "tree" else None)
    cross = kind == "cross"
    blk.check(blk.run(cross), cross=cross, seqs=range(0, n, 9))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dense_rotation_of_more_rows_than_a_wave(dtype):
    """More tiles of rows than the rotation has blocks, so that a block takes several: 1,130 x 8 rows of a KV head."""
    blk = Block(64, 32, 4, 8, [40, 25], [1000, 130], "dense", dtype)
    blk.check(blk.run(cross=True), cross=True)
