"""kvq_decode_attention_score with queries up to fp32's largest: a cap holds their scores, without one the largest wins."""
import numpy as np
import pytest

from score_util import Scored
from test_gpu_score_values import set_role

pytestmark = pytest.mark.gpu


def capped_check(blk, got, cap):
    """A score is off by 2^-17.6 A at most (score_util), far more than the cap here: a score of less than 2^-16 A, all but
    cancelled, has no sign in fp32 and its head is left out.  The others' sizes leave no doubt, or their rows are of ordinary
    size: bound of the cap's size."""
    import oracle
    checked = 0
    for b, length in enumerate(blk.lens):
        kh, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), blk.hkv, blk.page, blk.table[b], length)
        ref, mag, size = oracle.score.attention(blk.q[b:b + 1], kh, vh, blk.r, blk.hq // blk.hkv, cap)
        bound = 2.0 ** -16 * (1 + cap) * np.sqrt((mag[0] ** 2).mean(-1, keepdims=True))
        assert np.isfinite(got[b]).all()
        for j in range(blk.hq):
            h = j // (blk.hq // blk.hkv)
            a = kh[:, h] @ (blk.q[b, j].astype(np.float64) @ blk.r[h]) / np.sqrt(128.0)
            if size[0, j] * 2.0 ** -16 > 1 and np.abs(a).min() < 2.0 ** -16 * size[0, j]:
                continue
            checked += 1
            err = np.abs(got[b, j] - ref[0, j]).max()
            assert err <= bound[j, 0], (b, j, err, bound[j, 0])
    assert checked >= blk.hq


@pytest.mark.parametrize("scale", [1e17, 1e19, 1e30, 1e36, 3e37])
@pytest.mark.parametrize("hq,rot", [(4, "identity"), (8, "dense")])
@pytest.mark.parametrize("k_scale", [1.0, 5000.0])
def test_capped_scores_of_the_largest_queries(scale, hq, rot, k_scale):
    blk = Scored(51, hq, 1, 16, [130, 70, 1000], rot=rot, cap=5.0, q_scale=scale, k_scale=k_scale)
    capped_check(blk, blk.run(), 5.0)


@pytest.mark.parametrize("largest", [2.0 ** 126, float(np.finfo(np.float32).max)])
def test_capped_scores_of_fp32s_largest(largest):
    blk = Scored(52, 4, 2, 8, [300, 64], rot="identity", cap=30.0)
    blk.q[:] = np.where(blk.rng.random(blk.q.shape) < 0.5, -largest, largest).astype(np.float32)
    capped_check(blk, blk.run(), 30.0)


@pytest.mark.parametrize("scale", [1e17, 1e30, 1e36])
def test_heads_of_every_size_beside_one_another(scale):
    """One head of a group large, the others as they are without it, bit for bit."""
    blk = Scored(53, 8, 1, 16, [500, 77], rot="dense", cap=20.0)
    clean = blk.run()
    blk.q[:, 5] *= np.float32(scale)
    got = blk.run()
    capped_check(blk, got, 20.0)
    got[:, 5] = clean[:, 5]
    assert (got == clean).all()


@pytest.mark.parametrize("size", [1e15, 1e20, 1e36, float(np.finfo(np.float32).max)])
def test_without_a_cap_the_largest_score_wins(size):
    """One key ahead of all others: as a softmax of one token, however large its score (beyond fp32's largest too)."""
    for at in (0, 17, 299):
        blk = Scored(54, 4, 2, 16, [300], rot="identity")
        for h in range(2):
            k = np.full(300, -0.25)
            k[at] = 0.5
            set_role(blk, 0, 0, h, np.zeros(300), k)
        blk.q[:] = np.float32(size)
        got = blk.run()
        import oracle
        _, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), 2, 16, blk.table[0], 300)
        for j in range(4):
            v = vh[at, j // 2]
            # a weight of 1 as it is: three fp32 roundings of a value, and the two halves' 2^-22 of it
            assert (np.abs(got[0, j] - v) <= 2.0 ** -20 * np.abs(v).max()).all()


def test_nan_in_a_large_query_stays_in_its_head():
    blk = Scored(55, 8, 2, 16, [100, 50])
    blk.q[:, 3] *= np.float32(1e36)
    clean = blk.run()
    blk.q[0, 5] *= np.float32(1e36)
    blk.q[0, 5, 7] = np.nan
    got = blk.run()
    assert np.isnan(got[0, 5]).all()
    got[0, 5] = clean[0, 5]
    assert (got == clean).all()
