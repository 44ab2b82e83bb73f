"""Bad pages at the attention with kvq_score are flagged; a decode does not see their tokens, a chunk leaves the other
sequences as they are."""
import numpy as np
import pytest

from score_util import Scored

pytestmark = pytest.mark.gpu


def without(blk, b, page):
    """What sequence b is without the tokens of a page: shorter, for calls that do not go by positions."""
    n = -(-blk.lens[b] // blk.page)
    keep = [i for i in range(n) if i != page]
    row = blk.table[b].copy()
    row[:len(keep)] = blk.table[b, keep]
    return row, blk.lens[b] - min(blk.page, blk.lens[b] - page * blk.page)


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("bad", [0, 3, 4, 5, 17, "last"])
@pytest.mark.parametrize("value", [-1, "past"])
@pytest.mark.parametrize("hq,cap", [(4, 0.0), (8, 20.0)])
def test_a_decode_does_not_see_a_bad_page(page, bad, value, hq, cap):
    blk = Scored(71, hq, 1, page, [900, 50, 200], cap=cap, rot="dense")
    # what earlier calls left where the page would be
    before = Scored(72, hq, 1, page, [4000] * 16, v_scale=3000.0, k_scale=50.0)
    before.launch(before.device())
    at = -(-900 // page) - 1 if bad == "last" else bad
    d = blk.device()
    d["table"][0, at] = -1 if value == -1 else blk.blocks
    blk.launch(d)
    with pytest.raises(blk.kvq.KvqError):
        blk.kvq.kvq_device_check()
    got = d["o"].cpu().numpy()
    blk.check(got, seqs=[1, 2])
    blk.table[0], blk.lens[0] = without(blk, 0, at)
    blk.check(got, seqs=[0])


@pytest.mark.parametrize("page", [8, 16])
def test_a_sequence_of_bad_pages_alone_is_zero(page):
    blk = Scored(73, 4, 2, page, [40, 300])
    d = blk.device()
    d["table"][0] = -7
    blk.launch(d)
    with pytest.raises(blk.kvq.KvqError):
        blk.kvq.kvq_device_check()
    got = d["o"].cpu().numpy()
    assert np.all(got[0] == 0)
    blk.check(got, seqs=[1])


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("bad", [0, 7, 17])
def test_a_chunk_with_a_bad_page_leaves_the_others_alone(page, bad):
    """Its own sequence's rows are unspecified."""
    blk = Scored(74, 8, 2, page, [400, 130, 260], [40, 130, 3], cap=20.0, window=300, rot="dense")
    clean = blk.run()
    d = blk.device()
    d["table"][0, -(-100 // page) + bad] = blk.blocks + 3  # seen by every query: the windows start before 100
    blk.launch(d)
    with pytest.raises(blk.kvq.KvqError):
        blk.kvq.kvq_device_check()
    got = d["o"].cpu().numpy()
    assert np.array_equal(got[40:], clean[40:])
    blk.check(got, seqs=[1, 2])
