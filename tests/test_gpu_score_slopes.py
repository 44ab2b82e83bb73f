"""Attention with kvq_score under slopes of any finite size: from 10^5 on the nearest token (the farthest, below 0) is alone."""
import numpy as np
import pytest

import gpu_util as gu
from score_util import Scored

pytestmark = pytest.mark.gpu

BIG = float(np.finfo(np.float32).max)


class Sloped(Scored):
    def score(self):
        return self.kvq.Score(cap=self.cap, slopes=gu.dev(self.slopes), window=self.window,
                              prefix_lens=None if self.prefix is None else gu.dev_i32(self.prefix))


@pytest.mark.parametrize("form", ["decode", "chunk", "long chunk"])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("window,prefix", [(0, 0), (50, 0), (50, 20), (0, 690)])
@pytest.mark.parametrize("sizes", [(1e5, -1e5, 1e20, -1e20), (1e37, -1e37, BIG, -BIG)])
def test_slopes_of_any_size(form, cap, window, prefix, sizes):
    import oracle
    lens = [700, 130]
    ns = {"decode": None, "chunk": [5, 2], "long chunk": [100, 130]}[form]
    blk = Sloped(61, 4, 1, 16, lens, ns, cap=cap, window=window, prefix=[prefix, min(prefix, 100)] if prefix else None)
    blk.slopes = np.array(sizes, np.float32)
    got = blk.run()
    for b, length in enumerate(lens):
        _, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), 1, 16, blk.table[b], length)
        n, pre = blk.ns[b], 0 if blk.prefix is None else int(blk.prefix[b])
        for i in range(n):
            t, s = length - n + i, np.arange(length)
            seen = s[((s <= t) & ((s > t - window) if window else True)) | (s < pre)]
            far = np.abs(t - seen)
            for j, slope in enumerate(sizes):
                best = seen[far == (far.min() if slope > 0 else far.max())]
                if best.size > 1:
                    continue  # as far before the query as behind it: the scores decide
                v = vh[best[0], 0]
                # one weight of 1: the value's own roundings and the 2^-22 of the weight's two halves
                assert (np.abs(got[blk.cu[b] + i, j] - v) <= 2.0 ** -19 * np.abs(v).max()).all(), (b, i, j)
