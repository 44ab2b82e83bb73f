"""Cross attention over a long context behind a token with most of the weight."""
import numpy as np
import pytest

import gpu_util as gu
from test_gpu_query_block import REL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gqa,n", [(1, 2), (8, 3), (8, 8)])  # 2, 24 and 64 rows a KV head: each size of row tile
def test_the_tail_behind_a_token_with_most_of_the_weight(gqa, n):
    """One token 16 to 22 nats above 131,071 equal ones, whose values are all at the same end of their range: the
    readout in closed form; the 131,071 weigh between 1.5 % and 4e-5 together.

    Bound: that of test_gpu_query_block (A = the token's logit, all products of one sign), and the running sums, whose
    roundings are of one sign when the tokens are equal.  A sequence is one CTA's: 1,024 tiles are added one after the
    other in fp32, an addition off by 2^-24 of the sum at most, so each sum by 2^-14 of itself: sum p (to which the
    output, |o| <= 1 + 3 * 0.015, is relative), sum p mid (mid 0.5 for the first token, 1.5 for the others) and
    sum p (c - 1.5) (1.5 for all).  2^-14 (1.05 + 0.53 + 1.5) < 2^-14 * 3.1."""
    kvq, torch = gu.kvq_lib(), gu.torch_cuda()
    page, hkv, tokens, seqs = 16, 8, 1 << 17, 19  # 152 units: each is one CTA's
    hq, blocks = hkv * gqa, tokens // page
    pool = np.zeros((blocks, hkv, 72 * page), np.uint8)
    value = np.where(np.arange(128) % 4 == 0, 0, 3)          # codes of every token but the first
    byte = value.reshape(32, 4) @ np.array([1, 4, 16, 64])
    pool[:, :, 32 * page:64 * page] = np.tile(byte.astype(np.uint8), page)
    key, val = np.zeros((page, 2), np.float16), np.zeros((page, 2), np.float16)
    val[:, 0] = 1.0
    pool[:, :, 64 * page:68 * page] = key.reshape(-1).view(np.uint8)
    pool[:, :, 68 * page:] = val.reshape(-1).view(np.uint8)
    pool[0, :, 32 * page:32 * page + 32] = 0                 # the first: key 1 in every channel, value -1
    pool[0, :, 64 * page:64 * page + 4] = np.array([0, 1], np.float16).view(np.uint8)
    pool[0, :, 68 * page:68 * page + 4] = np.array([1, -1], np.float16).view(np.uint8)
    logits = np.linspace(16, 22, n * hq).reshape(n, hq)
    q = np.tile((logits / np.sqrt(128))[None, :, :, None], (seqs, 1, 1, 128)).astype(np.float32).reshape(seqs * n, hq, 128)
    logits = q[:n, :, 0].astype(np.float64) * np.sqrt(128)
    lay = kvq.make_layout(page, hkv, hq, blocks, blocks)
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    ws = torch.empty(kvq.kvq_query_block_workspace_size(lay, seqs, seqs * n, n, tokens), dtype=torch.uint8, device="cuda")
    o = torch.empty(seqs * n, hq, 128, device="cuda")
    kvq.kvq_cross_attention(lay, d(q), d(np.arange(seqs + 1, dtype=np.int32) * n), n,
                            d(np.full(seqs, tokens, np.int32)), tokens,
                            d(np.tile(np.arange(blocks, dtype=np.int32), (seqs, 1))), kvq.DeviceRot("identity"), d(pool), ws, o)
    kvq.kvq_device_check()
    tail = (tokens - 1) * np.exp(-logits)[..., None]
    want = (-1.0 + tail * value) / (1.0 + tail)
    mag = (1.0 + tail * value) / (1.0 + tail)
    bound = REL * (1 + logits) * np.sqrt((mag ** 2).mean(-1)) + 3.1 * 2.0 ** -14
    err = np.abs(o.cpu().numpy().reshape(seqs, n, hq, 128) - want).max(-1)
    assert np.all(err <= bound), float((err / bound).max())
