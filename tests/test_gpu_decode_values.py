"""kvq_decode_attention and its windowed form over records of any value scale, against the fp64 oracle.

Error bound, as in score_util for the other one-query kernel, with this one's fields at bits 0 .. 8 (keys) and 0 .. 9
(values) instead of 4 .. 8 and 7 .. 9: a product loses up to 4 and 7 bits more, so 2^-17.6 A becomes 2^-13.6 A and 2^-19 of
the largest weight 2^-12: held to 2^-11 (1 + A) of the row's root mean square of sum p |v|."""
import numpy as np
import pytest

import gpu_util as gu
from int2_kv_cache_gb300 import workloads as W
from score_util import Scored, row_attention
from test_gpu_score_values import ramp, value_scales
from test_gpu_window import _gpu_window, _mu, _oracle_windows

pytestmark = pytest.mark.gpu

REL = 2.0 ** -11


def check(blk, splits=0):
    import oracle
    d = blk.device()
    size = blk.kvq.kvq_decode_workspace_size(d["lay"], len(blk.lens), d["max_len"], splits)
    ws = blk.torch.full((size,), 0xA5, dtype=blk.torch.uint8, device="cuda")
    blk.kvq.kvq_decode_attention(d["lay"], d["q"], d["lens"], d["max_len"], d["table"], d["rot"], d["pool"], ws, d["o"],
                                 n_splits=splits)
    blk.kvq.kvq_device_check()
    got = d["o"].cpu().numpy()
    for b, n in enumerate(blk.lens):
        kh, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), blk.hkv, blk.page, blk.table[b], n)
        ref, mag, size = row_attention(blk.q[b], kh, vh, np.zeros(n), blk.r, blk.hq // blk.hkv, 0.0, None)
        bound = REL * (1 + size)[:, None] * np.sqrt((mag ** 2).mean(-1, keepdims=True))
        assert np.isfinite(got[b]).all() and (np.abs(got[b] - ref) <= bound).all(), (b, n)


@pytest.mark.parametrize("v_scale", [1e-6, 1.0, 3000.0])
@pytest.mark.parametrize("hq,hkv,page,splits", [(4, 2, 16, 0), (8, 1, 8, 3), (1, 1, 16, 0)])
def test_value_scales(v_scale, hq, hkv, page, splits):
    check(Scored(41, hq, hkv, page, [700, 33, 1], v_scale=v_scale, q_scale=2.0, rot="dense"), splits)


@pytest.mark.parametrize("hq", [4, 8])
def test_the_largest_value_scales(hq):
    blk = Scored(42, hq, 1, 16, [400, 70])
    value_scales(blk, lambda pos, rng: rng.uniform(20000, 43000, pos.size))
    check(blk)
    value_scales(blk, lambda pos, rng: np.full(pos.size, 65504.0), zero=lambda pos, rng: np.zeros(pos.size))
    check(blk)


@pytest.mark.parametrize("scale", [1100.0, 33000.0])
@pytest.mark.parametrize("last", [5.9, 40.0])
def test_scores_that_rise_behind_the_first(scale, last):
    blk = Scored(43, 4, 1, 16, [300], rot="identity")
    ramp(blk, lambda pos: last * pos / 300.0)
    value_scales(blk, lambda pos, rng: np.full(pos.size, scale))
    check(blk)


@pytest.mark.parametrize("hq,page,length", [(4, 16, 3000), (8, 8, 900), (2, 16, 20000)])
def test_scales_of_every_size_beside_one_another(hq, page, length):
    blk = Scored(44, hq, 1, page, [length, 130], q_scale=2.0)
    value_scales(blk, lambda pos, rng: 2.0 ** rng.uniform(-20, 15, pos.size))
    check(blk)
    for first, then in ((0.0, 3e-6), (3e-6, 20000.0), (20000.0, 3e-6), (0.0, 20000.0)):
        value_scales(blk, lambda pos, rng: np.where(pos < pos.size // 2, first, then) * rng.uniform(0.5, 2, pos.size))
        check(blk)


@pytest.mark.parametrize("factor", [1e-5, 3000.0])
@pytest.mark.parametrize("hq,hkv,page", [(4, 1, 16), (8, 1, 8), (4, 2, 16)])
def test_value_scales_beside_windows(hq, hkv, page, factor):
    """The tokens behind the windows with values `factor` times as large."""
    import oracle
    case = W.decode_case(45, [1000, 300, 65], hq, hkv, 128, "dense", "bf16", page_tokens=page, n_cal=256)
    g = gu.GpuCase(case)
    sink, recent = 64, 64
    regions = _oracle_windows(g, (sink, recent), _mu(case), [np.array([0, n]) for n in g.lengths])
    pool, _ = g.oracle_pool()
    meta = pool.reshape(-1, hkv, 72 * page)[:, :, 68 * page:]
    meta[:] = (np.ascontiguousarray(meta).view(np.float16).astype(np.float64) * factor).astype(np.float16).view(np.uint8)
    win = _gpu_window(g, (sink, recent))
    flat = np.concatenate([r.reshape(-1) for r in regions])
    win.buf[:flat.size] = g.torch.from_numpy(flat).cuda()
    q, max_len = case.queries(), int(g.lengths.max())
    ws = g.torch.empty(g.kvq.kvq_decode_workspace_size_win(g.layout, 3, max_len, win, 0), dtype=g.torch.uint8, device="cuda")
    out = g.torch.full((3, hq, 128), float("nan"), device="cuda")
    g.kvq.kvq_decode_attention_win(g.layout, gu.dev(q, "bf16"), gu.dev_i32(g.lengths), max_len, g.table, g.rot_k, g.rot_v,
                                   g.torch.from_numpy(pool).cuda(), win, ws, out)
    g.kvq.kvq_device_check()
    got = out.cpu().numpy()
    for b, n in enumerate(int(x) for x in g.lengths):
        kh, vh = oracle.cache.dequantized_sequence(pool, hkv, page, case.block_table[b], n)
        wp, wk, wv = oracle.window.read_window(regions[b], n, sink, recent)
        ref = oracle.window.decode_attention_windowed(q[b], kh, vh, wp, wk, wv, g.r_k, g.r_v, case.gqa, n, sink, recent)
        assert np.isfinite(got[b]).all() and gu.out_err(got[b], ref) <= gu.OUT_TOL, (b, n)
