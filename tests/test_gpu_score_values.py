"""Attention with kvq_score over records of any value scale, one query a sequence and chunks, against the fp64 oracle.

Bounds as in score_util: they are in units of sum p |v|, whatever the size of v.  What the one-query kernel adds at odd
scales is far inside: a weight times its scale is held to 2^-36 where the largest is 2^-8 or more."""
import numpy as np
import pytest

from score_util import CHUNK_REL, Scored, row_attention

pytestmark = pytest.mark.gpu


def scored(form, seed, hq, hkv, page, lens, **kw):
    return Scored(seed, hq, hkv, page, lens, None if form == "decode" else [min(3, n) for n in lens], **kw)


def places(blk, b):
    """Page and slot of every cached token of sequence b."""
    pos = np.arange(blk.lens[b])
    return pos, blk.table[b, pos // blk.page], pos % blk.page


def set_role(blk, role, b, h, scale, zero):
    """Scale and zero of every token of a sequence and head; codes of scale 0 are 0."""
    pos, block, slot = places(blk, b)
    meta = np.stack([scale, zero], -1).astype(np.float16).view(np.uint8)
    blk.pool[block[:, None], h, (64 + 4 * role) * blk.page + 4 * slot[:, None] + np.arange(4)] = meta
    none = np.flatnonzero(meta.view(np.float16)[:, 0] == 0)
    blk.pool[block[none, None], h, 32 * blk.page * role + 32 * slot[none, None] + np.arange(32)] = 0


def value_scales(blk, scale, zero=None):
    """The value scales of every head: scale(positions, rng), zeros at -1.5 of them or zero(positions, rng)."""
    for b in range(len(blk.lens)):
        for h in range(blk.hkv):
            pos = np.arange(blk.lens[b])
            s = np.asarray(scale(pos, blk.rng), np.float64)
            set_role(blk, 1, b, h, s, -1.5 * s if zero is None else zero(pos, blk.rng))


def ramp(blk, rise):
    """Keys and queries whose base-2 scores are rise(position): constant keys, queries of ones."""
    blk.q[:] = 1.0
    for b in range(len(blk.lens)):
        pos = np.arange(blk.lens[b])
        for h in range(blk.hkv):
            set_role(blk, 0, b, h, 0.0 * pos, rise(pos) * np.log(2.0) / np.sqrt(128.0))


def check(blk, got):
    """As blk.check, but a chunk counts a value record of scale 0 as one of scale 2^-24 (include/kvq.h): its centred codes and
    its zero each carry 1.5 2^-24, so that sum p |v| is that much more, p being 1 at most."""
    if blk.decode:
        blk.check(got)
        return
    import oracle
    for b, (n, length) in enumerate(zip(blk.ns, blk.lens)):
        kh, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), blk.hkv, blk.page, blk.table[b], length)
        for i in range(n):
            end = length - n + i + 1
            row = int(blk.cu[b]) + i
            ref, mag, size = row_attention(blk.q[row], kh[:end], vh[:end], np.zeros(end), blk.r, blk.hq // blk.hkv, 0.0, None)
            mag = mag + 1.5 * 2.0 ** -24
            bound = CHUNK_REL * (1 + size)[:, None] * np.sqrt((mag ** 2).mean(-1, keepdims=True))
            assert (np.abs(got[row] - ref) <= bound).all(), float((np.abs(got[row] - ref) / bound).max())


@pytest.mark.parametrize("form", ["decode", "chunk"])
@pytest.mark.parametrize("v_scale", [1e-6, 1e-4, 50.0, 3000.0])
@pytest.mark.parametrize("hq,hkv,page", [(4, 2, 16), (8, 1, 8), (1, 1, 16)])
def test_value_scales(form, v_scale, hq, hkv, page):
    blk = scored(form, 31, hq, hkv, page, [700, 33, 1], v_scale=v_scale, q_scale=2.0, rot="dense", window=600, cap=20.0)
    blk.check(blk.run())


@pytest.mark.parametrize("form", ["decode", "chunk"])
@pytest.mark.parametrize("hq", [4, 8])
def test_the_largest_value_scales(form, hq):
    """Up to fp16's largest: scale and zero of 20,000 to 43,000."""
    blk = scored(form, 32, hq, 1, 16, [400, 70])
    value_scales(blk, lambda pos, rng: rng.uniform(20000, 43000, pos.size))
    blk.check(blk.run())
    value_scales(blk, lambda pos, rng: np.full(pos.size, 65504.0), zero=lambda pos, rng: np.zeros(pos.size))
    blk.check(blk.run())


@pytest.mark.parametrize("form", ["decode", "chunk"])
@pytest.mark.parametrize("scale", [1100.0, 2000.0, 33000.0])
@pytest.mark.parametrize("last", [0.9, 5.9, 40.0])
def test_scores_that_rise_behind_the_first(form, scale, last):
    """Later tokens a little above the first maximum, where its reference stays, and far above it."""
    blk = scored(form, 33, 4, 1, 16, [300], rot="identity")
    ramp(blk, lambda pos: last * pos / 300.0)
    value_scales(blk, lambda pos, rng: np.full(pos.size, scale))
    blk.check(blk.run())


@pytest.mark.parametrize("form", ["decode", "chunk"])
@pytest.mark.parametrize("hq,page,length", [(4, 16, 3000), (8, 8, 900), (2, 16, 20000)])
def test_scales_of_every_size_beside_one_another(form, hq, page, length):
    """From 2^-20 to 2^15 in random order; each half of the context with a size of its own, scale 0 among them."""
    blk = scored(form, 34, hq, 1, page, [length, 130], q_scale=2.0)
    value_scales(blk, lambda pos, rng: 2.0 ** rng.uniform(-20, 15, pos.size))
    blk.check(blk.run())
    for first, then in ((0.0, 3e-6), (3e-6, 20000.0), (20000.0, 3e-6), (0.0, 20000.0)):
        value_scales(blk, lambda pos, rng: np.where(pos < pos.size // 2, first, then) * rng.uniform(0.5, 2, pos.size))
        check(blk, blk.run())


@pytest.mark.parametrize("form", ["decode", "chunk"])
@pytest.mark.parametrize("down", [3.0, 12.0, 30.0, 60.0])
def test_large_scales_where_nothing_looks(form, down):
    """Tokens 2^down below the others in weight with scales up to 2^35 above theirs, in every order."""
    for order in (0, 1):
        blk = scored(form, 35, 4, 1, 16, [500], rot="identity")
        ramp(blk, lambda pos: np.where((pos // 50) % 2 == order, -down, 0.01 * (pos % 7)))
        value_scales(blk, lambda pos, rng: np.where((pos // 50) % 2 == order, 30000.0, 1e-6 * rng.uniform(1, 2, pos.size)))
        blk.check(blk.run())


@pytest.mark.parametrize("form", ["decode", "chunk"])
def test_values_of_zero_are_zero(form):
    blk = scored(form, 36, 8, 2, 16, [300, 40])
    value_scales(blk, lambda pos, rng: np.zeros(pos.size))
    check(blk, blk.run())  # a decode's bound is 0
