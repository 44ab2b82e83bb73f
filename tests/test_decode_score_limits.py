"""Lengths near 2^31 at the entry points of the decode (no GPU)."""
import ctypes

import pytest

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
LONGEST = 2 ** 31 - 257


@pytest.fixture(scope="module")
def kvq():
    from int2_kv_cache_gb300 import _build
    _build.build()
    import int2_kv_cache_gb300 as m
    m.lib()
    return m


def _layout(kvq, page=16, hkv=1, hq=4):
    return kvq.make_layout(page, hkv, hq, 16, (2 ** 31 - page) // page)


def _decode(kvq, lay, max_len, n=1):
    # a workspace of no bytes: every size that is not refused is reported as too small
    return kvq.lib().kvq_decode_attention_score(ctypes.byref(lay), n, FAKE, 1, FAKE, max_len, FAKE, kvq.KvqRot(0, None, None),
                                                FAKE, ctypes.byref(kvq.KvqScore(0.0, None, 0, None)), FAKE, 0, FAKE, None)


def _err(kvq):
    return kvq.lib().kvq_last_error().decode()


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("more", [1, 192, 225, 240])
def test_decode_score_refuses_lengths_past_its_index_range(kvq, page, more):
    assert _decode(kvq, _layout(kvq, page), LONGEST + more) == kvq.KVQ_EUNSUPPORTED and "max_seq_len" in _err(kvq)
    assert _decode(kvq, _layout(kvq, page), LONGEST) == kvq.KVQ_EINVAL and "workspace" in _err(kvq)


def test_chunk_counts_do_not_wrap(kvq):
    """From 2^31 - 31 tokens on the count of a sequence's chunks was negative, and any number of them accepted."""
    size = ctypes.c_size_t()
    for max_len in (2 ** 31 - 1000, 2 ** 31 - 31, 2 ** 31 - 1):
        lay = _layout(kvq)
        call = lambda n: kvq.lib().kvq_decode_workspace_size(ctypes.byref(lay), n, max_len, 0, ctypes.byref(size))  # noqa: E731
        assert call(15) == kvq.KVQ_OK
        assert call(17) == kvq.KVQ_EUNSUPPORTED, max_len  # 17 * 67,108,833 chunks and more: 2^30 is the limit
    sizes = []
    for max_len in (2 ** 31 - 1000, 2 ** 31 - 1):
        lay = _layout(kvq)
        assert kvq.lib().kvq_decode_workspace_size(ctypes.byref(lay), 1, max_len, 0, ctypes.byref(size)) == kvq.KVQ_OK
        sizes.append(size.value)
    assert sizes[0] == sizes[1]
