"""Host-side checks of the page plan, tree / cross attention and tree commit entry points (no GPU)."""
import ctypes

import pytest

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def kvq():
    from int2_kv_cache_gb300 import _build
    _build.build()
    import int2_kv_cache_gb300 as m
    m.lib()
    return m


def _layout(kvq, **kw):
    d = dict(page_tokens=16, n_kv_heads=8, n_q_heads=32, num_blocks=100, max_blocks_per_seq=10)
    d.update(kw)
    return kvq.make_layout(**d)


def _tree(kvq, lay, name="kvq_tree_attention", **kw):
    a = dict(n_seqs=2, total=8, q=FAKE, dtype=1, cu=FAKE, max_q=4, parents=FAKE, lens=FAKE, max_len=160, table=FAKE,
             rot=kvq.KvqRot(0, None, None), pool=FAKE, ws=FAKE, ws_bytes=1 << 30, o=FAKE)
    a.update(kw)
    par = (a["parents"],) if name == "kvq_tree_attention" else ()
    return getattr(kvq.lib(), name)(ctypes.byref(lay), a["n_seqs"], a["total"], a["q"], a["dtype"], a["cu"], a["max_q"],
                                    *par, a["lens"], a["max_len"], a["table"], a["rot"], a["pool"], a["ws"],
                                    a["ws_bytes"], a["o"], None)


@pytest.mark.parametrize("name", ["kvq_tree_attention", "kvq_cross_attention"])
def test_query_block_rejects_bad_arguments(kvq, name):
    lay = _layout(kvq)
    err = lambda: kvq.lib().kvq_last_error().decode()  # noqa: E731
    for field in ("q", "cu", "lens", "table", "pool", "ws", "o"):
        assert _tree(kvq, lay, name, **{field: None}) == kvq.KVQ_EINVAL and "NULL" in err(), field
    for field in ("q", "pool", "ws", "o"):
        assert _tree(kvq, lay, name, **{field: FAKE + 4}) == kvq.KVQ_EINVAL and "aligned" in err(), field
    for field in ("cu", "lens", "table"):
        assert _tree(kvq, lay, name, **{field: FAKE + 2}) == kvq.KVQ_EINVAL and "aligned" in err(), field
    assert _tree(kvq, lay, name, max_len=161) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, max_len=-1) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, total=-1) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, max_q=-1) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, dtype=3) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, ws_bytes=16) == kvq.KVQ_EINVAL and "workspace" in err()
    assert _tree(kvq, lay, name, rot=kvq.KvqRot(2, None, None)) == kvq.KVQ_EINVAL
    assert _tree(kvq, lay, name, n_seqs=65536) == kvq.KVQ_EUNSUPPORTED
    assert _tree(kvq, lay, name, total=(1 << 31) - 1) == kvq.KVQ_EUNSUPPORTED
    assert _tree(kvq, _layout(kvq, n_q_heads=24), name) == kvq.KVQ_EUNSUPPORTED
    long = _layout(kvq, n_kv_heads=1, n_q_heads=1, max_blocks_per_seq=(1 << 27) - 1)
    assert _tree(kvq, long, name, n_seqs=1, max_len=(1 << 31) - 16) == kvq.KVQ_EUNSUPPORTED
    assert "2^31" in err()
    bad = _layout(kvq)
    bad.head_dim = 64
    assert _tree(kvq, bad, name) == kvq.KVQ_EUNSUPPORTED
    # nothing to do
    assert _tree(kvq, lay, name, n_seqs=0, q=None, cu=None) == kvq.KVQ_OK
    assert _tree(kvq, lay, name, total=0, q=None, o=None) == kvq.KVQ_OK
    assert _tree(kvq, lay, name, max_q=0, q=None, o=None) == kvq.KVQ_OK


def test_tree_size_limit(kvq):
    lay = _layout(kvq, num_blocks=1000, max_blocks_per_seq=500)
    assert _tree(kvq, lay, total=4000, max_q=1025, max_len=8000) == kvq.KVQ_EUNSUPPORTED
    assert "1024" in kvq.lib().kvq_last_error().decode()
    assert _tree(kvq, lay, total=4000, max_q=1025, max_len=8000, parents=FAKE + 2) == kvq.KVQ_EUNSUPPORTED
    assert _tree(kvq, lay, total=4000, max_q=1024, max_len=8000, parents=FAKE + 2) == kvq.KVQ_EINVAL


def test_workspace_sizes(kvq):
    lay = _layout(kvq)
    small = kvq.kvq_query_block_workspace_size(lay, 1, 1, 1, 16)
    assert small > 0 and kvq.kvq_query_block_workspace_size(lay, 4, 4096, 64, 160) >= 4096 * 32 * 512
    with pytest.raises(kvq.KvqError):
        kvq.kvq_query_block_workspace_size(lay, -1, 1, 1, 16)
    assert kvq.kvq_plan_workspace_size(65535) > kvq.kvq_plan_workspace_size(1) > 0
    for n in (0, 65536):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_plan_workspace_size(n)


def _plan(kvq, lay, **kw):
    a = dict(n=4, old=FAKE, new=FAKE, table=FAKE, ring=FAKE, rin=FAKE, rout=FAKE + 16, max_new=7, cu=FAKE, slots=FAKE,
             ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return kvq.lib().kvq_plan_pages(ctypes.byref(lay), a["n"], a["old"], a["new"], a["table"], a["ring"], a["rin"],
                                    a["rout"], a["max_new"], a["cu"], a["slots"], a["ws"], a["ws_bytes"], None)


def test_plan_rejects_bad_arguments(kvq):
    lay = _layout(kvq)
    for field in ("old", "new", "table", "ring", "rin", "rout", "cu", "slots", "ws"):
        assert _plan(kvq, lay, **{field: None}) == kvq.KVQ_EINVAL, field
    for field in ("rin", "rout", "slots", "ws"):
        assert _plan(kvq, lay, **{field: FAKE + 8}) == kvq.KVQ_EINVAL, field
    assert _plan(kvq, lay, rout=FAKE) == kvq.KVQ_EINVAL and b"alias" in kvq.lib().kvq_last_error()
    assert _plan(kvq, lay, max_new=-1) == kvq.KVQ_EINVAL
    assert _plan(kvq, lay, n=0) == kvq.KVQ_EINVAL
    assert _plan(kvq, lay, n=65536) == kvq.KVQ_EINVAL
    assert _plan(kvq, lay, ws_bytes=8) == kvq.KVQ_EINVAL
    assert _plan(kvq, _layout(kvq, page_tokens=32)) == kvq.KVQ_EUNSUPPORTED
    assert _plan(kvq, _layout(kvq, max_blocks_per_seq=1 << 28)) == kvq.KVQ_EUNSUPPORTED


def _commit(kvq, lay, **kw):
    a = dict(n=4, total=9, acc_n=3, cu=FAKE, acc=FAKE, n_acc=FAKE, slots=FAKE, lens=FAKE, new=FAKE + 64, pool=FAKE)
    a.update(kw)
    return kvq.lib().kvq_tree_commit(ctypes.byref(lay), a["n"], a["total"], a["acc_n"], a["cu"], a["acc"], a["n_acc"],
                                     a["slots"], a["lens"], a["new"], a["pool"], None)


def test_commit_rejects_bad_arguments(kvq):
    lay = _layout(kvq)
    for field in ("cu", "acc", "n_acc", "slots", "lens", "new", "pool"):
        assert _commit(kvq, lay, **{field: None}) == kvq.KVQ_EINVAL, field
    assert _commit(kvq, lay, new=FAKE) == kvq.KVQ_EINVAL
    assert _commit(kvq, lay, total=-1) == kvq.KVQ_EINVAL
    assert _commit(kvq, lay, acc_n=-1) == kvq.KVQ_EINVAL
    assert _commit(kvq, lay, n=65536) == kvq.KVQ_EUNSUPPORTED
    assert _commit(kvq, lay, n=0, cu=None) == kvq.KVQ_OK


def test_binding_rejects_types_shapes_and_host_tensors(kvq):
    torch = pytest.importorskip("torch")
    lay = _layout(kvq)
    i32, i64 = torch.int32, torch.int64
    z = lambda *s, dt=i32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        kvq.kvq_plan_pages(lay, z(2, dt=i64), z(2), z(2, 10), z(100), z(2, dt=i64), z(2, dt=i64), z(3), z(5, dt=i64), z(9))
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        kvq.kvq_plan_pages(lay, z(2), z(2), z(2, 10), z(100), z(2, dt=i64), z(2, dt=i64), z(3), z(5, dt=i64), z(9))
    with pytest.raises((TypeError, ValueError)):
        kvq.kvq_tree_attention(lay, torch.zeros(4, 32, 128), z(2), 4, None, z(1), 16, z(1, 10), kvq.DeviceRot("identity"),
                               z(9, dt=torch.uint8), z(9, dt=torch.uint8), torch.zeros(4, 32, 128))


def test_commit_rejects_new_lens_over_its_inputs(kvq):
    """The warps of a sequence read the path and its length on their own while one writes new_lens."""
    lay = _layout(kvq)
    far = dict(cu=FAKE, acc=FAKE + 0x1000, n_acc=FAKE + 0x2000, lens=FAKE + 0x3000, slots=FAKE + 0x4000, pool=FAKE + 0x8000)
    for name, size in (("cu", 5), ("acc", 12), ("n_acc", 4), ("lens", 4)):  # entries: 4 sequences, paths of up to 3
        for at in (far[name], far[name] + 4 * (size - 1), far[name] - 12):
            assert _commit(kvq, lay, **far, new=at) == kvq.KVQ_EINVAL, (name, at - far[name])
            assert b"overlap" in kvq.lib().kvq_last_error()


def test_plan_rejects_cu_new_over_the_lengths(kvq):
    """Every block reads the lengths on its own while cu_new is written."""
    lay = _layout(kvq)
    far = dict(old=FAKE, new=FAKE + 0x1000, table=FAKE + 0x2000, ring=FAKE + 0x3000, rin=FAKE + 0x4000, rout=FAKE + 0x5000,
               slots=FAKE + 0x6000, ws=FAKE + 0x8000)
    for name in ("old", "new"):
        for at in (far[name], far[name] + 12, far[name] - 16):  # 4 lengths, 5 entries of cu_new
            assert _plan(kvq, lay, **far, cu=at) == kvq.KVQ_EINVAL, (name, at - far[name])
            assert b"overlap" in kvq.lib().kvq_last_error()


@pytest.mark.parametrize("name", ["kvq_tree_attention", "kvq_cross_attention"])
def test_binding_rejects_rotations_of_other_types_and_shapes(kvq, name):
    """The kernels index a rotation by KV head, as fp32: one of fewer heads, or of another type, is read wrongly."""
    torch = pytest.importorskip("torch")
    lay = _layout(kvq)
    i32, u8 = torch.int32, torch.uint8
    z = lambda *s, dt=i32: torch.zeros(*s, dtype=dt)  # noqa: E731

    def call(rot):
        mid = (None,) if name == "kvq_tree_attention" else ()
        getattr(kvq, name)(lay, torch.zeros(4, 32, 128), z(2), 4, *mid, z(1), 16, z(1, 10), rot, z(8 * 16 * 72 * 100, dt=u8),
                           z(9, dt=u8), torch.zeros(4, 32, 128))

    f64, ones = torch.float64, torch.ones
    for rot in (kvq.DeviceRot("signed_hadamard", signs=ones(8, 128, dtype=f64)),
                kvq.DeviceRot("dense", dense=ones(8, 128, 128, dtype=torch.bfloat16))):
        with pytest.raises(TypeError, match="rot_k"):
            call(rot)
    for rot in (kvq.DeviceRot("signed_hadamard", signs=ones(1, 128)), kvq.DeviceRot("signed_hadamard", signs=ones(7, 128)),
                kvq.DeviceRot("dense", dense=ones(1, 128, 128)), kvq.DeviceRot("dense", dense=ones(8, 128))):
        with pytest.raises(ValueError, match="rot_k.* has shape"):
            call(rot)
    for rot in (kvq.DeviceRot("signed_hadamard"), kvq.DeviceRot("dense", signs=ones(8, 128))):
        with pytest.raises(ValueError, match="rot_k"):
            call(rot)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        call(kvq.DeviceRot("dense", dense=ones(8, 128, 128)))
    with pytest.raises(ValueError, match="contiguous|not on the current"):
        call(kvq.DeviceRot("dense", dense=ones(128, 128, 8).permute(2, 0, 1)))
