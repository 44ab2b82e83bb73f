"""GPU parity of tree / chunk / cross attention over the INT2 cache against the fp64 oracle.

The pools are drawn directly (random codes, fp16 scales and zeros): attention is defined on any pool.

Error bound.  With A = ||q'|| max ||k_hat|| / sqrt(128) over a row's visible positions, a logit is a sum of 128
products whose magnitudes sum to at most A (Cauchy-Schwarz).  The rotation and the product are sums of 128 terms
with relative roundings u = 2^-24; roundings of independent sign add like sqrt(128) u = 2^-20.5, so a logit is off
by at most about 2 * 2^-20.5 A = 2^-19.5 A, a weight by that plus its own few u (exponential, split into two
halves of 11 bits: 2^-22), and the readout by twice the weight's relative error times sum p |v_hat| (numerator
and denominator).  Held to: |error| <= 2^-18 (1 + A) sum_s p_s |v_hat_s|, per channel, where sum p |v| is
replaced by the row's root mean square over channels (a channel can have all its values near zero)."""
import numpy as np
import pytest

import gpu_util as gu
from int2_kv_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18


def make_pool(rng, blocks, hkv, page, k_scale=1.0, v_scale=1.0):
    """Random codes; fp16 scale > 0 and zero such that values are roughly centred."""
    pool = np.zeros((blocks, hkv, 72 * page), np.uint8)
    pool[:, :, :64 * page] = rng.integers(0, 256, (blocks, hkv, 64 * page), dtype=np.uint8)
    for role, size in ((0, k_scale), (1, v_scale)):
        s = size * np.exp(0.5 * rng.normal(size=(blocks, hkv, page, 1)))
        z = -1.5 * s + 0.2 * s * rng.normal(size=s.shape)
        meta = np.concatenate([s, z], -1).astype(np.float16)
        pool[:, :, (64 + 4 * role) * page:(68 + 4 * role) * page] = meta.reshape(blocks, hkv, -1).view(np.uint8)
    return pool


def set_meta(pool, page, role, block, slot, scale, zero):
    at = (64 + 4 * role) * page + 4 * slot
    pool[block, :, at:at + 4] = np.array([scale, zero], np.float16).view(np.uint8)


class Block:
    """One call's inputs on host and device."""

    def __init__(self, seed, hq, hkv, page, lens, ns, rot="dense", dtype="f32", parents=None, q_scale=1.0, spare_rows=0,
                 k_scale=1.0, v_scale=1.0, gap=0):
        import oracle
        self.kvq, self.torch = gu.kvq_lib(), gu.torch_cuda()
        self.rng = rng = np.random.default_rng([77, seed])
        self.hq, self.hkv, self.page, self.dtype = hq, hkv, page, dtype
        self.lens, self.ns = list(lens), list(ns)
        self.mb = max(1, max(-(-x // page) for x in lens))
        need = sum(-(-x // page) for x in lens)
        self.blocks = need + 2
        ids = rng.permutation(self.blocks)
        self.table = np.zeros((len(lens), self.mb), np.int32)
        at = 0
        for b, x in enumerate(lens):
            self.table[b, :-(-x // page)] = ids[at:at - (-x // page)]
            at += -(-x // page)
        self.pool = make_pool(rng, self.blocks, hkv, page, k_scale, v_scale)
        self.cu = np.concatenate([[gap], gap + np.cumsum(ns)]).astype(np.int32)
        self.total = int(self.cu[-1]) + spare_rows
        q = rng.normal(size=(self.total, hq, 128)) * q_scale
        self.q = W.round_bf16(q.astype(np.float32)) if dtype == "bf16" else q.astype(np.float32)
        self.rot = W.make_rot(rot, 5, seed, hkv)
        self.r = oracle.rotations.rot_matrices(self.rot, hkv)
        self.parents = None
        if parents is not None:
            self.parents = np.full(self.total, -1, np.int32)
            for b, n in enumerate(ns):
                self.parents[self.cu[b]:self.cu[b] + n] = parents(rng, n)

    def layout(self):
        return self.kvq.make_layout(self.page, self.hkv, self.hq, self.blocks, self.mb)

    def device(self):
        t, i = self.torch, gu.dev_i32
        lay, max_q, max_len = self.layout(), max(self.ns), max(self.lens)
        size = self.kvq.kvq_query_block_workspace_size(lay, len(self.ns), self.total, max_q, max_len)
        return dict(lay=lay, q=gu.dev(self.q, self.dtype), cu=i(self.cu), max_q=max_q, lens=i(self.lens),
                    max_len=max_len, table=i(self.table), rot=self.kvq.DeviceRot.from_spec(self.rot),
                    pool=t.from_numpy(self.pool).cuda(), ws=t.full((size,), 0xA5, dtype=t.uint8, device="cuda"),
                    o=t.full((self.total, self.hq, 128), 7.25, device="cuda"),
                    parents=None if self.parents is None else i(self.parents))

    def launch(self, d, cross=False, stream=None):
        if cross:
            self.kvq.kvq_cross_attention(d["lay"], d["q"], d["cu"], d["max_q"], d["lens"], d["max_len"], d["table"],
                                         d["rot"], d["pool"], d["ws"], d["o"], stream=stream)
        else:
            self.kvq.kvq_tree_attention(d["lay"], d["q"], d["cu"], d["max_q"], d["parents"], d["lens"], d["max_len"],
                                        d["table"], d["rot"], d["pool"], d["ws"], d["o"], stream=stream)

    def run(self, cross=False):
        d = self.device()
        self.launch(d, cross)
        self.kvq.kvq_device_check()
        return d["o"].cpu().numpy()

    def check(self, got, cross=False, seqs=None):
        import oracle
        worst = 0.0
        for b in (range(len(self.ns)) if seqs is None else seqs):
            n, length, c0 = self.ns[b], self.lens[b], self.cu[b]
            kh, vh = oracle.cache.dequantized_sequence(self.pool.reshape(-1), self.hkv, self.page, self.table[b], length)
            see = None
            if not cross:
                see = oracle.tree.visible(n, length, None if self.parents is None else self.parents[c0:c0 + n])
            ref, mag, size = oracle.tree.block_attention(self.q[c0:c0 + n], kh, vh, self.r, self.hq // self.hkv, see)
            g = got[c0:c0 + n]
            assert np.isfinite(g).all()
            assert np.all(g[mag.sum(-1) == 0] == 0)
            bound = REL * (1 + size)[..., None] * np.sqrt((mag ** 2).mean(-1, keepdims=True))
            err = np.abs(g - ref)
            some = np.broadcast_to(bound > 0, err.shape)
            if some.any():
                worst = max(worst, float((err[some] / np.broadcast_to(bound, err.shape)[some]).max()))
        assert worst <= 1.0, worst
        inside = np.zeros(self.total, bool)
        inside[self.cu[0]:self.cu[-1]] = True
        assert np.all(got[~inside] == 7.25)
        return worst


def random_tree(rng, n):
    return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]


def star(rng, n):
    return [-1] * n


def comb(rng, n):  # a spine with a leaf at every node
    return [-1] + [(i - 1) // 2 * 2 if i % 2 else i - 2 for i in range(1, n)]


TREES = [
    # hq, hkv, page, lens, drafts, rot, dtype, parents
    (1, 1, 16, [1], [1], "identity", "f32", star),
    (2, 2, 8, [5, 8], [5, 8], "dense", "f32", random_tree),           # nothing before the drafts
    (4, 1, 16, [127, 128, 129], [3, 1, 7], "dense", "bf16", random_tree),
    (8, 1, 16, [300, 17], [2, 2], "signed_hadamard", "f32", star),
    (8, 4, 8, [1000, 63, 257], [16, 33, 8], "dense", "bf16", random_tree),
    (16, 2, 16, [520, 129], [9, 65], "dense", "f32", comb),           # 72 and 520 rows a KV head
    (32, 8, 16, [2049], [31], "signed_hadamard", "bf16", random_tree),
    (3, 3, 8, [70, 641, 9], [64, 1, 0], "identity", "bf16", random_tree),
    (4, 2, 16, [400], [300], "dense", "bf16", random_tree),           # a tree over several row tiles and key tiles
    (2, 1, 8, [300], [300], "identity", "f32", star),                 # slices in which a row sees nothing
    (1, 1, 16, [1030], [1024], "signed_hadamard", "bf16", random_tree),  # the largest tree
]


@pytest.mark.parametrize("hq,hkv,page,lens,ns,rot,dtype,shape", TREES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_tree(hq, hkv, page, lens, ns, rot, dtype, shape):
    blk = Block(1, hq, hkv, page, lens, ns, rot, dtype, shape, spare_rows=2)
    blk.check(blk.run())


CHAINS = [
    (4, 4, 16, [1, 2, 40], [1, 2, 33], "dense", "f32"),
    (8, 2, 16, [700, 128, 0], [130, 128, 0], "dense", "bf16"),
    (16, 2, 8, [333], [200], "signed_hadamard", "bf16"),
    (2, 1, 16, [1500], [1100], "identity", "f32"),                    # longer than any tree may be
]


@pytest.mark.parametrize("hq,hkv,page,lens,ns,rot,dtype", CHAINS, ids=str)
def test_chain(hq, hkv, page, lens, ns, rot, dtype):
    blk = Block(2, hq, hkv, page, lens, ns, rot, dtype)
    blk.check(blk.run())


CROSS = [
    (1, 1, 8, [1], [1], "identity", "f32"),
    (16, 16, 16, [150, 0, 37], [1, 5, 1], "dense", "bf16"),           # a sequence without states: zeros
    (8, 2, 16, [1000, 129], [40, 3], "dense", "f32"),
    (8, 1, 8, [64, 257, 31], [17, 0, 8], "signed_hadamard", "bf16"),
    (4, 4, 16, [385], [447], "dense", "bf16"),
]


@pytest.mark.parametrize("hq,hkv,page,lens,ns,rot,dtype", CROSS, ids=str)
def test_cross(hq, hkv, page, lens, ns, rot, dtype):
    blk = Block(3, hq, hkv, page, lens, ns, rot, dtype, spare_rows=1, gap=3)
    blk.check(blk.run(cross=True), cross=True)


@pytest.mark.parametrize("n", [127, 128, 129, 300])
@pytest.mark.parametrize("cross", [False, True])
def test_many_short_sequences(n, cross):
    """Around the number of sequences up to which every block lists the work itself; several units a slice."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, n).tolist()
    ns = [int(rng.integers(0, 12)) if cross else int(rng.integers(0, min(12, x) + 1)) for x in lens]
    blk = Block(20, 8, 4, 8, lens, ns, "dense", "bf16")
    blk.check(blk.run(cross), cross=cross, seqs=range(0, n, 5))


@pytest.mark.parametrize("hq,n", [(2, 5), (8, 3), (8, 30)])  # 10, 24 and 240 rows: each size of row tile
def test_logits_that_keep_rising(hq, n):
    """Keys that grow along the sequence, so that the running maximum passes every reference again and again."""
    blk = Block(21, hq, 1, 16, [2100], [n], "dense", "f32", random_tree, q_scale=3.0)
    for pos in range(2100):
        s = 0.02 * 1.0035 ** pos
        set_meta(blk.pool, 16, 0, blk.table[0, pos // 16], pos % 16, s, -1.5 * s)
    blk.check(blk.run())


def test_many_sequences_and_long_contexts():
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 90, 200).tolist() + [20011]
    ns = [int(rng.integers(1, min(5, x) + 1)) for x in lens]
    blk = Block(4, 8, 2, 16, lens, ns, "signed_hadamard", "bf16", random_tree)
    blk.check(blk.run(), seqs=[0, 7, 101, 199, 200])


@pytest.mark.parametrize("q_scale", [1e-3, 30.0])
@pytest.mark.parametrize("ns", [[9, 20], [2, 4], [5, 8]])
def test_flat_and_peaked_softmax(q_scale, ns):
    blk = Block(5, 8, 2, 16, [3001, 260], ns, "dense", "f32", random_tree, q_scale=q_scale)
    blk.check(blk.run())


@pytest.mark.parametrize("k_scale,v_scale", [(1e-3, 1e-3), (50.0, 3000.0), (1e-6, 1e-6)])
def test_extreme_scales(k_scale, v_scale):
    """fp16 scales near their largest and in their subnormal range (some of them exactly 0)."""
    blk = Block(6, 4, 1, 16, [500], [12], "dense", "f32", random_tree, k_scale=k_scale, v_scale=v_scale)
    blk.check(blk.run())


def test_queries_of_very_different_size_in_one_tile():
    blk = Block(7, 4, 1, 16, [400], [16], "dense", "f32", random_tree)
    blk.q *= (10.0 ** np.linspace(-6, 1.5, 16)).astype(np.float32)[:, None, None]
    blk.check(blk.run())


def test_values_of_very_different_scale():
    """A token with a large weight and a tiny scale beside tokens with large scales, and constant groups (scale 0)."""
    blk = Block(8, 2, 1, 16, [300], [6], "identity", "f32", random_tree)
    for i, s in enumerate([0.0, 6e-8, 1e-4, 200.0, 0.0, 1.0] * 40):
        set_meta(blk.pool, 16, 1, blk.table[0, i // 16], i % 16, s, -1.5 * s + 0.25)
        if i % 7 == 0:
            set_meta(blk.pool, 16, 0, blk.table[0, i // 16], i % 16, 0.0, 0.125)
    blk.check(blk.run())


@pytest.mark.parametrize("poison", [np.nan, np.inf, -np.inf, 65504.0, -65504.0])
def test_what_is_not_seen_does_not_count(poison):
    """NaN, infinities and the type's extremes in the slots behind a sequence and in drafts off a row's path."""
    lens, n, page = [133], [8], 16
    parents = [-1, 0, 1, -1, 3, 4, 5, -1]  # paths 0-1-2, 3-4-5-6, 7
    blk = Block(9, 4, 2, page, lens, n, "dense", "f32", lambda rng, k: parents)
    for pos in [128, 129, 130, 131, *range(133, 144)]:  # drafts 3 .. 6, and behind the end
        for role in (0, 1):
            set_meta(blk.pool, page, role, blk.table[0, pos // page], pos % page, poison, poison)
    got = blk.run()
    for pos in [128, 129, 130, 131, *range(133, 144)]:
        for role in (0, 1):
            set_meta(blk.pool, page, role, blk.table[0, pos // page], pos % page, 1.0, 0.0)
    seen = [0, 1, 2, 7]
    import oracle
    kh, vh = oracle.cache.dequantized_sequence(blk.pool.reshape(-1), 2, page, blk.table[0], 133)
    ref, mag, size = oracle.tree.block_attention(blk.q, kh, vh, blk.r, 2, oracle.tree.visible(8, 133, parents))
    bound = REL * (1 + size)[..., None] * np.sqrt((mag ** 2).mean(-1, keepdims=True))
    assert np.all(np.abs(got - ref)[seen] <= bound[seen])


def test_a_bad_query_row_spoils_only_itself():
    blk = Block(10, 4, 2, 16, [200, 90], [7, 5], "dense", "f32", random_tree)
    ref = blk.run()
    blk.q[3, 1] = np.inf
    blk.q[9, 2, 5] = np.nan
    got = blk.run()
    keep = np.ones((12, 4), bool)
    keep[3, 1] = keep[9, 2] = False
    np.testing.assert_allclose(got[keep], ref[keep], rtol=0, atol=2e-5 * np.abs(ref).max())


def test_same_bits_every_time_and_on_another_stream():
    blk = Block(11, 8, 2, 16, [1500, 700, 90], [13, 5, 60], "dense", "bf16", random_tree)
    a = blk.run()
    assert np.array_equal(a, blk.run())
    d = blk.device()
    side = blk.torch.cuda.Stream()
    blk.torch.cuda.synchronize()
    blk.launch(d, stream=side)
    side.synchronize()
    assert np.array_equal(a, d["o"].cpu().numpy())


def test_captured_and_replayed_with_new_inputs():
    blk = Block(12, 8, 2, 16, [700, 333], [9, 30], "signed_hadamard", "bf16", random_tree)
    d = blk.device()
    blk.launch(d)
    blk.torch.cuda.synchronize()
    graph = blk.torch.cuda.CUDAGraph()
    with blk.torch.cuda.graph(graph):
        blk.launch(d)
    other = Block(13, 8, 2, 16, [650, 333], [7, 30], "signed_hadamard", "bf16", random_tree)
    other.lens, other.ns = [650, 333], [7, 30]
    d["q"][:other.total].copy_(gu.dev(other.q, "bf16"))
    d["cu"].copy_(gu.dev_i32(other.cu))
    d["lens"].copy_(gu.dev_i32(other.lens))
    d["parents"][:other.total].copy_(gu.dev_i32(other.parents))
    d["o"].fill_(7.25)
    graph.replay()
    blk.kvq.kvq_device_check()
    got = d["o"].cpu().numpy()
    other.pool, other.table, other.rot, other.r = blk.pool, blk.table, blk.rot, blk.r
    other.total = blk.total
    other.check(got)


def test_pool_beyond_four_gigabytes():
    torch, kvq = gu.torch_cuda(), gu.kvq_lib()
    hkv, page = 8, 16
    blocks = (5 << 30) // (hkv * 72 * page)
    blk = Block(14, 8, hkv, page, [200], [10], "identity", "f32", random_tree)
    d = blk.device()
    lay = kvq.make_layout(page, hkv, 8, blocks, blk.mb)
    big = torch.zeros(blocks, hkv, 72 * page, dtype=torch.uint8, device="cuda")
    far = blocks - 1 - np.arange(blk.mb)
    for i in range(blk.mb):
        big[int(far[i])] = d["pool"][int(blk.table[0, i])]
    d["lay"], d["pool"], d["table"] = lay, big, gu.dev_i32(far[None])
    blk.launch(d)
    kvq.kvq_device_check()
    blk.check(d["o"].cpu().numpy())


def test_one_query_equals_the_decode():
    """A single query against everything is kvq_decode_attention (to both kernels' rounding)."""
    blk = Block(15, 32, 8, 16, [1000, 77, 2048], [1, 1, 1], "dense", "bf16")
    d = blk.device()
    blk.launch(d, cross=True)
    kvq, torch = blk.kvq, blk.torch
    ws = torch.empty(kvq.kvq_decode_workspace_size(d["lay"], 3, 2048), dtype=torch.uint8, device="cuda")
    o = torch.empty(3, 32, 128, device="cuda")
    kvq.kvq_decode_attention(d["lay"], d["q"], d["lens"], 2048, d["table"], d["rot"], d["pool"], ws, o)
    kvq.kvq_device_check()
    blk.check(d["o"].cpu().numpy(), cross=True)
    assert gu.out_err(d["o"].cpu().numpy(), o.cpu().numpy()) <= gu.OUT_TOL


def _flagged(blk, d, cross=False):
    blk.launch(d, cross)
    with pytest.raises(blk.kvq.KvqError) as e:
        blk.kvq.kvq_device_check()
    assert e.value.status == blk.kvq.KVQ_EDEVICE_FLAG
    blk.kvq.kvq_device_check()  # cleared
    return d["o"].cpu().numpy()


def test_bad_lengths_and_pages_are_flagged_and_the_rest_is_right():
    blk = Block(16, 4, 2, 16, [90, 50, 140], [5, 4, 6], "dense", "f32", random_tree)
    d = blk.device()
    d["lens"].copy_(gu.dev_i32([90, 3, 140]))  # more drafts than tokens
    blk.check(_flagged(blk, d), seqs=[0, 2])
    for bad in (-1, blk.blocks):
        d = blk.device()
        d["table"][1, 2] = bad
        got = _flagged(blk, d)
        blk.check(got, seqs=[0, 2])
    d = blk.device()
    d["cu"].copy_(gu.dev_i32([0, 5, 9, 10_000]))
    blk.check(_flagged(blk, d), seqs=[0, 1])


def test_bad_parents_are_flagged_and_taken_as_roots():
    blk = Block(17, 4, 2, 16, [60], [6], "dense", "f32", lambda rng, n: [-1, 0, 1, 1, 0, 4])
    d = blk.device()
    d["parents"].copy_(gu.dev_i32([-1, 0, 5, 1, -7, 4]))
    got = _flagged(blk, d)
    blk.parents = np.array([-1, 0, -1, 1, -1, 4], np.int32)
    blk.check(got)


def test_two_calls_at_once_with_a_workspace_each():
    blocks = [Block(41, 8, 2, 16, [3000, 700], [13, 40], "dense", "bf16", random_tree),
              Block(42, 2, 1, 8, [2500, 90, 33], [5, 2, 1], "signed_hadamard", "f32", random_tree)]
    want = [b.run() for b in blocks]
    ds = [b.device() for b in blocks]
    torch = blocks[0].torch
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, d, s in zip(blocks, ds, streams):
            b.launch(d, stream=s)
    torch.cuda.synchronize()
    blocks[0].kvq.kvq_device_check()
    for w, d in zip(want, ds):
        assert np.array_equal(w, d["o"].cpu().numpy())
