"""kvq_plan_pages and kvq_tree_commit against the oracle (whole numbers: equal), and a speculative step end to end."""
import numpy as np
import pytest

import gpu_util as gu
from int2_kv_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu


class Pages:
    def __init__(self, seed, n, page, mb, blocks, head=None):
        self.kvq, self.torch = gu.kvq_lib(), gu.torch_cuda()
        self.rng = np.random.default_rng([5, seed])
        self.n, self.page, self.mb, self.blocks = n, page, mb, blocks
        self.table = np.full((n, mb), -9, np.int64)
        self.ring = self.rng.permutation(blocks)
        self.head = 3 * blocks + int(self.rng.integers(blocks)) if head is None else head
        self.ring = np.roll(self.ring, self.head % blocks)
        self.tail = self.head + blocks
        self.lens = np.zeros(n, np.int64)
        self.lay = self.kvq.make_layout(page, 1, 1, blocks, mb)

    def step(self, new, max_new, expect_ok=True):
        import oracle
        t = self.torch
        table, ring = gu.dev_i32(self.table), gu.dev_i32(self.ring)
        rin = t.tensor([self.head, self.tail], device="cuda")
        rout = t.zeros(2, dtype=t.int64, device="cuda")
        cu = t.full((self.n + 1,), 77, dtype=t.int32, device="cuda")
        slots = t.full((max_new,), 77, dtype=t.int64, device="cuda")
        ws = t.empty(self.kvq.kvq_plan_workspace_size(self.n), dtype=t.uint8, device="cuda")
        self.kvq.kvq_plan_pages(self.lay, gu.dev_i32(self.lens), gu.dev_i32(new), table, ring, rin, rout, cu, slots, ws)
        if expect_ok:
            self.kvq.kvq_device_check()
        else:
            with pytest.raises(self.kvq.KvqError, match="plan"):
                self.kvq.kvq_device_check()
        want = oracle.tree.plan_pages(self.page, self.blocks, self.lens, new, self.table, self.ring, self.head,
                                      self.tail, max_new)
        got = (table, ring, rout[0], rout[1], cu, slots)
        for name, g, w in zip(("table", "ring", "head", "tail", "cu", "slots"), got, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
        if expect_ok:
            self.table, self.ring, self.head, self.tail = want[:4]
            self.lens = np.asarray(new, np.int64)


@pytest.mark.parametrize("n,page", [(1, 16), (5, 8), (1023, 16), (1024, 8), (1025, 16), (5000, 8), (16384, 8), (16385, 16)])
def test_plans_over_many_steps(n, page):
    p = Pages(n, n, page, 9, 9 * n + 3)
    for _ in range(6):
        new = p.rng.integers(0, 9 * page + 1, n)
        keep = p.rng.random(n) < 0.3
        new[keep] = p.lens[keep]
        p.step(new, int(np.maximum(new - p.lens, 0).sum()) + int(p.rng.integers(0, 5)))


def test_one_long_request_and_none_at_all():
    p = Pages(2, 1, 16, 5000, 5000, head=0)
    p.step([80000], 80000)
    p.step([80000], 0)
    p.step([1], 3)
    p.step([1], 1)


@pytest.mark.parametrize("n", [3, 1500, 17000])
def test_refused_plans_change_nothing(n):
    p = Pages(3, n, 8, 4, 3 * n)
    p.step(np.full(n, 17), 17 * n)                                # every page is taken
    p.step(np.full(n, 32), 17 * n, expect_ok=False)               # too few pages
    p.step(np.full(n, 24), 7 * n - 1, expect_ok=False)            # more tokens than max_new
    for bad in (33, -1, 2**31 - 1):
        new = p.lens.copy()
        new[n // 2] = bad
        p.step(new, 100, expect_ok=False)
    good = (p.head, p.tail)
    for bad in ((-1, 5), (10, 9), (0, 3 * n + 1)):
        p.head, p.tail = bad
        p.step(p.lens, 4, expect_ok=False)
    p.head, p.tail = good
    p.step(np.zeros(n, np.int64), 0)


def test_a_page_id_outside_the_pool_is_flagged():
    p = Pages(4, 2, 16, 3, 6)
    p.ring[(p.head + 1) % 6] = 6
    t = p.torch
    table, ring = gu.dev_i32(p.table), gu.dev_i32(p.ring)
    rout, cu = t.zeros(2, dtype=t.int64, device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    slots = t.zeros(60, dtype=t.int64, device="cuda")
    ws = t.empty(p.kvq.kvq_plan_workspace_size(2), dtype=t.uint8, device="cuda")
    p.kvq.kvq_plan_pages(p.lay, gu.dev_i32([0, 0]), gu.dev_i32([32, 5]), table, ring,
                         t.tensor([p.head, p.tail], device="cuda"), rout, cu, slots, ws)
    with pytest.raises(p.kvq.KvqError, match="block-table"):
        p.kvq.kvq_device_check()
    s = slots.cpu().numpy()
    assert np.all(s[16:32] == -1) and np.all(s[:16] >= 0) and np.all(s[32:37] >= 0) and np.all(s[37:] == -1)


COMMITS = [
    # page, heads, drafts, accepted paths
    (16, 1, [1], [[0]]),
    (8, 3, [5, 9, 0, 4], [[1, 2, 4], [], [], [0, 1, 2, 3]]),
    (16, 8, [64], [[2, 3, 9, 40, 63]]),
    (8, 9, [100, 70], [list(range(3, 99, 2)), list(range(21, 70))]),  # paths longer than a warp's batch
]


@pytest.mark.parametrize("page,h,ns,paths", COMMITS, ids=lambda v: str(v)[:30])
def test_commit(page, h, ns, paths):
    import oracle
    kvq, torch, rng = gu.kvq_lib(), gu.torch_cuda(), np.random.default_rng(8)
    n, total = len(ns), sum(ns)
    blocks = total // page + 3
    slots = rng.permutation(blocks * page)[:total].astype(np.int64)
    cu = np.concatenate([[0], np.cumsum(ns)])
    most = max(map(len, paths)) + 1
    acc = np.full((n, most), 2**31 - 1, np.int64)  # entries behind a path are not read
    for b, x in enumerate(paths):
        acc[b, :len(x)] = x
    n_acc = np.array([len(x) for x in paths])
    lens = np.array(ns) + 37
    pool = rng.integers(0, 256, blocks * h * 72 * page, dtype=np.uint8)
    d = torch.from_numpy(pool.copy()).cuda()
    new = torch.zeros(n, dtype=torch.int32, device="cuda")
    kvq.kvq_tree_commit(kvq.make_layout(page, h, h, blocks, 1), gu.dev_i32(cu), gu.dev_i32(acc), gu.dev_i32(n_acc),
                        torch.from_numpy(slots).cuda(), gu.dev_i32(lens), new, d)
    kvq.kvq_device_check()
    want, want_lens = oracle.tree.commit(pool, h, page, cu, acc, n_acc, slots, lens)
    assert np.array_equal(d.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), want_lens)


def test_bad_paths_are_flagged_and_move_nothing():
    kvq, torch, rng = gu.kvq_lib(), gu.torch_cuda(), np.random.default_rng(9)
    page, h, blocks = 16, 2, 4
    pool = rng.integers(0, 256, blocks * h * 72 * page, dtype=np.uint8)
    slots = torch.arange(20, 30, device="cuda")
    lay = kvq.make_layout(page, h, h, blocks, 1)
    for acc, n_acc, lens, new_len in (([3, 2], 2, 40, 30), ([1, 10], 2, 40, 30), ([-1, 2], 2, 40, 30), ([1, 2], 3, 40, 30),
                                      ([1, 2], -1, 40, 30), ([1, 1], 2, 40, 30), ([1, 2], 2, 9, 9)):
        d = torch.from_numpy(pool.copy()).cuda()
        new = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvq.kvq_tree_commit(lay, gu.dev_i32([0, 10]), gu.dev_i32([acc]), gu.dev_i32([n_acc]), slots, gu.dev_i32([lens]),
                            new, d)
        with pytest.raises(kvq.KvqError, match="path"):
            kvq.kvq_device_check()
        assert np.array_equal(d.cpu().numpy(), pool) and int(new[0]) == new_len
    # a slot outside the pool: that move is left out
    slots[3] = blocks * page
    d = torch.from_numpy(pool.copy()).cuda()
    kvq.kvq_tree_commit(lay, gu.dev_i32([0, 10]), gu.dev_i32([[3]]), gu.dev_i32([1]), slots, gu.dev_i32([40]), new, d)
    with pytest.raises(kvq.KvqError, match="block-table"):
        kvq.kvq_device_check()
    assert np.array_equal(d.cpu().numpy(), pool)


@pytest.mark.parametrize("rot,dtype,page", [("dense", "bf16", 16), ("signed_hadamard", "f32", 8)])
def test_speculative_step_equals_decoding_one_token_at_a_time(rot, dtype, page):
    """plan -> append the drafts -> tree attention -> commit the path -> plan -> decode, for three requests that
    share one pool: the accepted rows are what kvq_decode_step gives token by token, and the cache bytes are equal."""
    hq, hkv, base = 8, 2, [45, 130, 8]
    parents = [[-1, 0, 0, 1, 2, 4], [-1, -1, 1], [-1, 0, 1, 2, 0]]
    paths = [[0, 2, 4, 5], [1, 2], [0, 1, 2, 3]]
    ns, n = [len(x) for x in parents], 3
    case = W.decode_case(71, [b + k for b, k in zip(base, ns)], hq, hkv, 128, rot, dtype, page_tokens=page, clip_k=0.95,
                         spare_blocks=4, n_cal=128)
    g = gu.GpuCase(case)
    kvq, torch = g.kvq, g.torch
    mb = 20
    blocks = 3 * mb
    lay = kvq.make_layout(page, hkv, hq, blocks, mb)
    rng = np.random.default_rng(3)
    kv = [case.kv(b) for b in range(n)]
    queries = rng.normal(size=(sum(ns), hq, 128)).astype(np.float32)
    queries = W.round_bf16(queries)
    i64 = dict(dtype=torch.int64, device="cuda")
    table = torch.zeros(n, mb, dtype=torch.int32, device="cuda")
    ring = gu.dev_i32(rng.permutation(blocks))
    counters = [torch.tensor([0, blocks], device="cuda"), torch.zeros(2, **i64)]
    pws = torch.empty(kvq.kvq_plan_workspace_size(n), dtype=torch.uint8, device="cuda")
    pool = torch.zeros(kvq.kvq_pool_bytes(lay), dtype=torch.uint8, device="cuda")

    def plan(old, new, room):
        cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        slots = torch.zeros(room, **i64)
        kvq.kvq_plan_pages(lay, old, new, table, ring, counters[0], counters[1], cu, slots, pws)
        counters.reverse()
        return cu, slots

    def append(rows, cu, start):
        ks = np.concatenate([kv[b][0][r] for b, r in enumerate(rows)])
        vs = np.concatenate([kv[b][1][r] for b, r in enumerate(rows)])
        kvq.kvq_quantize_append(lay, gu.dev(ks, dtype), gu.dev(vs, dtype), cu, start, table, g.rot_k, g.rot_v,
                                g.mu_rot_dev, case.clip_k, case.clip_v, pool)

    zero, l0 = gu.dev_i32([0] * n), gu.dev_i32(base)
    cu, _ = plan(zero, l0, sum(base))
    append([list(range(b)) for b in base], cu, zero)
    grown = gu.dev_i32([b + k for b, k in zip(base, ns)])
    cu, slots = plan(l0, grown, sum(ns))
    append([list(range(b, b + k)) for b, k in zip(base, ns)], cu, l0)
    o = torch.zeros(sum(ns), hq, 128, device="cuda")
    most = max(b + k for b, k in zip(base, ns))
    ws = torch.empty(kvq.kvq_query_block_workspace_size(lay, n, sum(ns), max(ns), most), dtype=torch.uint8, device="cuda")
    kvq.kvq_tree_attention(lay, gu.dev(queries, dtype), cu, max(ns), gu.dev_i32(sum(parents, [])), grown, most, table,
                           g.rot_k, pool, ws, o)
    depth = max(map(len, paths))
    acc = gu.dev_i32([x + [0] * (depth - len(x)) for x in paths])
    new_lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    kvq.kvq_tree_commit(lay, cu, acc, gu.dev_i32([len(x) for x in paths]), slots, grown, new_lens, pool)
    plan(grown, new_lens, 0)
    kvq.kvq_device_check()
    assert new_lens.tolist() == [b + len(x) for b, x in zip(base, paths)]
    held = sum(-(-x // page) for x in new_lens.tolist())
    assert int(counters[0][1] - counters[0][0]) == blocks - held

    # the same tokens one at a time into a pool of their own
    alone = torch.zeros_like(pool)
    own_table = gu.dev_i32(np.arange(n * mb).reshape(n, mb))
    start = np.concatenate([[0], np.cumsum(base)])
    ks, vs = (np.concatenate([kv[b][i][:base[b]] for b in range(n)]) for i in (0, 1))
    kvq.kvq_quantize_append(lay, gu.dev(ks, dtype), gu.dev(vs, dtype), gu.dev_i32(start), zero, own_table, g.rot_k,
                            g.rot_v, g.mu_rot_dev, case.clip_k, case.clip_v, alone)
    dws = torch.empty(kvq.kvq_decode_workspace_size(lay, n, mb * page), dtype=torch.uint8, device="cuda")
    step_o = torch.zeros(n, hq, 128, device="cuda")
    first = np.concatenate([[0], np.cumsum(ns)])
    for i in range(depth):
        live = [b for b in range(n) if i < len(paths[b])]
        rows = [base[b] + paths[b][i] if b in live else 0 for b in range(n)]
        lens = [base[b] + i + 1 if b in live else 0 for b in range(n)]
        qs = np.stack([queries[first[b] + paths[b][i]] if b in live else queries[0] for b in range(n)])
        kvq.kvq_decode_step(lay, gu.dev(qs, dtype), gu.dev(np.stack([kv[b][0][rows[b]] for b in range(n)]), dtype),
                            gu.dev(np.stack([kv[b][1][rows[b]] for b in range(n)]), dtype), gu.dev_i32(lens), mb * page,
                            own_table, g.rot_k, g.rot_v, g.mu_rot_dev, case.clip_k, case.clip_v, alone, dws, step_o)
        for b in live:
            got = o[first[b] + paths[b][i]].cpu().numpy()
            assert gu.out_err(got, step_o[b].cpu().numpy()) <= gu.OUT_TOL, (b, i)
    kvq.kvq_device_check()
    for b in range(n):
        length = base[b] + len(paths[b])
        for which in ("k", "v"):
            for x, y in zip(gu.seq_codes_meta(pool.cpu().numpy(), hkv, page, table[b].cpu().numpy(), length, which),
                            gu.seq_codes_meta(alone.cpu().numpy(), hkv, page, own_table[b].cpu().numpy(), length, which)):
                assert np.array_equal(x, y)


@pytest.mark.parametrize("n", [4, 1100])  # both sizes of the plan's blocks
def test_a_captured_grow_commit_shrink_step_replays(n):
    """One graph: grow by the drafts, commit, give pages back, with the ring's counters going from one pair to the other
    and back; replayed with new drafts and paths, it follows the oracle."""
    import oracle
    page, mb, h, most = 8, 12, 2, 6
    p = Pages(31, n, page, mb, mb * n)
    kvq, t, rng, blocks = p.kvq, p.torch, p.rng, p.blocks
    lay = kvq.make_layout(page, h, h, blocks, mb)
    pool = rng.integers(0, 256, blocks * h * 72 * page, dtype=np.uint8)
    d_pool, table, ring = t.from_numpy(pool.copy()).cuda(), gu.dev_i32(p.table), gu.dev_i32(p.ring)
    pairs = [t.tensor([p.head, p.tail], device="cuda"), t.zeros(2, dtype=t.int64, device="cuda")]
    lens, grown, kept = (t.zeros(n, dtype=t.int32, device="cuda") for _ in range(3))
    acc, n_acc = t.zeros(n, most, dtype=t.int32, device="cuda"), t.zeros(n, dtype=t.int32, device="cuda")
    cu, cu2 = (t.zeros(n + 1, dtype=t.int32, device="cuda") for _ in range(2))
    slots, none = t.zeros(most * n, dtype=t.int64, device="cuda"), t.zeros(0, dtype=t.int64, device="cuda")
    ws = t.empty(kvq.kvq_plan_workspace_size(n), dtype=t.uint8, device="cuda")

    def step():
        kvq.kvq_plan_pages(lay, lens, grown, table, ring, pairs[0], pairs[1], cu, slots, ws)
        kvq.kvq_tree_commit(lay, cu, acc, n_acc, slots, grown, kept, d_pool)
        kvq.kvq_plan_pages(lay, grown, kept, table, ring, pairs[1], pairs[0], cu2, none, ws)
        lens.copy_(kept)

    step()  # nothing grows: changes nothing
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    at = np.zeros(n, np.int64)
    for _ in range(5):
        drafts = rng.integers(0, most + 1, n)
        count = np.array([rng.integers(0, x + 1) for x in drafts])
        paths = np.zeros((n, most), np.int64)
        for b in range(n):
            paths[b, :count[b]] = np.sort(rng.permutation(drafts[b])[:count[b]])
        grown.copy_(gu.dev_i32(at + drafts))
        acc.copy_(gu.dev_i32(paths))
        n_acc.copy_(gu.dev_i32(count))
        graph.replay()
        kvq.kvq_device_check()
        p.table, p.ring, p.head, p.tail, c, s = oracle.tree.plan_pages(
            page, blocks, at, at + drafts, p.table, p.ring, p.head, p.tail, most * n)
        pool, new = oracle.tree.commit(pool, h, page, c, paths, count, s, at + drafts)
        p.table, p.ring, p.head, p.tail = oracle.tree.plan_pages(
            page, blocks, at + drafts, new, p.table, p.ring, p.head, p.tail, 0)[:4]
        at = np.asarray(new, np.int64)
        for name, g, w in (("table", table, p.table), ("ring", ring, p.ring), ("counters", pairs[0], [p.head, p.tail]),
                           ("lens", lens, at), ("slots", slots, s), ("pool", d_pool, pool)):
            np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


def test_commit_with_its_arrays_side_by_side_in_one_buffer():
    import oracle
    kvq, torch, rng = gu.kvq_lib(), gu.torch_cuda(), np.random.default_rng(10)
    page, h, ns, paths = 8, 3, [5, 9, 4], [[1, 2, 4], [], [0, 2]]
    n, total, most = 3, sum(ns), 3
    cu, blocks = np.concatenate([[0], np.cumsum(ns)]), 4
    acc = np.array([x + [7] * (most - len(x)) for x in paths])
    n_acc, lens = np.array([len(x) for x in paths]), np.array(ns) + 20
    slots = rng.permutation(blocks * page)[:total].astype(np.int64)
    pool = rng.integers(0, 256, blocks * h * 72 * page, dtype=np.uint8)
    buf = gu.dev_i32(np.concatenate([cu, acc.ravel(), [-1] * n, n_acc, lens]))
    at = np.cumsum([0, n + 1, n * most, n, n, n])
    d_cu, d_acc, new, d_n_acc, d_lens = (buf[i:j] for i, j in zip(at, at[1:]))
    d = torch.from_numpy(pool.copy()).cuda()
    kvq.kvq_tree_commit(kvq.make_layout(page, h, h, blocks, 1), d_cu, d_acc.view(n, most), d_n_acc,
                        torch.from_numpy(slots).cuda(), d_lens, new, d)
    kvq.kvq_device_check()
    want, want_lens = oracle.tree.commit(pool, h, page, cu, acc, n_acc, slots, lens)
    assert np.array_equal(d.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), want_lens)
    with pytest.raises(kvq.KvqError, match="overlap"):
        kvq.kvq_tree_commit(kvq.make_layout(page, h, h, blocks, 1), d_cu, d_acc.view(n, most), d_n_acc,
                            torch.from_numpy(slots).cuda(), d_lens, d_n_acc, d)
