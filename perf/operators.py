"""The speculative-decoding and cross-attention operators over the paged INT2 cache, as measured cases.

* ``tree``    attention of a tree of drafted tokens (or, ``nodes`` in a row, a causal chunk) over the cache;
* ``cross``   attention of query blocks over cached encoder states of another length;
* ``plan``    block tables, the free-page ring and the slot map from the requests' old and new lengths;
* ``commit``  the accepted path's cache records moved to the front of the draft's slots.

``run`` computes each either in its plain form (elementary torch operations in fp32 / int64) or, with ``own``
set, through the package's entry points.  ``exact`` is the definition in fp64, written apart.

The cache pool is uint8 [num_blocks][H_kv][72 P]: per (page, head) K codes (32 bytes a token), V codes, then
(fp16 scale, fp16 zero) of the keys and of the values; a value is zero + scale * code.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------
def _attn(name, kind, seqs, ctx, nodes, hq, hkv, page, rot, dtype, ragged, tree=False):
    c = dict(kind=kind, seqs=seqs, ctx=ctx, nodes=nodes, hq=hq, hkv=hkv, page=page, rot=rot, dtype=dtype,
             ragged=ragged, tree=tree)
    return dict(c, name=name) if name else c


def _plan(name, seqs, ctx, new, shrink, page):
    c = dict(kind="plan", seqs=seqs, ctx=ctx, new=new, shrink=shrink, page=page)
    return dict(c, name=name) if name else c


def _commit(name, seqs, nodes, depth, hkv, page):
    c = dict(kind="commit", seqs=seqs, nodes=nodes, depth=depth, hkv=hkv, page=page)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's speculative step: a tree of 8 drafts on a short context; latency counts
        _attn("tree_1x8_on_1k", "tree", 1, 1000, 8, 32, 8, 16, "dense", "bf16", False, True),
        # a serving batch verifying trees of 32 drafts on 16k contexts (the decode benchmark's geometry)
        _attn("tree_16x32_on_16k", "tree", 16, 16384, 32, 32, 8, 16, "dense", "bf16", False, True),
        # ragged requests: lengths and draft counts all different, 8 query heads a KV head, small pages, fp32
        _attn("tree_ragged_7_g8", "tree", 7, 9001, 61, 64, 8, 8, "signed_hadamard", "f32", True, True),
        # a chunk of a long prompt against what is cached already (a chain, not a tree)
        _attn("chunk_4x512_on_8k", "tree", 4, 8704, 512, 32, 8, 16, "dense", "bf16", False, False),
        # one decoder token a sequence against 1500 encoder states
        _attn("cross_16x1_to_1500", "cross", 16, 1500, 1, 16, 16, 16, "signed_hadamard", "bf16", False),
        # a decoder's whole prompt against 1500 encoder states, odd query counts
        _attn("cross_8x447_to_1500", "cross", 8, 1500, 447, 16, 16, 16, "dense", "bf16", False),
        # ragged queries and states, one sequence without states, fp32
        _attn("cross_ragged_33", "cross", 33, 4099, 40, 16, 4, 8, "identity", "f32", True),
        # page plan of one decode step of 256 requests (some of them finished or rolled back)
        _plan("plan_256_step", 256, 16384, 1, 0.2, 16),
        # page plan of a prefill wave: 64 prompts of up to 8k new tokens
        _plan("plan_64_prefill", 64, 9000, 8192, 0.0, 16),
        # page plan of many short requests
        _plan("plan_8191_mixed", 8191, 2000, 33, 0.4, 8),
        # commit after the verification of a batch of small trees
        _commit("commit_16x32", 16, 32, 5, 8, 16),
        # commit of a large batch with deep acceptances
        _commit("commit_512x64", 512, 64, 24, 8, 16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "cross", "cross", "plan", "commit"])
    if kind in ("tree", "cross"):
        hkv = rng.choice([1, 2, 4, 5, 8, 16])
        gqa = rng.choice([1, 2, 4, 8])
        page = rng.choice([8, 16])
        rot = rng.choice(["dense", "signed_hadamard", "identity"])
        dtype = rng.choice(["bf16", "f32"])
        tree = kind == "tree" and rng.random() < 0.7
        while True:
            seqs, ctx = _log_int(rng, 1, 40), _log_int(rng, 16, 24000)
            nodes = _log_int(rng, 1, 128 if tree else 700)
            rows = seqs * nodes * gqa * hkv
            # no dearer than the largest listed case, padded score matrices that fit
            if nodes <= ctx and rows * ctx * 512 < 2.0e11 and rows * ctx * 4 < 3.0e9 and seqs * ctx * hkv < 2.5e6:
                break
        return _attn(None, kind, seqs, ctx, nodes, hkv * gqa, hkv, page, rot, dtype, rng.random() < 0.7, tree)
    if kind == "plan":
        while True:
            seqs, new = _log_int(rng, 1, 12000), _log_int(rng, 1, 8192)
            if seqs * new < 600000:
                break
        return _plan(None, seqs, _log_int(rng, 64, 16000) + new, new, rng.choice([0.0, 0.1, 0.5]), rng.choice([8, 16]))
    nodes = _log_int(rng, 1, 128)
    return _commit(None, _log_int(rng, 1, 512), nodes, rng.randint(1, min(nodes, 24)), rng.choice([1, 2, 4, 8]),
                   rng.choice([8, 16]))


def _shape_rng(case):
    """Lengths belong to the case, not to the seed: work() has to know them."""
    return random.Random("|".join(f"{k}={case[k]}" for k in sorted(case) if k != "name"))


def _attn_lens(case):
    """(cached tokens incl. drafts, queries) per sequence."""
    r, n = _shape_rng(case), case["seqs"]
    if not case["ragged"]:
        return [case["ctx"]] * n, [case["nodes"]] * n
    lens, qs = [], []
    for b in range(n):
        q = case["nodes"] if b == 0 else r.randint(1, case["nodes"])
        low = q if case["kind"] == "tree" else 1
        s = case["ctx"] if b == 0 else r.randint(low, case["ctx"])
        if case["kind"] == "cross" and n > 2 and b == n // 2:
            s = 0
        lens.append(s)
        qs.append(q)
    return lens, qs


def _plan_lens(case):
    r = _shape_rng(case)
    old, new = [], []
    for b in range(case["seqs"]):
        n = case["new"] if case["new"] == 1 else r.randint(1, case["new"])
        o = r.randint(0, case["ctx"] - n)
        if r.random() < case["shrink"]:
            old.append(o + n)
            new.append(r.randint(0, o + n) if r.random() < 0.3 else o)
        else:
            old.append(o)
            new.append(o + n)
    return old, new


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _quantized_pool(gen, blocks, hkv, page):
    """A pool of packed 2-bit codes of normal keys and values (rotated caches look normal per group)."""
    pool = torch.empty(blocks, hkv, 72 * page, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * page * 128))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        for role in range(2):
            x = torch.randn(n, hkv, page, 128, generator=gen, device=DEV)
            x *= torch.exp(0.4 * torch.randn(n, hkv, page, 1, generator=gen, device=DEV))
            lo, hi = 0.95 * x.amin(-1, keepdim=True), 0.95 * x.amax(-1, keepdim=True)
            s, z = ((hi - lo) / 3).half(), lo.half()
            c = torch.clamp(torch.round((x - z.float()) / s.float()), 0, 3).to(torch.uint8)
            c = c.view(n, hkv, page, 32, 4)
            c = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
            pool[i:i + n, :, 32 * page * role:32 * page * (role + 1)] = c.reshape(n, hkv, -1)
            meta = torch.cat([s, z], -1).contiguous().view(torch.uint8)
            pool[i:i + n, :, 64 * page + 4 * page * role:64 * page + 4 * page * (role + 1)] = meta.reshape(n, hkv, -1)
    return pool


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _commit_shape(case):
    """(drafts, accepted) per sequence."""
    r = _shape_rng(case)
    xs = [r.randint(max(1, case["nodes"] // 2), case["nodes"]) for _ in range(case["seqs"])]
    return xs, [r.randint(0, min(case["depth"], x)) for x in xs]


def _prepare_attn(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = random.Random(seed)
    lens, qs = _attn_lens(case)
    page, hq, hkv, n = case["page"], case["hq"], case["hkv"], case["seqs"]
    mb = max(1, max(-(-s // page) for s in lens))
    need = sum(-(-s // page) for s in lens)
    blocks = need + 3
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(n, mb, dtype=torch.int32, device=DEV)
    at = 0
    for b, s in enumerate(lens):
        p = -(-s // page)
        table[b, :p] = order[at:at + p]
        at += p
    total = sum(qs)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    scale = torch.exp(torch.empty(1, hq, 1, device=DEV).uniform_(math.log(0.5), math.log(3.0), generator=gen))
    q = (torch.randn(total, hq, 128, generator=gen, device=DEV) * scale).to(dt)
    cu = [0]
    for x in qs:
        cu.append(cu[-1] + x)
    parents = None
    if case["tree"]:
        # drafts in breadth-first order, as a drafting step adds levels: a parent comes before its children
        parents = _i32([r.randint(max(-1, i // 3 - 3), i - 1) if i else -1 for x in qs for i in range(x)])
    signs = dense = None
    if case["rot"] == "signed_hadamard":
        signs = torch.where(torch.rand(hkv, 128, generator=gen, device=DEV) < 0.5, -1.0, 1.0)
    elif case["rot"] == "dense":
        dense = torch.linalg.qr(torch.randn(hkv, 128, 128, generator=gen, device=DEV, dtype=torch.float64))[0].float().contiguous()
    return dict(case=case, lens=_i32(lens), max_len=max(lens), cu=_i32(cu), max_q=max(qs), total=total, q=q,
                parents=parents, table=table, pool=_quantized_pool(gen, blocks, hkv, page), blocks=blocks,
                signs=signs, dense=dense)


def _prepare_plan(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    old, new = _plan_lens(case)
    page, n = case["page"], case["seqs"]
    pages = lambda x: -(-x // page)  # noqa: E731
    held = sum(pages(o) for o in old)
    taken = sum(max(0, pages(a) - pages(o)) for o, a in zip(old, new))
    blocks = held + taken + 1000
    mb = max(1, max(pages(max(o, a)) for o, a in zip(old, new)))
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    lens = torch.tensor([pages(o) for o in old], device=DEV)
    first = torch.cumsum(lens, 0) - lens
    col = torch.arange(mb, device=DEV)[None]
    table = torch.where(col < lens[:, None], order[(first[:, None] + col).clamp(max=blocks - 1)], torch.zeros_like(order[:1]))
    free = blocks - held
    start = random.Random(seed).randrange(blocks)  # the ring has turned for a while
    head = 5 * blocks + start
    ring = torch.full((blocks,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free, device=DEV)) % blocks] = order[held:]
    max_new = sum(max(0, a - o) for o, a in zip(old, new)) + 7
    return dict(case=case, old=_i32(old), new=_i32(new), table=table.contiguous(), ring=ring, blocks=blocks,
                ring_in=torch.tensor([head, head + free], dtype=torch.int64, device=DEV),
                ring_out=torch.empty(2, dtype=torch.int64, device=DEV),
                cu=torch.empty(n + 1, dtype=torch.int32, device=DEV),
                slots=torch.empty(max_new, dtype=torch.int64, device=DEV), max_new=max_new)


def _prepare_commit(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = random.Random(seed)
    n, page, nodes, hkv = case["seqs"], case["page"], case["nodes"], case["hkv"]
    per = -(-nodes // page) + 1
    blocks = n * per
    order = torch.randperm(blocks, generator=gen, device=DEV)
    cu, slot_b, slot_i, base, acc, n_acc = [0], [], [], [], [], []
    for b, (x, k) in enumerate(zip(*_commit_shape(case))):
        base.append(r.randrange(page))
        cu.append(cu[-1] + x)
        slot_b += [b] * x
        slot_i += [base[b] + i for i in range(x)]
        path = sorted(r.sample(range(x), k))
        acc.append(path + [-1] * (case["depth"] - k))
        n_acc.append(k)
    sb, si = torch.tensor(slot_b, device=DEV), torch.tensor(slot_i, device=DEV)
    slots = order[sb * per + si // page] * page + si % page
    lens = [16 * page + base[b] + cu[b + 1] - cu[b] for b in range(n)]
    pool = torch.randint(0, 256, (blocks, hkv, 72 * page), generator=gen, device=DEV, dtype=torch.uint8)
    return dict(case=case, cu=_i32(cu), accepted=_i32(acc), n_accepted=_i32(n_acc), slots=slots, lens=_i32(lens),
                new_lens=torch.empty(n, dtype=torch.int32, device=DEV), pool=pool, blocks=blocks)


def prepare(case, seed):
    make = {"tree": _prepare_attn, "cross": _prepare_attn, "plan": _prepare_plan, "commit": _prepare_commit}
    return make[case["kind"]](case, seed)


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------
def _hadamard():
    h = torch.ones(1, 1, device=DEV)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(128.0)


def _plain_cache(rec, page, role):
    """Records [B, pages, H, 72 P] -> dequantized fp32 [B, H, tokens, 128] of the keys (0) or the values (1)."""
    b, n, h, _ = rec.shape
    codes = rec[..., 32 * page * role:32 * page * (role + 1)].reshape(b, n, h, page, 32, 1)
    codes = (codes >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=DEV)) & 3
    meta = rec[..., 64 * page + 4 * page * role:64 * page + 4 * page * (role + 1)].contiguous().view(torch.float16)
    meta = meta.reshape(b, n, h, page, 2).float()
    x = codes.reshape(b, n, h, page, 128).float() * meta[..., :1] + meta[..., 1:]
    return x.transpose(1, 2).reshape(b, h, n * page, 128)


def _plain_attn(st):
    case = st["case"]
    page, hq, hkv = case["page"], case["hq"], case["hkv"]
    g = hq // hkv
    q = st["q"].float().view(st["total"], hkv, g, 128)
    if st["signs"] is not None:
        q = (q * st["signs"][None, :, None, :]) @ _hadamard()
    elif st["dense"] is not None:
        q = torch.einsum("thgc,hcd->thgd", q, st["dense"])
    lens, cu = st["lens"].long(), st["cu"].long()
    n, mq, ms = case["seqs"], st["max_q"], st["table"].shape[1] * page
    nq = cu[1:] - cu[:-1]
    t = torch.arange(st["total"], device=DEV)
    b_of = torch.searchsorted(cu[1:], t, right=True)
    i_of = t - cu[b_of]
    qp = torch.zeros(n, hkv, mq, g, 128, device=DEV)
    qp[b_of, :, i_of] = q
    rec = st["pool"][st["table"].long()]
    scores = qp.view(n, hkv, mq * g, 128) @ _plain_cache(rec, page, 0).transpose(2, 3)
    scores *= 1.0 / math.sqrt(128.0)
    s = torch.arange(ms, device=DEV)
    see = (s < lens[:, None])[:, None, :].expand(n, mq, ms)
    if case["kind"] == "tree":
        node = s - (lens - nq)[:, None]  # draft index of a position, negative before the drafts
        if st["parents"] is None:
            anc = torch.ones(mq, mq, device=DEV).tril().bool().expand(n, mq, mq)
        else:
            link = torch.eye(mq, device=DEV).repeat(n, 1, 1)
            par = st["parents"].long()
            has = par >= 0
            link[b_of[has], i_of[has], par[has]] = 1.0
            for _ in range(max(1, (mq - 1).bit_length())):  # ancestors by repeated squaring
                link = ((link @ link) > 0).float()
            anc = link > 0
        at = node.clamp(0, mq - 1)[:, None, :].expand(n, mq, ms)
        see = see & ((node < 0)[:, None, :] | torch.gather(anc, 2, at))
    see = see[:, None, :, None, :]
    scores = scores.view(n, hkv, mq, g, ms).masked_fill_(~see, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3.0e38)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(n, hkv, mq * g, ms) @ _plain_cache(rec, page, 1)
    o = o.view(n, hkv, mq, g, 128) / total.clamp(min=1e-30)
    return {"o": o[b_of, :, i_of].reshape(st["total"], hq, 128)}


def _plain_plan(st):
    page, nb = st["case"]["page"], st["blocks"]
    old, new = st["old"].long(), st["new"].long()
    p0, p1 = (old + page - 1) // page, (new + page - 1) // page
    grow, take, give = (new - old).clamp(min=0), (p1 - p0).clamp(min=0), (p0 - p1).clamp(min=0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(grow, 0)])
    take_at, give_at = torch.cumsum(take, 0) - take, torch.cumsum(give, 0) - give
    head, tail = st["ring_in"][0], st["ring_in"][1]
    table, ring = st["table"], st["ring"]
    seq = torch.arange(old.numel(), device=DEV)
    # pages given back go to the tail, in (sequence, page) order
    b = torch.repeat_interleave(seq, give)
    k = torch.arange(b.numel(), device=DEV)
    back = table[b, p1[b] + k - give_at[b]]
    # pages taken come from the head
    tb = torch.repeat_interleave(seq, take)
    tk = torch.arange(tb.numel(), device=DEV)
    table[tb, p0[tb] + tk - take_at[tb]] = ring[(head + tk) % nb]
    ring[(tail + k) % nb] = back
    # slots of the new tokens
    t = torch.repeat_interleave(seq, grow)
    pos = old[t] + torch.arange(t.numel(), device=DEV) - cu[t]
    slots = torch.full((st["max_new"],), -1, dtype=torch.int64, device=DEV)
    slots[:t.numel()] = table[t, pos // page].long() * page + pos % page
    return {"table": table, "ring": ring, "counters": torch.stack([head + take.sum(), tail + give.sum()]),
            "cu": cu.to(torch.int32), "slots": slots}


def _plain_commit(st):
    page = st["case"]["page"]
    cu, acc, n_acc, slots = st["cu"].long(), st["accepted"].long(), st["n_accepted"].long(), st["slots"]
    keep = torch.arange(acc.shape[1], device=DEV)[None] < n_acc[:, None]
    b, i = torch.nonzero(keep, as_tuple=True)
    src, dst = slots[cu[b] + acc[b, i]], slots[cu[b] + i]
    nb, h = st["pool"].shape[:2]
    codes = st["pool"][:, :, :64 * page].view(nb, h, 2, page, 32)
    meta = st["pool"][:, :, 64 * page:].view(nb, h, 2, page, 4)
    for part in (codes, meta):
        part[dst // page, :, :, dst % page] = part[src // page, :, :, src % page]
    new_lens = st["lens"] - (st["cu"][1:] - st["cu"][:-1]) + st["n_accepted"]
    return {"pool": st["pool"], "new_lens": new_lens}


# ---------------------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------------------
def _own_attn(st):
    import int2_kv_cache_gb300 as kvq
    case = st["case"]
    if "ws" not in st:  # what a serving program keeps: the layout, the rotation, the workspace, the output buffer
        st["lay"] = kvq.make_layout(case["page"], case["hkv"], case["hq"], st["blocks"], st["table"].shape[1])
        st["rot"] = kvq.DeviceRot(case["rot"], signs=st["signs"], dense=st["dense"])
        size = kvq.kvq_query_block_workspace_size(st["lay"], case["seqs"], st["total"], st["max_q"], st["max_len"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        st["o"] = torch.empty(st["total"], case["hq"], 128, device=DEV)
    if case["kind"] == "tree":
        kvq.kvq_tree_attention(st["lay"], st["q"], st["cu"], st["max_q"], st["parents"], st["lens"], st["max_len"],
                               st["table"], st["rot"], st["pool"], st["ws"], st["o"])
    else:
        kvq.kvq_cross_attention(st["lay"], st["q"], st["cu"], st["max_q"], st["lens"], st["max_len"], st["table"],
                                st["rot"], st["pool"], st["ws"], st["o"])
    return {"o": st["o"]}


def _own_plan(st):
    import int2_kv_cache_gb300 as kvq
    if "ws" not in st:
        st["lay"] = kvq.make_layout(st["case"]["page"], 1, 1, st["blocks"], st["table"].shape[1])
        st["ws"] = torch.empty(kvq.kvq_plan_workspace_size(st["case"]["seqs"]), dtype=torch.uint8, device=DEV)
    kvq.kvq_plan_pages(st["lay"], st["old"], st["new"], st["table"], st["ring"], st["ring_in"], st["ring_out"],
                       st["cu"], st["slots"], st["ws"])
    return {"table": st["table"], "ring": st["ring"], "counters": st["ring_out"], "cu": st["cu"], "slots": st["slots"]}


def _own_commit(st):
    import int2_kv_cache_gb300 as kvq
    if "lay" not in st:
        hkv = st["case"]["hkv"]
        st["lay"] = kvq.make_layout(st["case"]["page"], hkv, hkv, st["blocks"], 1)
    kvq.kvq_tree_commit(st["lay"], st["cu"], st["accepted"], st["n_accepted"], st["slots"], st["lens"],
                        st["new_lens"], st["pool"])
    return {"pool": st["pool"], "new_lens": st["new_lens"]}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"tree": _own_attn, "cross": _own_attn, "plan": _own_plan, "commit": _own_commit}[kind](state)
    return {"tree": _plain_attn, "cross": _plain_attn, "plan": _plain_plan, "commit": _plain_commit}[kind](state)


# ---------------------------------------------------------------------------------------------------------
# the least work, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------
def work(case):
    if case["kind"] in ("tree", "cross"):
        lens, qs = _attn_lens(case)
        hq, hkv, page = case["hq"], case["hkv"], case["page"]
        if case["kind"] == "cross":
            pairs = sum(s * n for s, n in zip(lens, qs))
        elif case["tree"]:
            pairs = sum((s - n) * n for s, n in zip(lens, qs))  # and the few ancestors
        else:
            pairs = sum((s - n) * n + n * (n + 1) // 2 for s, n in zip(lens, qs))
        total = sum(qs)
        size = 2 if case["dtype"] == "bf16" else 4
        dense = case["rot"] == "dense"
        by = sum(lens) * hkv * 72 + total * hq * 128 * (size + 4) + sum(-(-s // page) for s in lens) * 4 + 8 * len(lens)
        return {"bytes": by + (hkv * 65536 if dense else 0), "flops": 512 * pairs * hq + (total * hq * 32768 if dense else 0)}
    if case["kind"] == "plan":
        old, new = _plan_lens(case)
        page = case["page"]
        grow = sum(max(0, a - o) for o, a in zip(old, new))
        moved = sum(abs(-(-a // page) + -o // page) for o, a in zip(old, new))
        return {"bytes": 12 * len(old) + 8 * moved + 8 * grow, "flops": 0}
    kept = sum(_commit_shape(case)[1])
    return {"bytes": kept * (case["hkv"] * 144 + 20) + 16 * case["seqs"], "flops": 0}


def exact(case, seed):
    if case["kind"] not in ("tree", "cross"):
        return None  # whole numbers: they have to be equal
    st = prepare(case, seed)
    lens, qs = _attn_lens(case)
    page, hq, hkv = case["page"], case["hq"], case["hkv"]
    g = hq // hkv
    q = st["q"].double()
    if st["signs"] is not None:
        i = np.arange(128)
        parity = np.array([[bin(a & b).count("1") & 1 for a in i] for b in i])
        mats = torch.tensor((1.0 - 2.0 * parity) / np.sqrt(128.0), device=DEV)[None] * st["signs"].double()[:, :, None]
    elif st["dense"] is not None:
        mats = st["dense"].double()
    else:
        mats = torch.eye(128, dtype=torch.float64, device=DEV)[None].repeat(hkv, 1, 1)
    out = torch.zeros(st["total"], hq, 128, dtype=torch.float64, device=DEV)
    par = st["parents"].tolist() if st["parents"] is not None else None
    at = 0
    for b, (s, n) in enumerate(zip(lens, qs)):
        first, at = at, at + n
        if s == 0:
            continue
        pages = st["table"][b, :-(-s // page)].long()
        seen = np.ones((n, s), dtype=bool)
        if case["kind"] == "tree" and par is None:
            seen[:, s - n:] = np.arange(n)[:, None] >= np.arange(n)[None]
        elif case["kind"] == "tree":
            seen[:, s - n:] = False
            for i in range(n):
                j = i
                while j >= 0:
                    seen[i, s - n + j] = True
                    j = par[first + j]
        seen = torch.from_numpy(seen).to(DEV)
        for h in range(hkv):
            rec = st["pool"][pages, h]
            kv = []
            for role in (0, 1):
                byte = rec[:, 32 * page * role:32 * page * (role + 1)].reshape(-1, 32).long()
                c = torch.stack([torch.remainder(torch.div(byte, 4 ** f, rounding_mode="floor"), 4) for f in range(4)], -1)
                m = rec[:, (64 + 4 * role) * page:(68 + 4 * role) * page].contiguous().view(torch.float16).double().view(-1, 2)
                kv.append((m[:, 1:] + m[:, :1] * c.reshape(-1, 128).double())[:s])
            for j in range(h * g, (h + 1) * g):
                a = (q[first:at, j] @ mats[h]) @ kv[0].T / np.sqrt(128.0)
                out[first:at, j] = torch.softmax(a.masked_fill(~seen, -math.inf), -1) @ kv[1]
    return {"o": out}
