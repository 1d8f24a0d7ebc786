"""Operators that serve branching, multi-axis sequences over the paged shared KV cache: what is measured of them.

* ``chunk``: causal, windowed or tree-masked attention of a chunk of new tokens over a cache (yocopp_chunk_attn);
* ``rope``: the residual composition with rotary positions of one to four axes, appended to the cache, and the
  queries rotated with it (yocopp_rope_compose_append);
* ``resize``, ``fork``, ``compact``: pages of a cache given, taken back, shared, copied and moved together
  (yocopp_pages_resize, yocopp_pages_fork, yocopp_pages_compact).

``run`` computes an operator in its plain form (elementary torch operations, fp32 or fp64) where ``own`` is false,
and calls this repository's library where it is true.  ``exact`` evaluates the definitions in fp64 with plain loops.
Sequence lengths are a function of the case alone; values, block numbers and orders come from the seed.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LAM = 35.0
ALPHA = (0.04, 1.0 / 35 + 0.01, -0.03, 1.0 / 35 + 0.02)


# ----------------------------------------------------------------- cases
def listed():
    return [
        # speculative decoding of a small batch: trees of 16 draft tokens verified over about 1000 cached ones
        dict(name="chunk_tree_verify", op="chunk", batch=8, rows=16, context=1024, heads=32, kv_heads=8, dim=128,
             dtype="bf16", block=16, window=0, tree=True),
        # several new tokens of each of 32 long conversations (the benchmark's 32 x 8192), ragged: memory-bound
        dict(name="chunk_extend_32x8192", op="chunk", batch=32, rows=8, context=8192, heads=32, kv_heads=8, dim=128,
             dtype="bf16", block=64, window=0, tree=False),
        # one chunk of a long prompt prefilled over what is cached already: compute-bound
        dict(name="chunk_prefill_32768", op="chunk", batch=1, rows=2048, context=32768, heads=32, kv_heads=8, dim=128,
             dtype="bf16", block=64, window=0, tree=False),
        # a small fp32 model with a sliding window, odd sizes, contiguous cache
        dict(name="chunk_window_f32_d64", op="chunk", batch=5, rows=77, context=4099, heads=12, kv_heads=4, dim=64,
             dtype="f32", block=0, window=1000, tree=False),
        # one decode step of 32 sequences of a video model: three axes, one token each
        dict(name="rope_decode_32", op="rope", batch=32, rows=1, axes=3, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", block=64),
        # prompts of images and text, ragged, up to 4096 tokens each
        dict(name="rope_prefill_8x4096", op="rope", batch=8, rows=4096, axes=3, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, dtype="bf16", block=64),
        # a scheduler's step on a small server: rows grow, shrink and end; 12 cached layers
        dict(name="resize_8", op="resize", batch=8, row_blocks=16, block=64, pool=160, layers=12, kv_heads=8, dim=128,
             dtype="bf16"),
        # the same on a server of 256 rows with pages of 16 tokens, 65536 pages
        dict(name="resize_256", op="resize", batch=256, row_blocks=256, block=16, pool=65536, layers=1, kv_heads=2,
             dim=64, dtype="bf16"),
        # one prompt sampled 8 times: full pages shared, the last one copied in 12 layers
        dict(name="fork_share_8", op="fork", batch=16, forks=8, row_blocks=16, block=64, pool=160, layers=12,
             kv_heads=8, dim=128, dtype="bf16", deep=False),
        # four conversations of up to 8192 tokens copied whole
        dict(name="fork_deep_4x8192", op="fork", batch=8, forks=4, row_blocks=128, block=64, pool=1100, layers=4,
             kv_heads=8, dim=128, dtype="bf16", deep=True),
        # a small pool's holes closed
        dict(name="compact_256", op="compact", batch=16, row_blocks=12, block=64, pool=256, layers=2, kv_heads=8,
             dim=128, dtype="bf16", moves=20),
        # a large pool halved after most of its rows ended
        dict(name="compact_4096", op="compact", batch=64, row_blocks=48, block=64, pool=4096, layers=2, kv_heads=8,
             dim=128, dtype="bf16", moves=1400),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rope", "rope", "resize", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "chunk":
        dim, kv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
        tree = rng.random() < 0.3
        rows = _log(rng, 1, 64 if tree else 2048)
        context = _log(rng, 16, 32768)
        # scores of the padded plain form stay below the largest listed case's, and the cache below 1 GB
        most = 32 * 2048 * 34816 // (8 if dtype == "f32" else 1)
        batch = max(1, min(_log(rng, 1, 64), most // (heads * rows * (context + rows)),
                           (1 << 28) // (kv * dim * (context + rows))))
        while heads * rows * (context + rows) > most:
            context = context // 2 + 3
        window = 0 if tree or rng.random() < 0.6 else _log(rng, 1, context)
        return dict(op=op, batch=batch, rows=rows, context=context, heads=heads, kv_heads=kv, dim=dim, dtype=dtype,
                    block=rng.choice([0, 16, 32, 64, 128, 256]), window=window, tree=tree)
    if op == "rope":
        dim, kv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
        rows = _log(rng, 1, 4096)
        batch = max(1, min(_log(rng, 1, 64), 8 * 4096 // (rows * (2 if dtype == "f32" else 1))))
        rotary = rng.choice([dim, dim, dim // 2, dim // 2 + 6])
        return dict(op=op, batch=batch, rows=rows, axes=rng.choice([1, 2, 3, 4]), heads=kv * rng.choice([1, 2, 3, 4]),
                    kv_heads=kv, dim=dim, rotary=rotary, interleaved=rng.random() < 0.5, dtype=dtype,
                    block=rng.choice([0, 16, 32, 64, 128, 256]))
    block, kv, dim = rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    layers = rng.choice([1, 2, 4, 12])
    block_bytes = block * kv * dim * 2 * layers * (2 if dtype == "bf16" else 4)
    batch = _log(rng, 2, 256)
    row_blocks = max(2, min(_log(rng, 2, 512), (1 << 30) // (block_bytes * batch)))
    batch = max(2, min(batch, (1 << 30) // (block_bytes * row_blocks)))
    base = dict(op=op, batch=batch, row_blocks=row_blocks, block=block, layers=layers, kv_heads=kv, dim=dim,
                dtype=dtype)
    if op == "resize":
        return dict(base, pool=batch * row_blocks + rng.randrange(1, 40))
    if op == "fork":
        forks = max(1, batch // rng.choice([2, 3, 4]))
        return dict(base, forks=forks, pool=(batch + forks) * row_blocks + rng.randrange(1, 40),
                    deep=rng.random() < 0.3)
    pool = batch * row_blocks + rng.randrange(1, 400)
    return dict(base, pool=pool, moves=rng.randrange(0, _compact_live(base) // 2 + 1))


def _rng(case, what):
    keys = sorted(k for k in case if k != "name")
    return random.Random(what + "|" + "|".join("%s=%s" % (k, case[k]) for k in keys))


def _up(a, b):
    return -(-a // b)


def _chunk_lens(case):
    """(position of the first row, rows) of each sequence."""
    r = _rng(case, "chunk")
    ctx = [case["context"]] + [r.randint(max(0, case["context"] // 2), case["context"]) for _ in range(case["batch"] - 1)]
    rows = [case["rows"]] + [r.randint(max(1, case["rows"] // 2), case["rows"]) for _ in range(case["batch"] - 1)]
    return ctx, rows


def _rope_lens(case):
    r = _rng(case, "rope")
    rows = [case["rows"]] + [r.randint(max(1, case["rows"] // 2), case["rows"]) for _ in range(case["batch"] - 1)]
    return [r.randint(0, 40) for _ in rows], rows


def _capacity(case, most):
    return _up(most, case["block"]) * case["block"] if case["block"] else most


def _resize_plan(case):
    """Lengths before (in blocks) and after (in tokens) of each row, and the prefix (in blocks) that each odd row
    shares with the row before it.  The pool always has room: fresh blocks are no more than released or spare ones."""
    r, M, bs = _rng(case, "resize"), case["row_blocks"], case["block"]
    have = [r.randint(1, max(1, M - 1)) for _ in range(case["batch"])]
    share = [min(have[i - 1], have[i]) // 2 if i % 2 else 0 for i in range(case["batch"])]
    lens = []
    for i in range(case["batch"]):
        kind = r.random()
        if kind < 0.25:                                     # the sequence has ended
            lens.append(0)
        elif kind < 0.5:                                    # drafts rolled back, half of them into a shared page
            both = share[i] if i % 2 else share[i + 1] if i + 1 < case["batch"] else 0
            into = both if both and r.random() < 0.5 else 0
            lens.append(r.randint((into - 1) * bs + 1, into * bs - 1) if into else r.randint(1, have[i] * bs))
        else:                                               # grows by up to two pages
            lens.append(min(M * bs, have[i] * bs + r.randint(1, 2 * bs)))
    return have, share, lens


def _fork_plan(case):
    """Source row and length of each fork; forks[i] goes to row batch - forks + i."""
    r = _rng(case, "fork")
    src_rows = case["batch"] - case["forks"]
    most = case["row_blocks"] * case["block"]
    held = [most - r.randint(0, most // 2) for _ in range(src_rows)]
    src = [i % max(1, src_rows) if case["deep"] else r.randrange(src_rows) for i in range(case["forks"])]
    return held, src, [held[s] - r.randint(0, held[s] // 4) for s in src]


def _compact_held(case):
    r = _rng({k: v for k, v in case.items() if k not in ("pool", "moves")}, "compact")
    return [r.randint(0, case["row_blocks"]) for _ in range(case["batch"])]


def _compact_live(case):
    return sum(_compact_held(case))


# ----------------------------------------------------------------- inputs
class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cum(x):
    out = [0]
    for v in x:
        out.append(out[-1] + v)
    return out


def _prepare_chunk(c, seed, s):
    g, dt = _gen(seed), DT[c["dtype"]]
    ctx, rows = _chunk_lens(c)
    s.cap = _capacity(c, max(a + b for a, b in zip(ctx, rows)))
    s.total = sum(rows)
    if c["block"]:
        per = s.cap // c["block"]
        s.table = torch.randperm(c["batch"] * per, generator=g, device="cuda").int().reshape(c["batch"], per)
        shape = (c["batch"] * per, c["kv_heads"], c["block"], c["dim"])
    else:
        s.table, shape = None, (c["batch"], c["kv_heads"], s.cap, c["dim"])
    s.k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    s.v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    s.q = torch.randn((s.total, c["heads"], c["dim"]), generator=g, device="cuda", dtype=dt) * 2
    s.pos, s.cu = _i32(ctx), _i32(_cum(rows))
    s.max_q = max(rows)
    s.tree = None
    if c["tree"]:
        # a node sees the cached tokens, itself and its ancestors: node j's parent is one of the nodes before it
        r, masks = random.Random(seed), []
        for n in rows:
            m = []
            for j in range(n):
                m.append((1 << j) | (m[r.randrange(max(0, j - 4), j)] if j else 0))
            masks += [x - (1 << 64) if x >> 63 else x for x in m]
        s.tree = torch.tensor(masks, dtype=torch.int64, device="cuda")
    s.out = torch.empty_like(s.q)
    if own:
        import decode_attention_yocopp_b200 as y
        s.cache = y.make_cache(s.k, s.v, s.table)
        s.ws = y.alloc_chunk_workspace(s.cache, c["heads"])


def _sections(c):
    pairs, axes = c["rotary"] // 2, c["axes"]
    return [pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes)]


def _prepare_rope(c, seed, s):
    g, dt = _gen(seed), DT[c["dtype"]]
    start, rows = _rope_lens(c)
    s.total, s.cap = sum(rows), _capacity(c, max(a + b for a, b in zip(start, rows)))
    if c["block"]:
        per = s.cap // c["block"]
        s.table = torch.randperm(c["batch"] * per, generator=g, device="cuda").int().reshape(c["batch"], per)
        shape = (c["batch"] * per, c["kv_heads"], c["block"], c["dim"])
    else:
        s.table, shape = None, (c["batch"], c["kv_heads"], s.cap, c["dim"])
    s.k, s.v = (torch.zeros(shape, device="cuda", dtype=dt) for _ in range(2))
    s.raw = [torch.randn((s.total, c["kv_heads"], c["dim"]), generator=g, device="cuda", dtype=dt) for _ in range(4)]
    s.q = torch.randn((s.total, c["heads"], c["dim"]), generator=g, device="cuda", dtype=dt)
    s.q_out = torch.empty_like(s.q)
    # far positions on the time axis, as in a long video; rows and columns of frames on the others
    s.positions = torch.randint(0, 1 << 20, (c["axes"], s.total), generator=g, device="cuda", dtype=torch.int32)
    if c["axes"] > 1:
        s.positions[1:] %= 1024
    s.pos, s.cu = _i32(start), _i32(_cum(rows))
    s.axis = torch.tensor([a for a, n in enumerate(_sections(c)) for _ in range(n)], device="cuda")
    s.inv = 10000.0 ** (-torch.arange(c["rotary"] // 2, dtype=torch.float64, device="cuda") * 2 / c["rotary"])
    if own:
        import decode_attention_yocopp_b200 as y
        s.cache = y.make_cache(s.k, s.v, s.table)
        s.rope = y.make_rope(c["rotary"], base=10000.0, sections=_sections(c), interleaved=c["interleaved"])


def _pool(c, g, s):
    s.pool = torch.randn((c["layers"], 2, c["pool"], c["kv_heads"], c["block"], c["dim"]), generator=g, device="cuda",
                         dtype=DT[c["dtype"]])


def _pages_state(c, s, rows, refs):
    """The page table and the reference counts in one buffer, as they stand before the step and as the step leaves
    them: a pass starts from the former, so that it can be made again."""
    B, M = c["batch"], c["row_blocks"]
    before = torch.full((B * M + c["pool"],), -1, dtype=torch.int32)
    for b, row in enumerate(rows):
        before[b * M: b * M + len(row)] = torch.tensor(row, dtype=torch.int32)
    before[B * M:] = torch.tensor(refs, dtype=torch.int32)
    s.before = before.cuda()
    s.now = s.before.clone()
    s.table, s.refs = s.now[: B * M].view(B, M), s.now[B * M:]
    s.rows = rows
    s.held = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        import decode_attention_yocopp_b200 as y
        s.caches = y.cache_list([y.make_cache(s.pool[i, 0], s.pool[i, 1], s.table) for i in range(c["layers"])])
        s.ws = y.alloc_pages_workspace(s.caches)


def _prepare_resize(c, seed, s):
    r = random.Random(seed)
    have, share, lens = _resize_plan(c)
    ids = list(range(c["pool"]))
    r.shuffle(ids)
    rows, refs = [], [0] * c["pool"]
    for b in range(c["batch"]):
        row = rows[b - 1][: share[b]] if share[b] else []
        while len(row) < have[b]:
            row.append(ids.pop())
        for x in row:
            refs[x] += 1
        rows.append(row)
    order = list(range(c["batch"]))
    r.shuffle(order)
    _pool(c, _gen(seed), s)
    _pages_state(c, s, rows, refs)
    s.order, s.lens_list = order, [lens[b] for b in order]
    s.seqs, s.lens = _i32(order), _i32(s.lens_list)


def _prepare_fork(c, seed, s):
    r = random.Random(seed)
    held, src, lens = _fork_plan(c)
    ids = list(range(c["pool"]))
    r.shuffle(ids)
    rows, refs = [], [0] * c["pool"]
    for n in held:
        rows.append([ids.pop() for _ in range(_up(n, c["block"]))])
        for x in rows[-1]:
            refs[x] = 1
    rows += [[] for _ in range(c["forks"])]
    dst = list(range(c["batch"] - c["forks"], c["batch"]))
    r.shuffle(dst)
    _pool(c, _gen(seed), s)
    _pages_state(c, s, rows, refs)
    s.src_list, s.dst_list, s.lens_list = src, dst, lens
    s.src, s.dst, s.lens = _i32(src), _i32(dst), _i32(lens)


def _prepare_compact(c, seed, s):
    r = random.Random(seed)
    held, live = _compact_held(c), _compact_live(c)
    moves = min(c["moves"], live, c["pool"] - live)
    low, high = list(range(live)), list(range(live, c["pool"]))
    r.shuffle(low)
    r.shuffle(high)
    ids = low[moves:] + high[:moves]
    r.shuffle(ids)
    rows, refs = [], [0] * c["pool"]
    for n in held:
        rows.append([ids.pop() for _ in range(n)])
        for x in rows[-1]:
            refs[x] = 1
    _pool(c, _gen(seed), s)
    _pages_state(c, s, rows, refs)
    s.live = torch.empty(1, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    s = State()
    s.case = case
    {"chunk": _prepare_chunk, "rope": _prepare_rope, "resize": _prepare_resize, "fork": _prepare_fork,
     "compact": _prepare_compact}[case["op"]](case, seed, s)
    return s


# ----------------------------------------------------------------- the plain forms
def _plain_chunk(s):
    c = s.case
    k, v = s.k, s.v
    if s.table is not None:
        t = s.table.long()
        k, v = (x[t].transpose(1, 2).reshape(c["batch"], c["kv_heads"], s.cap, c["dim"]) for x in (k, v))
    k, v = k.float(), v.float()
    B, n, H, G, d = c["batch"], s.max_q, c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    j = torch.arange(n, device="cuda")
    start, rows = s.cu[:-1].long(), (s.cu[1:] - s.cu[:-1]).long()
    real = j[None, :] < rows[:, None]                                        # [B, n]
    at = (start[:, None] + j[None, :]).clamp(max=s.total - 1)                # [B, n]
    q = s.q[at].float().reshape(B, n, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d)
    u = torch.arange(s.cap, device="cuda")
    p = s.pos.long()[:, None, None]
    mine = p + j[None, :, None]
    if s.tree is not None:
        bit = (u[None, None, :] - p).clamp(0, 63)
        see = (u < p) | ((s.tree[at][:, :, None] >> bit) & 1).bool() & (u - p < rows[:, None, None])
    else:
        see = u <= mine
        if c["window"]:
            see = see & (u > mine - c["window"])
    see = see & real[:, :, None]
    hide = ~see[:, None, :, None, :].expand(B, 1, n, G, s.cap).reshape(B, 1, n * G, s.cap)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).masked_fill_(hide, -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.reshape(B, H, n, G, d).permute(0, 2, 1, 3, 4).reshape(B * n, H * G, d)
    # rows of shorter chunks than the longest are padding: the k-th real one is the packed output's k-th
    place = torch.where(real, at, torch.full_like(at, s.total)).reshape(-1)
    out = torch.empty((s.total + 1, H * G, d), dtype=s.q.dtype, device="cuda")
    out[place] = o.to(s.q.dtype)
    return {"out": out[: s.total]}


def _rotate(x, cos, sin, rotary, interleaved):
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., : rotary // 2], x[..., rotary // 2: rotary])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((lo, hi), -1).flatten(-2) if interleaved else torch.cat((lo, hi), -1)
    return torch.cat((y, x[..., rotary:]), -1)


def _plain_rope(s):
    c = s.case
    a1, a2, b1, b2 = ALPHA
    angle = s.positions[s.axis].double().t() * s.inv                          # [total, pairs]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    K1, V1, Ki, Vi = (x.float() for x in s.raw)
    K = _rotate(LAM * (a1 * K1 + a2 * Ki), cos, sin, c["rotary"], c["interleaved"]).to(s.k.dtype)
    V = (LAM * (b1 * V1 + b2 * Vi)).to(s.v.dtype)
    t = torch.arange(s.total, device="cuda")
    b = torch.searchsorted(s.cu.long(), t, right=True) - 1
    at = s.pos.long()[b] + t - s.cu.long()[b]
    if s.table is not None:
        blk = s.table.long()[b, at // c["block"]]
        s.k[blk, :, at % c["block"]] = K
        s.v[blk, :, at % c["block"]] = V
    else:
        s.k[b, :, at] = K
        s.v[b, :, at] = V
    q = _rotate(s.q.float(), cos, sin, c["rotary"], c["interleaved"]).to(s.q.dtype)
    return {"k": s.k, "v": s.v, "q": q}


def _free_order(refs, most):
    """The numbers of the free blocks in ascending order, in the first places of a list of `most`."""
    free = refs == 0
    place = torch.where(free, torch.cumsum(free, 0) - 1, torch.full_like(refs, most, dtype=torch.int64)).clamp(max=most)
    order = torch.full((most + 1,), -1, dtype=torch.int64, device="cuda")
    order.scatter_(0, place, torch.arange(refs.numel(), device="cuda"))
    return order


def _copy_rows(pool, made, src, dst, rows):
    """Rows [0, rows[i]) of block src[i] to block dst[i] in every layer, where made[i]; the places of the others are
    filled up with the first such copy (or with nothing, where there is none)."""
    some, first = made.any(), made.int().argmax()
    src = torch.where(made, src, src[first])
    dst = torch.where(made, dst, torch.where(some, dst[first], src[first]))
    rows = torch.where(made, rows, torch.where(some, rows[first], torch.zeros_like(rows[0])))
    keep = torch.arange(pool.shape[4], device="cuda")[None, :] < rows[:, None]
    pool[:, :, dst] = torch.where(keep[None, None, :, None, :, None], pool[:, :, src], pool[:, :, dst])


def _plain_resize(s):
    c = s.case
    s.now.copy_(s.before)
    bs, M, n = c["block"], c["row_blocks"], s.seqs.numel()
    seq, lens = s.seqs.long(), s.lens.long()
    col = torch.arange(M, device="cuda")
    row = s.table[seq].long()
    have, need = (row >= 0).sum(1), (lens + bs - 1) // bs
    drop = (col >= need[:, None]) & (row >= 0)
    s.refs.index_add_(0, row.clamp(min=0).reshape(-1), -drop.reshape(-1).int())
    row = torch.where(drop, torch.full_like(row, -1), row)
    # a last page that is kept in part and still shared is replaced by a copy
    last = (need - 1).clamp(min=0)
    tail = row.gather(1, last[:, None])[:, 0]
    copy = (lens % bs > 0) & (need <= have) & (s.refs[tail.clamp(min=0)] > 1)
    want = (need - have).clamp(min=0) + copy.long()
    end = torch.cumsum(want, 0)
    base = end - want
    order = _free_order(s.refs, n * M + n)
    given = end <= (s.refs == 0).sum()
    grow = (col >= have[:, None]) & (col < need[:, None]) & given[:, None]
    fresh = order[(base[:, None] + col - have[:, None]).clamp(0, n * M)]
    row = torch.where(grow, fresh, row)
    s.refs.index_add_(0, torch.where(grow, fresh, torch.zeros_like(fresh)).reshape(-1), grow.reshape(-1).int())
    copy = copy & given
    new = torch.where(copy, order[base.clamp(0, n * M)], tail.clamp(min=0))
    s.refs.index_add_(0, tail.clamp(min=0), -copy.int())
    s.refs.index_add_(0, new, copy.int())
    _copy_rows(s.pool, copy, tail.clamp(min=0), new, lens % bs)
    row.scatter_(1, last[:, None], torch.where(copy, new, row.gather(1, last[:, None])[:, 0])[:, None])
    s.table[seq] = row.int()
    return {"table": s.table, "refs": s.refs, "held": torch.where(given | (want == 0), need, -1).int(), "pool": s.pool}


def _plain_fork(s):
    c = s.case
    s.now.copy_(s.before)
    bs, M, n = c["block"], c["row_blocks"], s.src.numel()
    src, dst, lens = s.src.long(), s.dst.long(), s.lens.long()
    col = torch.arange(M, device="cuda")
    old = s.table[src].long()
    need, full = (lens + bs - 1) // bs, lens // bs
    if c["deep"]:
        full = torch.zeros_like(full)
    shared, own_page = col < full[:, None], (col >= full[:, None]) & (col < need[:, None])
    want = need - full
    end = torch.cumsum(want, 0)
    order = _free_order(s.refs, n * M + n)
    given = (end <= (s.refs == 0).sum())[:, None]
    fresh = order[((end - want)[:, None] + col - full[:, None]).clamp(0, n * M)]
    row = torch.where(shared & given, old, torch.where(own_page & given, fresh, torch.full_like(old, -1)))
    s.refs.index_add_(0, row.clamp(min=0).reshape(-1), (row >= 0).reshape(-1).int())
    made = (own_page & given).reshape(-1)
    at = old.clamp(min=0).reshape(-1)
    tokens = (lens[:, None] - col * bs).clamp(0, bs).reshape(-1)
    fresh = fresh.reshape(-1)
    if c["deep"]:
        _copy_rows(s.pool, made, at, fresh, tokens)
    else:  # at most the last page of each row
        pick = torch.arange(n, device="cuda") * M + (need - 1).clamp(min=0)
        _copy_rows(s.pool, made[pick], at[pick], fresh[pick], tokens[pick])
    s.table[dst] = row.int()
    return {"table": s.table, "refs": s.refs, "held": torch.where(given[:, 0] | (want == 0), need, -1).int(), "pool": s.pool}


def _plain_compact(s):
    c = s.case
    s.now.copy_(s.before)
    used = s.refs > 0
    live = used.sum()
    ids = torch.arange(c["pool"], device="cuda")
    hole, mover = ~used & (ids < live), used & (ids >= live)
    # the k-th used block past the end goes to the k-th hole before it
    end = torch.full((c["pool"] + 1,), c["pool"], dtype=torch.int64, device="cuda")
    holes = end.clone().scatter_(0, torch.where(hole, torch.cumsum(hole, 0) - 1, end[:1]), ids)
    to = torch.where(mover, holes[(torch.cumsum(mover, 0) - 1).clamp(min=0)], ids)
    _move(s.pool, mover, to)
    row = s.table.long()
    s.table.copy_(torch.where(row >= 0, to[row.clamp(min=0)], row).int())
    refs = torch.zeros_like(s.refs).scatter_add_(0, to, torch.where(used, s.refs, torch.zeros_like(s.refs)))
    s.refs.copy_(refs)
    return {"table": s.table, "refs": s.refs, "live": live.int().reshape(1), "pool": s.pool}


def _move(pool, mover, to):
    src = mover.nonzero()[:, 0]
    pool[:, :, to[src]] = pool[:, :, src]


# ----------------------------------------------------------------- the library's calls
def _own_chunk(s):
    import decode_attention_yocopp_b200 as y
    c = s.case
    y.yocopp_chunk_attn(s.q, s.cache, s.out, s.ws, pos=s.pos, cu_q=s.cu, max_q=s.max_q, tree_mask=s.tree,
                        window=c["window"])
    return {"out": s.out}


def _own_rope(s):
    import decode_attention_yocopp_b200 as y
    y.yocopp_rope_compose_append(*s.raw, ALPHA, LAM, s.rope, s.positions, s.cache, s.pos, q=s.q, q_out=s.q_out,
                                 cu_new=s.cu)
    return {"k": s.k, "v": s.v, "q": s.q_out}


def _own_resize(s):
    import decode_attention_yocopp_b200 as y
    s.now.copy_(s.before)
    held = s.held[: s.seqs.numel()]
    y.yocopp_pages_resize(s.caches, s.refs, s.seqs, s.lens, held, s.ws)
    return {"table": s.table, "refs": s.refs, "held": held, "pool": s.pool}


def _own_fork(s):
    import decode_attention_yocopp_b200 as y
    s.now.copy_(s.before)
    held = s.held[: s.src.numel()]
    y.yocopp_pages_fork(s.caches, s.refs, s.src, s.dst, s.lens, held, s.ws, deep=s.case["deep"])
    return {"table": s.table, "refs": s.refs, "held": held, "pool": s.pool}


def _own_compact(s):
    import decode_attention_yocopp_b200 as y
    s.now.copy_(s.before)
    y.yocopp_pages_compact(s.caches, s.refs, s.live, s.ws)
    return {"table": s.table, "refs": s.refs, "live": s.live, "pool": s.pool}


def run(state):
    op = state.case["op"]
    if own:
        return {"chunk": _own_chunk, "rope": _own_rope, "resize": _own_resize, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"chunk": _plain_chunk, "rope": _plain_rope, "resize": _plain_resize, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# ----------------------------------------------------------------- the least that a pass reads, writes and computes
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "chunk":
        ctx, rows = _chunk_lens(c)
        seen = keys = 0
        for p, n in zip(ctx, rows):
            if c["window"]:
                seen += sum(min(p + j + 1, c["window"]) for j in range(n))
                keys += min(p + n, c["window"] + n - 1)
            elif c["tree"]:
                seen, keys = seen + n * (p + 1 + n // 2), keys + p + n
            else:
                seen, keys = seen + n * p + n * (n + 1) // 2, keys + p + n
        io = 2 * sum(rows) * c["heads"] * c["dim"] * e + (8 * sum(rows) if c["tree"] else 0)
        return {"bytes": 2 * keys * c["kv_heads"] * c["dim"] * e + io, "flops": 4 * seen * c["heads"] * c["dim"]}
    if c["op"] == "rope":
        t = sum(_rope_lens(c)[1])
        return {"bytes": t * (c["dim"] * e * (6 * c["kv_heads"] + 2 * c["heads"]) + 4 * c["axes"]),
                "flops": t * c["dim"] * (9 * c["kv_heads"] + 3 * c["heads"])}
    plane = 2 * c["layers"] * c["kv_heads"] * c["dim"] * e          # bytes of one token in every layer
    ints = 4 * c["pool"]                                             # the reference counts, read once
    if c["op"] == "resize":
        have, share, lens = _resize_plan(c)
        bs, moved, tokens = c["block"], 0, 0
        left = [min(have[b], _up(lens[b], bs)) for b in range(c["batch"])]
        for b, n in enumerate(lens):
            need = _up(n, bs)
            moved += abs(need - have[b])
            other = b - 1 if b % 2 else b + 1
            both = share[max(b, other)] if other < c["batch"] else 0
            if n % bs and need <= have[b] and need <= both and need <= left[other]:
                tokens += n % bs
        return {"bytes": 2 * tokens * plane + ints + 16 * moved + 12 * len(lens), "flops": 0}
    if c["op"] == "fork":
        _, _, lens = _fork_plan(c)
        tokens = sum(lens) if c["deep"] else sum(n % c["block"] for n in lens)
        return {"bytes": 2 * tokens * plane + ints + 16 * sum(_up(n, c["block"]) for n in lens), "flops": 0}
    live = _compact_live(c)
    moves = min(c["moves"], live, c["pool"] - live)
    return {"bytes": 2 * moves * c["block"] * plane + ints + 8 * moves + 8 * live, "flops": 0}


# ----------------------------------------------------------------- the definitions in fp64
def _exact_chunk(c, s):
    ctx, rows = _chunk_lens(c)
    G, first, out = c["heads"] // c["kv_heads"], 0, torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    for b, (p, n) in enumerate(zip(ctx, rows)):
        T = p + n
        if s.table is None:
            keys, vals = s.k[b, :, :T], s.v[b, :, :T]
        else:
            blocks = s.table[b, : _up(T, c["block"])].tolist()
            keys, vals = (torch.cat([x[i] for i in blocks], 1)[:, :T] for x in (s.k, s.v))
        hidden = torch.zeros((n, T), dtype=torch.bool, device="cuda")
        if c["tree"]:
            bits = s.tree[first: first + n].tolist()
            hidden[:, p:] = torch.tensor([[not (m >> i) & 1 for i in range(n)] for m in bits], device="cuda")
        else:
            own_place = torch.arange(p, T, device="cuda")[:, None] - torch.arange(T, device="cuda")[None, :]
            hidden = (own_place < 0) | ((own_place >= c["window"]) if c["window"] else False)
        for h in range(c["heads"]):
            x = s.q[first: first + n, h].double() @ keys[h // G].double().T / c["dim"] ** 0.5
            out[first: first + n, h] = torch.softmax(x.masked_fill(hidden, -math.inf), 1) @ vals[h // G].double()
        first += n
    return {"out": out}


def _exact_rope(c, s):
    start, rows = _rope_lens(c)
    a1, a2, b1, b2 = ALPHA
    k, v = s.k.double(), s.v.double()
    half = c["rotary"] // 2
    angle = torch.empty((s.total, half), dtype=torch.float64, device="cuda")
    pair = 0
    for a, n in enumerate(_sections(c)):
        for _ in range(n):
            angle[:, pair] = s.positions[a].double() / 10000.0 ** (2 * pair / c["rotary"])
            pair += 1
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def rotated(x):
        x = x.clone()
        if c["interleaved"]:
            lo, hi = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        else:
            lo, hi = x[..., :half], x[..., half: 2 * half]
        z = torch.complex(lo.clone(), hi.clone()) * turn
        lo.copy_(z.real)
        hi.copy_(z.imag)
        return x

    K1, V1, Ki, Vi = (x.double() for x in s.raw)
    K, V = rotated(LAM * (a1 * K1 + a2 * Ki)), LAM * (b1 * V1 + b2 * Vi)
    first = 0
    for b, (p, n) in enumerate(zip(start, rows)):
        i = 0
        while i < n:  # up to the end of the page, or of the chunk
            at = p + i
            m = min(n - i, c["block"] - at % c["block"]) if c["block"] else n
            page, slot = (int(s.table[b, at // c["block"]]), at % c["block"]) if c["block"] else (b, at)
            k[page, :, slot: slot + m] = K[first + i: first + i + m].transpose(0, 1)
            v[page, :, slot: slot + m] = V[first + i: first + i + m].transpose(0, 1)
            i += m
        first += n
    return {"k": k, "v": v, "q": rotated(s.q.double())}


def _exact_pages(c, s):
    """The pool after the step, moved with lists: pages hold copies, so the values are those of the inputs."""
    bs, rows = c["block"], [list(r) for r in s.rows]
    refs = [0] * c["pool"]
    for row in rows:
        for x in row:
            refs[x] += 1
    copies = []
    if c["op"] == "resize":
        have = {b: len(rows[b]) for b in s.order}
        for b, n in zip(s.order, s.lens_list):
            while len(rows[b]) > _up(n, bs):
                refs[rows[b].pop()] -= 1
        free = [i for i, x in enumerate(refs) if x == 0][::-1]
        after = list(refs)
        for b, n in zip(s.order, s.lens_list):
            need = _up(n, bs)
            part = bool(n % bs and need <= have[b] and after[rows[b][need - 1]] > 1)
            want = max(0, need - have[b]) + part
            if want > len(free):
                break
            got = [free.pop() for _ in range(want)]
            if part:
                copies.append((rows[b][-1], got[0], n % bs))
            rows[b] = rows[b][:-1] + got if part else rows[b] + got
    elif c["op"] == "fork":
        free = [i for i, x in enumerate(refs) if x == 0][::-1]
        for a, n in zip(s.src_list, s.lens_list):
            for i in range(0 if c["deep"] else n // bs, _up(n, bs)):
                copies.append((rows[a][i], free.pop(), min(bs, n - i * bs)))
    else:
        live = sum(x > 0 for x in refs)
        holes = [i for i in range(live) if refs[i] == 0]
        copies = [(i, holes.pop(0), bs) for i in range(live, c["pool"]) if refs[i] > 0]
    pool = s.pool.clone()
    for a, b, n in copies:
        pool[:, :, b, :, :n] = s.pool[:, :, a, :, :n]
    return {"table": None, "refs": None, "live" if c["op"] == "compact" else "held": None, "pool": pool}


def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "rope": _exact_rope}.get(case["op"], _exact_pages)(case, s)
