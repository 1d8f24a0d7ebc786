"""GPU parity of yocopp_chunk_attn (a chunk of new tokens over a cache: causal,
windowed, tree-masked) against a plain fp64 implementation.

Every cache position outside the sequences holds NaN, so a read of one poisons
the output.  Tolerances (tolerance()), first order, per output element, with w
the exact softmax weights and A = sum_u w_u |V_u| + |out|:
* a score s is an fp32 sum of head_dim products: |ds| <= g = head_dim 2^-23
  scale sum_c |q_c k_c| at most (products of bf16 are exact; twice the bound of
  an fp32 sum, as the tensor cores' sums may truncate), plus 4 2^-24 |s| for
  the scale and the difference from the maximum; a weight then is off by
  exp(2 ds) - 1, relative, numerator and row sum together;
* bf16: the probabilities are rounded to bf16 (2^-8 relative at most) and the
  exponential is within 2^-12: (2^-8 + 2^-12) A; the output is rounded: 2^-8 |out|;
* fp32: the exponential within 4 2^-24, sums of 64 terms and of the tiles:
  (68 + tiles) 2^-24 A.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def y():
    import decode_attention_yocopp_b200 as y
    y.load()
    y.yocopp_get_device_status(reset=True)
    return y


class Case:
    """Seeded inputs: cache (NaN outside the sequences), queries, masks."""

    def __init__(self, y, *, dtype="bf16", d=128, hkv=2, G=4, rows, pos, block=0, window=0, tree=None, seed=0,
                 capacity=0, scale=0.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.d, self.hkv, self.G, self.rows, self.pos = DT[dtype], d, hkv, G, list(rows), list(pos)
        self.window, self.scale, self.hq = window, scale, hkv * G
        B = len(self.rows)
        T = [a + b for a, b in zip(self.pos, self.rows)]
        cap = max(capacity, max(T), 1)
        self.K = [(torch.randn((hkv, t, d), generator=g) * 1.5).to(self.dt).cuda() for t in T]
        self.V = [torch.randn((hkv, t, d), generator=g).to(self.dt).cuda() for t in T]
        self.table = None
        if block:
            per = -(-cap // block)
            cap = per * block
            perm = torch.randperm(B * per + spare, generator=g)
            table = torch.full((B, per), -1, dtype=torch.int32)
            for b, t in enumerate(T):  # blocks past the sequence stay -1
                n = -(-t // block)
                table[b, :n] = perm[b * per: b * per + n].int()
            self.table = table.cuda()
            shape = (B * per + spare, hkv, block, d)
        else:
            shape = (B, hkv, cap, d)
        self.cap = cap
        self.k = torch.full(shape, float("nan"), dtype=self.dt, device="cuda")
        self.v = torch.full(shape, float("nan"), dtype=self.dt, device="cuda")
        for b in range(B):
            self.put(b)
        self.total = sum(self.rows)
        self.q = torch.randn((self.total, self.hq, d), generator=g).to(self.dt).cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.rows)]), dtype=torch.int32, device="cuda")
        self.pos_t = torch.tensor(self.pos, dtype=torch.int32, device="cuda")
        self.words = None
        if tree is not None:
            self.words = [tree(b, j, n, g) for b, n in enumerate(self.rows) for j in range(n)]
            self.tree_t = torch.tensor([w - (1 << 64) if w >> 63 else w for w in self.words], dtype=torch.int64,
                                       device="cuda")
        else:
            self.tree_t = None
        self.cache = y.make_cache(self.k, self.v, self.table)
        self.ws = y.alloc_chunk_workspace(self.cache, self.hq)

    def put(self, b):
        """Sequence b's logical rows into the cache."""
        t = self.K[b].shape[1]
        if self.table is None:
            self.k[b, :, :t], self.v[b, :, :t] = self.K[b], self.V[b]
            return
        bs = self.k.shape[2]
        for i in range(-(-t // bs)):
            n = min(bs, t - i * bs)
            blk = int(self.table[b, i])
            self.k[blk, :, :n] = self.K[b][:, i * bs: i * bs + n]
            self.v[blk, :, :n] = self.V[b][:, i * bs: i * bs + n]

    def run(self, y, out=None, **kw):
        out = torch.full_like(self.q, float("nan")) if out is None else out
        y.yocopp_chunk_attn(self.q, self.cache, out, self.ws, pos=self.pos_t, cu_q=self.cu, max_q=max(self.rows),
                            tree_mask=self.tree_t, window=self.window, scale=self.scale, **kw)
        return out

    def reference(self):
        """(exact output, tolerance) in fp64."""
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        sc = self.scale or 1.0 / math.sqrt(self.d)
        first = 0
        for b, (p, n) in enumerate(zip(self.pos, self.rows)):
            if n == 0:
                continue
            T = p + n
            u, j = torch.arange(T, device="cuda"), torch.arange(n, device="cuda")
            if self.words is not None:
                see = torch.zeros((n, T), dtype=torch.bool)
                see[:, :p] = True
                for jj in range(n):
                    for c in range(n):
                        see[jj, p + c] = bool((self.words[first + jj] >> c) & 1)
                see = see.cuda()
            else:
                see = u[None, :] <= p + j[:, None]
                if self.window:
                    see &= u[None, :] > p + j[:, None] - self.window
            for h in range(self.hq):
                q = self.q[first: first + n, h].double()
                K, V = self.K[b][h // self.G].double(), self.V[b][h // self.G].double()
                s = (q @ K.T * sc).masked_fill(~see, -math.inf)
                top = s.amax(1, keepdim=True)
                w = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                L = w.sum(1, keepdim=True)
                w = w / torch.where(L == 0, torch.ones_like(L), L)
                # what is not seen takes no part, whatever it is
                o = torch.stack([w[i][see[i]] @ V[see[i]] for i in range(n)]) if not bool(torch.isfinite(V).all()) else w @ V
                out[first: first + n, h] = o
                Vf = torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0).abs()
                Kf = torch.nan_to_num(K, nan=0.0, posinf=0.0, neginf=0.0)
                A = w.nan_to_num() @ Vf + o.abs()
                g = self.d * 2.0 ** -23 * sc * (q.abs() @ Kf.abs().T).masked_fill(~see, 0).amax(1, keepdim=True)
                g = g + 4 * 2.0 ** -24 * s.masked_fill(~see, 0).abs().amax(1, keepdim=True)
                ds = torch.expm1(2 * g)
                if self.dt == torch.bfloat16:
                    tol[first: first + n, h] = (2.0 ** -8 + 2.0 ** -12 + ds) * A + 2.0 ** -8 * o.abs()
                else:
                    tol[first: first + n, h] = ((68 + T / 64) * 2.0 ** -24 + ds) * A
            first += n
        return out, tol

    def check(self, y, got=None):
        got = self.run(y) if got is None else got
        torch.cuda.synchronize()
        assert y.yocopp_get_device_status(reset=True) == 0
        ref, tol = self.reference()
        fine = torch.isfinite(ref)
        assert bool((torch.isfinite(got) == fine).all())
        over = ((got.double() - ref).abs() - tol * 1.001 - 1e-30)[fine]
        assert float(over.max()) <= 0, f"{int((over > 0).sum())} of {over.numel()} beyond the tolerance by {float(over.max())}"
        return got


def chain():
    """Random trees: node j sees itself and the ancestors of an earlier node."""
    masks = []

    def word(b, j, n, g):
        m = 1 << j
        if j == 0:
            masks.clear()
        else:
            m |= masks[int(torch.randint(max(0, j - 4), j, (1,), generator=g))]
        masks.append(m)
        return m
    return word


TYPES = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)]


@pytest.mark.parametrize("dtype,d", TYPES)
def test_one_token_each(y, dtype, d):
    Case(y, dtype=dtype, d=d, rows=[1, 1, 1], pos=[0, 5, 300], block=16, seed=1).check(y)


# rows per KV head of 1..32, ..64, ..128 and more (each row tile), around their edges
@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("rows,G", [([8, 3], 4), ([9], 4), ([16, 1], 4), ([32, 17], 4), ([33], 4), ([1], 3), ([65, 10], 5),
                                    ([257], 1), ([130, 2, 77], 3)])
def test_causal(y, dtype, d, rows, G):
    Case(y, dtype=dtype, d=d, G=G, rows=rows, pos=[100 + 61 * i for i in range(len(rows))], block=32, seed=2).check(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,rows", [(40, [1, 3]), (129, [2]), (300, [1, 2])])
def test_many_query_heads_for_one_kv_head(y, dtype, G, rows):
    Case(y, dtype=dtype, d=64, hkv=1, G=G, rows=rows, pos=[150, 7][: len(rows)], block=16, seed=2).check(y)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("block", [0, 16, 32, 64, 128, 256])
def test_layouts_and_context_edges(y, dtype, d, block):
    # contexts ending just before, at and past the end of a key tile; a capacity beyond the longest
    pos = [0, 62, 63, 64, 126, 127, 128, 255, 511]
    Case(y, dtype=dtype, d=d, hkv=1, G=2, rows=[1, 2, 1, 2, 1, 2, 1, 3, 2], pos=pos, block=block, capacity=600,
         seed=3).check(y)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("rows,pos,window", [([5], [400], 1), ([40, 3], [390, 0], 130), ([70], [1000], 64),
                                             ([200], [50], 37), ([3], [2], 1000), ([129], [600], 128)])
def test_window(y, dtype, d, rows, pos, window):
    Case(y, dtype=dtype, d=d, G=3, rows=rows, pos=pos, window=window, block=64, seed=4).check(y)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("rows,pos", [([16, 7], [200, 0]), ([64], [127]), ([33, 64], [100, 3]), ([1, 2], [0, 90])])
def test_tree(y, dtype, d, rows, pos):
    Case(y, dtype=dtype, d=d, rows=rows, pos=pos, tree=chain(), block=16, seed=5).check(y)


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("n", [6, 40])
def test_rows_that_see_nothing_give_zeros(y, dtype, d, n):
    c = Case(y, dtype=dtype, d=d, rows=[n, n], pos=[0, 3], tree=lambda b, j, n, g: 0 if j % 3 else (1 << n) - 1, seed=6)
    got = c.check(y)
    assert float(got[1].abs().max()) == 0 and float(got[n + 1].abs().max()) > 0


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("rows,pos,window,tree", [([5], [130], 0, False), ([40], [100], 0, False), ([70], [64], 0, False),
                                                  ([9], [300], 20, False), ([60], [300], 20, False),
                                                  ([12], [140], 0, True), ([64], [90], 0, True)])
def test_masked_places_may_hold_anything(y, dtype, d, rows, pos, window, tree):
    """NaN and infinities in keys and values that some rows see and others do not: the others' results are those of
    clean inputs, and the rows that see them are not finite where the exact result is not."""
    c = Case(y, dtype=dtype, d=d, G=2, rows=rows, pos=pos, window=window, block=16, seed=7,
             tree=(lambda b, j, n, g: 1 << j) if tree else None)
    n, p = rows[0], pos[0]
    clean = c.check(y)
    bad = p + n // 2
    c.V[0][0, bad, 3] = float("nan")
    c.V[0][1, bad, 5] = float("inf")
    if window:
        c.V[0][0, p - 2, 1] = -float("inf")
    c.K[0][1, p + n - 1, 7] = float("nan")
    c.put(0)
    got = c.run(y)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == 0
    for j in range(n):
        def sees(u):
            if tree:
                return u < p or u == p + j
            return u <= p + j and (not window or u > p + j - window)
        for h in range(c.hq):
            a, b = got[j, h].float(), clean[j, h].float()
            hit = torch.zeros(d, dtype=torch.bool, device="cuda")
            if h // 2 == 0:
                hit[3] |= sees(bad)
                hit[1] |= bool(window) and sees(p - 2)
            else:
                hit[5] |= sees(bad)
                hit |= sees(p + n - 1)
            assert torch.equal(torch.isfinite(a), ~hit), (j, h)
            # the same weights and products; only -0 and +0 terms may differ
            assert torch.allclose(a[~hit], b[~hit], rtol=0, atol=0), (j, h)


@pytest.mark.parametrize("dtype,d", TYPES)
def test_infinite_scores(y, dtype, d):
    c = Case(y, dtype=dtype, d=d, G=2, hkv=1, rows=[3], pos=[200], seed=8)
    c.K[0][0, 150] = 0
    c.K[0][0, 150, 0] = -float("inf")          # a score of -inf where q > 0: weight 0
    c.q[:, :, 0] = c.q[:, :, 0].abs() + 0.5
    c.put(0)
    c.check(y)
    c.K[0][0, 150, 0] = float("inf")           # +inf: the row is NaN
    c.put(0)
    got = c.run(y)
    torch.cuda.synchronize()
    assert bool(torch.isnan(got).all())


@pytest.mark.parametrize("dtype,d,G,n", [("bf16", 128, 4, 8), ("bf16", 128, 4, 200), ("bf16", 64, 8, 16),
                                         ("f32", 128, 2, 4), ("f32", 64, 4, 60)])
def test_long_context_split_over_all_sms(y, dtype, d, G, n):
    Case(y, dtype=dtype, d=d, hkv=1, G=G, rows=[n], pos=[20011], block=64, seed=9).check(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_some_empty(y, dtype):
    r = np.random.default_rng(10)
    rows = [int(x) for x in r.integers(0, 12, size=600)]
    pos = [int(x) for x in r.integers(0, 300, size=600)]
    Case(y, dtype=dtype, d=64, hkv=1, G=1, rows=rows, pos=pos, block=16, seed=10).check(y)


def test_uniform_rows_no_pos(y):
    c = Case(y, rows=[40, 40], pos=[0, 0], seed=11)
    out = torch.full_like(c.q, float("nan"))
    y.yocopp_chunk_attn(c.q, c.cache, out, c.ws, n_uniform=40)
    c.check(y, out)


def test_equals_prefill_and_decode(y):
    """The framework's other attentions of the same rows agree within both roundings."""
    c = Case(y, rows=[150], pos=[77], block=64, seed=12)
    got = c.check(y)
    out = torch.empty_like(c.q)
    y.yocopp_prefill_attn(c.q, c.cache, out, pos=c.pos_t, cu_q=c.cu, max_q=150)
    c.check(y, out)
    one = Case(y, rows=[1, 1], pos=[500, 77], block=64, seed=13)
    got = one.check(y)
    ws = y.alloc_workspace(one.cache, one.hq)
    y.yocopp_decode_attn(one.q, one.cache, one.pos_t + 1, got, ws)
    one.check(y, got)


def test_results_do_not_depend_on_timing(y):
    c = Case(y, rows=[8, 5, 30], pos=[9000, 100, 3000], block=64, seed=14)
    first = c.run(y)
    for _ in range(20):
        assert torch.equal(c.run(y).view(torch.int16), first.view(torch.int16))


def test_rows_behind_the_last_and_skipped_sequences_are_left(y):
    c = Case(y, rows=[4, 6, 5], pos=[10, 600, 20], capacity=606, seed=15)
    c.pos_t[1] = 601  # past the capacity
    q = torch.cat([c.q, c.q])
    out = torch.full_like(q, 7.0)
    y.yocopp_chunk_attn(q, c.cache, out, c.ws, pos=c.pos_t, cu_q=c.cu, max_q=6)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_ECAPACITY
    assert bool((out[4:10] == 7).all()) and bool((out[15:] == 7).all())
    ref, tol = c.reference()
    for s in (slice(0, 4), slice(10, 15)):
        assert bool(((out[s].double() - ref[s]).abs() <= tol[s]).all())


@pytest.mark.parametrize("dtype,rows", [("bf16", 4), ("bf16", 100), ("f32", 4), ("f32", 40)])
def test_invalid_inputs_on_the_device_are_recorded(y, dtype, rows):
    c = Case(y, dtype=dtype, rows=[rows, rows], pos=[100, 100], block=32, seed=16)
    good = c.check(y)
    c.table[1, 0] = 10 ** 6
    out = c.run(y)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    assert torch.equal(out[:rows], good[:rows])
    c.table[1, 0] = -1
    c.cu[1] = -3
    c.run(y)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    c.cu[1], c.cu[2] = rows, 2 * rows + 1  # past total_q
    out = c.run(y)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    assert torch.equal(out[:rows], good[:rows])


@pytest.mark.parametrize("dtype,rows", [("bf16", 4), ("bf16", 100), ("f32", 4)])
def test_a_wait_that_runs_out_is_recorded(y, dtype, rows):
    c = Case(y, dtype=dtype, rows=[rows], pos=[900], seed=17)
    y.yocopp_testing_set_decode_fault(0, 20_000_000)
    try:
        c.run(y)
        torch.cuda.synchronize()
        assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_ETIMEOUT
    finally:
        y.yocopp_testing_set_decode_fault(-1, 2_000_000_000)
    c.check(y)


@pytest.mark.parametrize("dtype,rows", [("bf16", 20), ("bf16", 70), ("f32", 20), ("f32", 3)])
def test_released_blocks_below_the_window(y, dtype, rows):
    c = Case(y, dtype=dtype, rows=[rows], pos=[700], window=100, block=16, seed=18)
    ref = c.check(y)
    gone = 601 // 16  # blocks wholly below the first window, which starts at 601
    blocks = c.table[0, :gone].long()
    c.k[blocks], c.v[blocks] = float("nan"), float("nan")
    c.table[0, :gone] = -1
    assert torch.equal(c.check(y), ref)


def test_graph_replay_with_new_inputs(y):
    c = Case(y, rows=[8, 3], pos=[3000, 200], block=64, seed=19)
    out = c.run(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(y, out)
    c.pos, c.rows = [2500, 100], [3, 8]
    c.pos_t.copy_(torch.tensor(c.pos))
    c.cu.copy_(torch.tensor([0, 3, 11]))
    c.K = [k[:, : p + n] if k.shape[1] >= p + n else k for k, p, n in zip(c.K, c.pos, c.rows)]
    c.V = [v[:, : p + n] if v.shape[1] >= p + n else v for v, p, n in zip(c.V, c.pos, c.rows)]
    c.q.copy_(c.q.roll(1, 0))
    out.fill_(float("nan"))
    g.replay()
    c.check(y, out)


def test_two_streams_with_their_own_workspaces(y):
    a = Case(y, rows=[8], pos=[9000], block=64, seed=20)
    b = Case(y, rows=[300], pos=[500], block=64, seed=21)
    outs = []
    torch.cuda.synchronize()
    for c in (a, b):
        s = torch.cuda.Stream()
        o = torch.full_like(c.q, float("nan"))
        outs.append(o)
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(10):
            c.run(y, o, stream=s)
    torch.cuda.synchronize()
    a.check(y, outs[0])
    b.check(y, outs[1])


def test_offsets_past_32_bits(y):
    """A pool of more than 4 GiB for each of K and V, the sequence's blocks at its end."""
    d, hkv, bs = 128, 8, 64
    blocks = (5 << 30) // (hkv * bs * d * 2)
    c = Case(y, hkv=hkv, rows=[6], pos=[300], block=bs, seed=22)
    k = torch.empty((blocks, hkv, bs, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    old = c.table[0].clone()
    for i in range(old.numel()):
        k[blocks - 1 - i], v[blocks - 1 - i] = c.k[int(old[i])], c.v[int(old[i])]
        c.table[0, i] = blocks - 1 - i
    c.cache = y.make_cache(k, v, c.table)
    c.check(y)


def test_binding_refuses_what_would_be_read_past_its_end(y):
    c = Case(y, rows=[3, 4], pos=[10, 20], tree=chain(), seed=23)
    out = torch.empty_like(c.q)
    ok = dict(pos=c.pos_t, cu_q=c.cu, max_q=4, tree_mask=c.tree_t)
    for kw in (dict(pos=c.pos_t[:1]), dict(cu_q=c.cu[:2]), dict(tree_mask=c.tree_t[:6]), dict(total_q=8), dict(num_q_heads=16)):
        with pytest.raises(TypeError):
            y.yocopp_chunk_attn(c.q, c.cache, out, c.ws, **{**ok, **kw})
    with pytest.raises(TypeError):
        y.yocopp_chunk_attn(c.q, c.cache, out[:, ::2], c.ws, **ok)
    with pytest.raises(y.YocoppError):
        y.yocopp_chunk_attn(c.q, c.cache, out, c.ws[: c.ws.numel() - 256], **ok)
    c.check(y)


def test_fewer_rows_than_the_tensor_has(y):
    c = Case(y, rows=[3, 4], pos=[10, 20], seed=24)
    big = torch.cat([c.q, c.q])
    out = torch.full_like(big, 5.0)
    y.yocopp_chunk_attn(big, c.cache, out, c.ws, pos=c.pos_t, cu_q=c.cu, total_q=7, max_q=4)
    assert bool((out[7:] == 5).all())
    c.check(y, out[:7].clone())
