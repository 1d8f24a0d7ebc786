"""GPU tests of the page operators (yocopp_pages_resize, _fork, _compact)
against plain Python lists: tables, reference counts and results are equal,
pools bit-equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def y():
    import decode_attention_yocopp_b200 as y
    y.load()
    y.yocopp_get_device_status(reset=True)
    return y


class Pool:
    """A pool of all layers and its model: rows = lists of block numbers."""

    def __init__(self, y, *, batch, mbps, blocks, block=16, layers=2, hkv=2, d=64, dtype=torch.bfloat16, seed=0):
        self.y, self.batch, self.mbps, self.blocks, self.bs, self.layers = y, batch, mbps, blocks, block, layers
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv = torch.randn((layers, 2, blocks, hkv, block, d), generator=g, device="cuda").to(dtype)
        self.model = self.kv.clone()
        self.table = torch.full((batch, mbps), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        self.rows = [[] for _ in range(batch)]
        self.count = [0] * blocks
        self.caches = y.cache_list([y.make_cache(self.kv[i, 0], self.kv[i, 1], self.table) for i in range(layers)])
        self.ws = y.alloc_pages_workspace(self.caches)
        self.ws.fill_(0x5A)  # it needs no clearing
        self.r = random.Random(seed)

    def scatter(self, lens):
        """Rows of the given lengths in blocks, in random blocks of the pool."""
        ids = list(range(self.blocks))
        self.r.shuffle(ids)
        for b, n in enumerate(lens):
            self.rows[b] = [ids.pop() for _ in range(n)]
            for x in self.rows[b]:
                self.count[x] = 1
        self.upload()

    def share(self, a, b, n):
        """Row b's first n blocks become row a's."""
        for x in self.rows[b][:n]:
            self.count[x] -= 1
        self.rows[b][:n] = self.rows[a][:n]
        for x in self.rows[b][:n]:
            self.count[x] += 1
        self.upload()

    def upload(self):
        t = torch.full((self.batch, self.mbps), -1, dtype=torch.int32)
        for b, row in enumerate(self.rows):
            t[b, : len(row)] = torch.tensor(row, dtype=torch.int32)
        self.table.copy_(t)
        self.refs.copy_(torch.tensor(self.count, dtype=torch.int32))

    def free(self):
        return [i for i, c in enumerate(self.count) if c == 0]

    def need(self, n):
        return -(-n // self.bs)

    # ---- the model
    def model_resize(self, seqs, lens):
        held, status, seen = [], 0, set()
        ok = []
        before = self.model.clone()
        have = {}
        for s, n in zip(seqs, lens):
            good = 0 <= s < self.batch and s not in seen
            seen.add(s)
            if good and not 0 <= n <= self.mbps * self.bs:
                good = False
                status = status or self.y.YOCOPP_ECAPACITY
            elif not good:
                status = status or self.y.YOCOPP_EDEVICE_CHECK
            ok.append(good)
            if good:
                have[s] = len(self.rows[s])
                while len(self.rows[s]) > self.need(n):
                    self.count[self.rows[s].pop()] -= 1
        free, after, full = self.free(), list(self.count), False
        for s, n, good in zip(seqs, lens, ok):
            if not good:
                held.append(-1)
                continue
            need = self.need(n)
            part = n % self.bs > 0 and need <= have[s] and after[self.rows[s][need - 1]] > 1
            want = max(0, need - have[s]) + part
            if want and (full or want > len(free)):
                full = True
                status = status or self.y.YOCOPP_ECAPACITY
                held.append(-1)
                continue
            got, free = free[:want], free[want:]
            if part:
                old = self.rows[s].pop()
                self.count[old] -= 1
                self.model[:, :, got[0], :, : n % self.bs] = before[:, :, old, :, : n % self.bs]
            self.rows[s] += got
            for x in got:
                self.count[x] = 1
            held.append(need)
        return held, status

    def model_fork(self, src, dst, lens, deep):
        held, status, seen = [], 0, set()
        free, full, before = self.free(), False, self.model.clone()
        old = [list(r) for r in self.rows]
        for a, b, n in zip(src, dst, lens):
            code = 0
            if not 0 <= b < self.batch or b in seen:
                code = self.y.YOCOPP_EDEVICE_CHECK
            elif not 0 <= n <= self.mbps * self.bs:
                code = self.y.YOCOPP_ECAPACITY
            elif not 0 <= a < self.batch or a == b or old[b]:
                code = self.y.YOCOPP_EDEVICE_CHECK
            elif self.need(n) > len(old[a]):
                code = self.y.YOCOPP_ECAPACITY
            seen.add(b)
            if code:
                status = status or code
                held.append(-1)
                continue
            keep = 0 if deep else n // self.bs
            want = self.need(n) - keep
            if want and (full or want > len(free)):
                full = True
                status = status or self.y.YOCOPP_ECAPACITY
                held.append(-1)
                continue
            got, free = free[:want], free[want:]
            for k, x in enumerate(got):
                m = min(self.bs, n - (keep + k) * self.bs)
                self.model[:, :, x, :, :m] = before[:, :, old[a][keep + k], :, :m]
            self.rows[b] = old[a][:keep] + got
            for x in self.rows[b]:
                self.count[x] += 1
            held.append(self.need(n))
        return held, status

    def model_compact(self):
        live = sum(c > 0 for c in self.count)
        holes = [i for i in range(live) if self.count[i] == 0]
        to = {i: holes.pop(0) for i in range(live, self.blocks) if self.count[i] > 0}
        before = self.model.clone()
        for a, b in to.items():
            self.model[:, :, b] = before[:, :, a]
            self.count[b], self.count[a] = self.count[a], 0
        self.rows = [[to.get(x, x) for x in r] for r in self.rows]
        return live

    # ---- the operators
    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def resize(self, seqs, lens, status=0):
        held = torch.full((len(seqs),), -9, dtype=torch.int32, device="cuda")
        self.y.yocopp_pages_resize(self.caches, self.refs, self.ints(seqs), self.ints(lens), held, self.ws)
        self.check(*self.model_resize(seqs, lens), held)
        return self

    def fork(self, src, dst, lens, deep=False):
        held = torch.full((len(src),), -9, dtype=torch.int32, device="cuda")
        self.y.yocopp_pages_fork(self.caches, self.refs, self.ints(src), self.ints(dst), self.ints(lens), held, self.ws,
                                 deep=deep)
        self.check(*self.model_fork(src, dst, lens, deep), held)
        return self

    def compact(self):
        live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        self.y.yocopp_pages_compact(self.caches, self.refs, live, self.ws)
        self.check([self.model_compact()], 0, live)
        return self

    def check(self, held, status, got):
        torch.cuda.synchronize()
        code = self.y.yocopp_get_device_status(reset=True)
        assert code == status if not status else code in (self.y.YOCOPP_ECAPACITY, self.y.YOCOPP_EDEVICE_CHECK)
        assert got.tolist() == held
        t = self.table.tolist()
        for b, row in enumerate(self.rows):
            assert t[b] == row + [-1] * (self.mbps - len(row)), b
        assert self.refs.tolist() == self.count
        assert torch.equal(self.kv, self.model)


def test_first_blocks_are_the_lowest(y):
    p = Pool(y, batch=3, mbps=4, blocks=10)
    p.resize([2, 0], [17, 16])
    assert p.rows[2] == [0, 1] and p.rows[0] == [2]
    p.resize([2, 1, 0], [0, 33, 64])


@pytest.mark.parametrize("dtype,d,block,layers,hkv", [(torch.bfloat16, 64, 16, 1, 1), (torch.float32, 128, 32, 3, 2),
                                                      (torch.bfloat16, 128, 64, 12, 8), (torch.bfloat16, 64, 128, 2, 3),
                                                      (torch.float32, 64, 256, 2, 5)])
def test_a_run_of_all_operators(y, dtype, d, block, layers, hkv):
    p = Pool(y, batch=12, mbps=7, blocks=90, block=block, layers=layers, hkv=hkv, d=d, dtype=dtype, seed=1)
    r = random.Random(2)
    for step in range(12):
        kind = step % 4
        if kind in (0, 1):
            seqs = r.sample(range(12), r.randint(1, 12))
            p.resize(seqs, [r.choice([0, r.randint(0, 7 * block), len(p.rows[s]) * block, 1]) for s in seqs])
        elif kind == 2:
            empty = [b for b in range(12) if not p.rows[b]] or [11]
            if p.rows[empty[0]]:
                p.resize([11], [0])
            full = [b for b in range(12) if p.rows[b]]
            if not full:
                continue
            src = [r.choice(full) for _ in empty]
            p.fork(src, empty, [r.randint(0, len(p.rows[a]) * block) for a in src], deep=bool(step & 4))
        else:
            p.compact()


def test_copy_on_write_of_a_shared_last_block(y):
    p = Pool(y, batch=4, mbps=4, blocks=12)
    p.scatter([3, 3, 2, 0])
    p.share(0, 1, 2)
    # row 1 cut into the block it shares, row 0 untouched; full blocks need no copy
    p.resize([1], [20])
    assert p.count[p.rows[0][1]] == 1
    p.share(0, 1, 1)
    p.resize([1], [16])
    assert p.rows[1] == [p.rows[0][0]]
    # both rows cut into a shared block in one call: both get their own
    p.resize([1], [0])
    p.fork([0], [1], [48])
    p.resize([0, 1], [40, 41])


@pytest.mark.parametrize("batch,blocks", [(300, 5000), (3, 9000), (8192, 20000)])
def test_large_pools(y, batch, blocks):
    """More requests than warps, pools over several CTAs."""
    p = Pool(y, batch=batch, mbps=6, blocks=blocks, layers=1, hkv=1, seed=3)
    r = random.Random(4)
    n = min(batch, blocks // 7)
    p.scatter([r.randint(0, 3) if b < n else 0 for b in range(batch)])
    seqs = list(range(batch))
    r.shuffle(seqs)
    p.resize(seqs, [r.randint(0, 30) if r.random() < 0.7 else 6 * 16 for _ in seqs])
    empty = [b for b in range(batch) if not p.rows[b]]
    full = [b for b in range(batch) if p.rows[b]]
    src = [r.choice(full) for _ in empty]
    p.fork(src, empty, [r.randint(0, len(p.rows[a]) * 16) for a in src])
    p.compact()


def test_blocks_run_out(y):
    p = Pool(y, batch=4, mbps=8, blocks=9)
    p.scatter([2, 2, 0, 0])
    # 5 spare: 3 given, 4 refused, the later one that needs any refused too, the one that needs none granted
    p.resize([2, 3, 0, 1], [48, 64, 33, 32])
    p.fork([0, 0], [3, 3], [32, 32])           # the same row twice
    p.resize([3], [0])
    p.fork([0], [3], [48])                     # more than the source holds
    p.fork([2], [3], [48], deep=True)          # too few blocks
    # no block for the copy on write: the row keeps what is left of it
    q = Pool(y, batch=2, mbps=4, blocks=3)
    q.scatter([3, 0])
    q.fork([0], [1], [48])
    q.resize([0], [40])


def test_requests_that_are_refused(y):
    p = Pool(y, batch=3, mbps=4, blocks=20)
    p.scatter([2, 3, 0])
    p.resize([-1, 3, 0, ][:3], [5, 5, 16])
    p.resize([1, 1], [10, 64])
    p.resize([0, 1, 2], [-5, 65, 2 ** 31 - 1])
    p.fork([0], [1], [16])                     # not empty
    p.fork([2], [2], [0])                      # itself
    p.fork([5], [2], [0])
    p.fork([0], [7], [0])
    p.fork([0], [2], [-1])
    p.fork([0, 2], [2, 1], [16, 1])


def test_empty_requests_and_full_pool(y):
    p = Pool(y, batch=2, mbps=4, blocks=8)
    p.compact()
    p.resize([0, 1], [64, 64])
    p.compact()
    p.resize([0, 1], [64, 64])
    p.resize([0], [0])
    p.compact()
    assert sorted(p.rows[1]) == [0, 1, 2, 3]
    held = torch.empty(0, dtype=torch.int32, device="cuda")
    y.yocopp_pages_resize(p.caches, p.refs, held, held, held, p.ws)


def test_damaged_tables_are_recorded_and_stay_in_bounds(y):
    p = Pool(y, batch=2, mbps=4, blocks=8)
    p.scatter([3, 0])
    p.table[0, 1] = 10 ** 6
    held = torch.empty(1, dtype=torch.int32, device="cuda")
    live = torch.empty(1, dtype=torch.int32, device="cuda")
    y.yocopp_pages_fork(p.caches, p.refs, p.ints([0]), p.ints([1]), p.ints([48]), held, p.ws, deep=True)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    y.yocopp_pages_compact(p.caches, p.refs, live, p.ws)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    y.yocopp_pages_resize(p.caches, p.refs, p.ints([0]), p.ints([0]), held, p.ws)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    # counted less often than it is named
    p = Pool(y, batch=2, mbps=4, blocks=8)
    p.scatter([2, 0])
    p.refs[p.rows[0][1]] = 0
    y.yocopp_pages_resize(p.caches, p.refs, p.ints([0]), p.ints([0]), held, p.ws)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    assert p.refs.min() == 0


def test_graph_replay(y):
    """A captured step (resize, fork) replayed on what the last one left."""
    p = Pool(y, batch=6, mbps=6, blocks=40, seed=5)
    p.scatter([2, 3, 1, 0, 0, 0])
    seqs, lens = p.ints([0, 1, 2]), p.ints([40, 48, 17])
    src, dst, flens = p.ints([0, 0]), p.ints([3, 4]), p.ints([40, 33])
    h1, h2 = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")

    def step():
        y.yocopp_pages_resize(p.caches, p.refs, seqs, lens, h1, p.ws)
        y.yocopp_pages_fork(p.caches, p.refs, src, dst, flens, h2, p.ws)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for sl, fl in (([40, 48, 17], [40, 33]), ([50, 0, 18], [7, 50])):
        lens.copy_(p.ints(sl))
        flens.copy_(p.ints(fl))
        g.replay()
        held1, s1 = p.model_resize([0, 1, 2], sl)
        held2, s2 = p.model_fork([0, 0], [3, 4], fl, False)
        p.check(held2, s1 or s2, h2)
        assert h1.tolist() == held1
        p.resize([3, 4], [0, 0])


def test_offsets_past_32_bits(y):
    blocks = (5 << 30) // (8 * 256 * 128 * 2)
    kv = torch.empty((2, blocks, 8, 256, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    refs = torch.ones(blocks, dtype=torch.int32, device="cuda")
    refs[blocks - 3:] = 0
    caches = y.cache_list([y.make_cache(kv[0], kv[1], table)])
    ws = y.alloc_pages_workspace(caches)
    table[0, 0] = blocks - 4
    kv[:, blocks - 4] = 3.0
    held = torch.empty(1, dtype=torch.int32, device="cuda")
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    y.yocopp_pages_fork(caches, refs, one(0), one(1), one(200), held, ws, deep=True)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == 0
    assert int(table[1, 0]) == blocks - 3 and bool((kv[:, blocks - 3, :, :200] == 3).all())
