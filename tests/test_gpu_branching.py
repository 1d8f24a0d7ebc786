"""The branching operators together, as a server uses them: pages are given, a
prompt with image positions is written and attended in two chunks, the sequence
is forked, each branch verifies a tree of drafts and keeps a part of it, rows
are rolled back and ended, and the pool is compacted.  After every step the
caches hold, for each sequence, the rows of a plain fp64 model of it (within a
rounding of the turned composition), and the attentions equal a plain fp64
softmax over what the cache holds.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

LAYERS, SHARED, HQ, HKV, D, BLOCK = 4, 2, 8, 2, 128, 16


@pytest.fixture(scope="module")
def y():
    import decode_attention_yocopp_b200 as y
    y.load()
    y.yocopp_get_device_status(reset=True)
    return y


class Server:
    """Stack, rope and the model: tokens of each row as (turned K, V) per layer."""

    def __init__(self, y, dtype, batch=6, blocks=40, mbps=12):
        from decode_attention_yocopp_b200.pipeline import SharedKVStack
        self.y, self.dtype = y, dtype
        self.g = torch.Generator().manual_seed(3)
        self.table = torch.zeros((batch, mbps), dtype=torch.int32, device="cuda")
        self.alpha = {2: (0.02, 1 / 35 + 0.003, -0.01, 1 / 35 + 0.004)}
        self.stack = SharedKVStack(LAYERS, batch, HQ, HKV, D, dtype, self.alpha, block_table=self.table, block_size=BLOCK,
                                   num_blocks=blocks)
        self.stack.start_pages()
        self.rope = y.make_rope(D, sections=[24, 20, 20])
        self.kv = [[torch.zeros((0, HKV, D), dtype=torch.float64, device="cuda") for _ in range(batch)] for _ in range(4)]

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype).cuda()

    def turned(self, x, positions):
        inv = torch.tensor([10000.0 ** (-2 * c / D) for c in range(D // 2)], dtype=torch.float64, device="cuda")
        axis = torch.tensor([0] * 24 + [1] * 20 + [2] * 20, device="cuda")
        ang = (positions.double()[axis].T * inv)[:, None]
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat((a * torch.cos(ang) - b * torch.sin(ang), b * torch.cos(ang) + a * torch.sin(ang)), -1)

    def step(self, rows, counts, tree=None, window=0):
        """New tokens of the rows: written in both cached layers, attended in layer 1 (over its own cache) and in
        the shared layer; checked against the model."""
        batch, st = self.table.shape[0], self.stack
        have = [self.kv[0][b].shape[0] for b in range(batch)]
        n = [counts[rows.index(b)] if b in rows else 0 for b in range(batch)]
        held = st.resize_pages(self.ints(rows), self.ints([have[b] + n[b] for b in rows]))
        assert held.tolist() == [-(-(have[b] + n[b]) // BLOCK) for b in rows]
        cu = self.ints([sum(n[:b]) for b in range(batch + 1)])
        pos, total = self.ints(have), sum(n)
        raw = [self.rand(total, HKV, D) for _ in range(4)]
        K1, V1, K2, V2 = raw
        positions = torch.randint(0, 500, (3, total), generator=self.g, dtype=torch.int32).cuda()
        words = None
        if tree is not None:
            words = torch.tensor([tree[j] for b in range(batch) for j in range(n[b])], dtype=torch.int64, device="cuda")
        outs = []
        for layer, (ki, vi) in ((1, (K1, V1)), (2, (K2, V2))):
            q = self.rand(total, HQ, D)
            qt, out = torch.empty_like(q), torch.empty_like(q)
            st.write_rope(layer, K1, V1, ki, vi, self.rope, positions, pos, q=q, q_out=qt, cu_new=cu)
            assert torch.equal(st.turn_queries(q.clone(), self.rope, positions), qt)
            a = [float(torch.tensor(x, dtype=torch.float32)) for x in st.layer_alpha(layer)]
            k = self.turned(35.0 * (a[0] * K1.double() + a[1] * ki.double()), positions)
            v = 35.0 * (a[2] * V1.double() + a[3] * vi.double())
            for b in range(batch):
                s = slice(sum(n[:b]), sum(n[: b + 1]))
                at = 2 * (layer - 1)
                self.kv[at][b], self.kv[at + 1][b] = (torch.cat((x, w[s])) for x, w in ((self.kv[at][b], k), (self.kv[at + 1][b], v)))
            st.chunk_attend(layer, qt, out, pos=pos, cu_q=cu, max_q=max(n), tree_mask=words, window=window)
            outs.append((layer, qt, out))
        torch.cuda.synchronize()
        assert self.y.yocopp_get_device_status(reset=True) == 0
        self.check_caches()
        for layer, qt, out in outs:
            self.check_attention(layer, qt, out, have, n, tree, window)

    def rows_of(self, layer, b):
        n = self.kv[0][b].shape[0]
        blocks = self.table[b, : -(-n // BLOCK)].long()
        return [x[layer][blocks].transpose(1, 2).reshape(-1, HKV, D)[:n] for x in (self.stack.k, self.stack.v)]

    def check_caches(self):
        half = 2.0 ** -8 if self.dtype == torch.bfloat16 else 2.0 ** -24
        for layer in (1, 2):
            for b in range(self.table.shape[0]):
                for got, want in zip(self.rows_of(layer, b), (self.kv[2 * layer - 2][b], self.kv[2 * layer - 1][b])):
                    # rounding, and fp32 composition and turn of terms up to 35 * 0.04 * 5 and their like
                    assert bool(((got.double() - want).abs() <= half * want.abs() + 40 * 2.0 ** -22).all()), (layer, b)

    def check_attention(self, layer, q, out, have, n, tree, window):
        for b in range(self.table.shape[0]):
            if n[b] == 0:
                continue
            k, v = (x.double() for x in self.rows_of(layer, b))
            s0 = sum(n[:b])
            u, j = torch.arange(k.shape[0], device="cuda"), torch.arange(n[b], device="cuda")
            if tree is not None:
                see = torch.tensor([[x < have[b] or bool((tree[r] >> (x - have[b])) & 1) for x in range(k.shape[0])]
                                    for r in range(n[b])], device="cuda")
            else:
                see = (u <= have[b] + j[:, None]) & (u > have[b] + j[:, None] - (window or 10 ** 9))
            for h in range(HQ):
                s = (q[s0: s0 + n[b], h].double() @ k[:, h // 4].T / math.sqrt(D)).masked_fill(~see, -math.inf)
                w = torch.softmax(s, 1)
                ref = w @ v[:, h // 4]
                A = w @ v[:, h // 4].abs() + ref.abs()
                # scores up to 40 in fp32: 2^-15 relative of a weight; probabilities and output in bf16: 2^-8 each
                tol = (2.0 ** -15 + (2.0 ** -8 if self.dtype == torch.bfloat16 else 0)) * A
                tol = tol + (2.0 ** -8 * ref.abs() if self.dtype == torch.bfloat16 else 0)
                assert bool(((out[s0: s0 + n[b], h].double() - ref).abs() <= tol).all()), (layer, b, h)

    def keep(self, b, n):
        for x in self.kv:
            x[b] = x[b][:n]

    def copy(self, a, b, n):
        for x in self.kv:
            x[b] = x[a][:n].clone()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_server_with_branches(y, dtype):
    s = Server(y, dtype)
    st = s.stack
    # two prompts in chunks, the second chunk windowed
    s.step([0, 4], [37, 20])
    s.step([0, 4], [50, 3], window=40)
    # three branches of row 0 (one of them of its first 60 tokens), one deep copy of row 4
    held = st.fork_pages(s.ints([0, 0, 0]), s.ints([1, 2, 3]), s.ints([87, 87, 60]))
    assert held.tolist() == [6, 6, 4]
    for b, n in ((1, 87), (2, 87), (3, 60)):
        s.copy(0, b, n)
    assert st.fork_pages(s.ints([4]), s.ints([5]), s.ints([23]), deep=True).tolist() == [2]
    s.copy(4, 5, 23)
    s.check_caches()
    # a tree of drafts on each branch: nodes 1, 2 follow 0; 3 follows 1; 4 follows 2
    s.step([1, 2, 3], [5, 5, 5], tree=[0b1, 0b11, 0b101, 0b1011, 0b10101])
    # one node of each path is kept: the others' tokens are rolled back (row 1 into the pages that it shares)
    for b, n in ((1, 80), (2, 88), (3, 61)):
        s.keep(b, n)
    assert st.resize_pages(s.ints([1, 2, 3]), s.ints([80, 88, 61])).tolist() == [5, 6, 4]
    s.check_caches()
    # row 0 cut in the middle of a shared page: what it writes next reaches no other row
    s.keep(0, 70)
    st.resize_pages(s.ints([0]), s.ints([70]))
    s.step([0, 1, 2, 3, 5], [9, 1, 2, 30, 1])
    # two rows end, the pool closes its holes, and the rest goes on
    s.keep(2, 0)
    s.keep(4, 0)
    st.resize_pages(s.ints([2, 4]), s.ints([0, 0]))
    live = int(st.compact_pages())
    assert live == int((st.block_refs > 0).sum()) and int((st.block_refs[live:] > 0).sum()) == 0
    s.check_caches()
    s.step([0, 1, 3], [1, 4, 1])
    assert y.yocopp_get_device_status(reset=True) == 0


def test_pages_need_paged_caches(y):
    from decode_attention_yocopp_b200.pipeline import SharedKVStack
    st = SharedKVStack(4, 1, 4, 1, 64, torch.float32, {2: (0, 1, 0, 1)}, capacity=64)
    with pytest.raises(ValueError):
        st.start_pages()
