"""GPU parity of yocopp_rope_compose_append (rotary positions of one to four
axes fused with the composition and the append, and applied to the queries)
against a plain fp64 implementation.

Tolerances: the cosine and sine of an angle reduced in fp64 are within
t = 4 2^-24 absolutely (the remainder rounded to fp32, at most half a turn:
pi 2^-25, and sincospif); the composed key is within 2^-22 |lambda| (|a1 x1| +
|a2 xi|) (fp32); a turned channel then is within (t + 2 2^-24) (|x| + |y|) plus
the composition's error of both, and the result is rounded: 2^-8 of it in bf16,
2^-24 in fp32.  Values: the bits of yocopp_compose_append.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LAM, ALPHA = 35.0, (0.04, 1 / 35 + 0.01, -0.03, 1 / 35 + 0.02)


@pytest.fixture(scope="module")
def y():
    import decode_attention_yocopp_b200 as y
    y.load()
    y.yocopp_get_device_status(reset=True)
    return y


class Case:
    def __init__(self, y, *, dtype="bf16", d=128, hkv=2, hq=6, rows=(5, 3), start=(0, 9), block=16, axes=3, rotary=None,
                 interleaved=False, far=1 << 20, seed=0, axis=None):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.d, self.hkv, self.rows, self.start, self.block = DT[dtype], d, hkv, rows, start, block
        self.rotary, self.interleaved, self.total = rotary or d, interleaved, sum(rows)
        pairs, B = self.rotary // 2, len(rows)
        self.axis = axis or [min(axes - 1, c * axes // pairs) for c in range(pairs)]
        cap = max(a + b for a, b in zip(start, rows)) + 3
        self.table = None
        if block:
            per = -(-cap // block)
            self.table = torch.randperm(B * per + 2, generator=g)[: B * per].int().reshape(B, per).cuda()
            shape = (B * per + 2, hkv, block, d)
        else:
            shape = (B, hkv, cap, d)
        self.k = torch.full(shape, 7.0, dtype=self.dt, device="cuda")
        self.v = torch.full(shape, 7.0, dtype=self.dt, device="cuda")
        self.raw = [torch.randn((self.total, hkv, d), generator=g).to(self.dt).cuda() for _ in range(4)]
        self.q = torch.randn((self.total, hq, d), generator=g).to(self.dt).cuda()
        self.positions = torch.randint(-far, far, (axes, self.total), generator=g, dtype=torch.int32).cuda()
        self.pos = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([sum(rows[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        self.cache = y.make_cache(self.k, self.v, self.table)
        self.rope = y.make_rope(self.rotary, sections=None, interleaved=interleaved, axis=self.axis)
        self.rope.num_axes = axes

    def turn(self, x, err):
        """fp64 x [total][h][d] and a bound of its error -> turned, bound."""
        pairs = self.rotary // 2
        inv = torch.tensor([10000.0 ** (-2 * c / self.rotary) for c in range(pairs)], dtype=torch.float64, device="cuda")
        ang = self.positions.double()[self.axis].T * inv
        # fp64 keeps the fraction of the angle to 2^-53 * 2^31; the reference reduces first all the same
        ang = torch.remainder(ang, 2 * math.pi)
        cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        lo = slice(0, 2 * pairs, 2) if self.interleaved else slice(0, pairs)
        hi = slice(1, 2 * pairs, 2) if self.interleaved else slice(pairs, 2 * pairs)
        out, e = x.clone(), err.clone()
        a, b = x[..., lo], x[..., hi]
        out[..., lo], out[..., hi] = a * cos - b * sin, b * cos + a * sin
        t = 6 * 2.0 ** -24
        both = t * (a.abs() + b.abs()) + err[..., lo] + err[..., hi]
        e[..., lo], e[..., hi] = both, both
        return out, e

    def run(self, y, **kw):
        self.q_out = torch.full_like(self.q, 7.0)
        y.yocopp_rope_compose_append(*self.raw, ALPHA, LAM, self.rope, self.positions, self.cache, self.pos, q=self.q,
                                     q_out=self.q_out, cu_new=self.cu, **kw)
        return self

    def cells(self):
        """(token, page, slot) of every row."""
        t = 0
        for b, (p, n) in enumerate(zip(self.start, self.rows)):
            for j in range(n):
                at = p + j
                yield (t, int(self.table[b, at // self.block]), at % self.block) if self.block else (t, b, at)
                t += 1

    def check(self, y):
        torch.cuda.synchronize()
        assert y.yocopp_get_device_status(reset=True) == 0
        half = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        K1, V1, Ki, Vi = (x.double() for x in self.raw)
        a = [float(torch.tensor(x, dtype=torch.float32)) for x in ALPHA]
        x = LAM * (a[0] * K1 + a[1] * Ki)
        e = 2.0 ** -22 * LAM * ((a[0] * K1).abs() + (a[1] * Ki).abs())
        want, tol = self.turn(x, e)
        # values: those of the existing append
        k2, v2 = torch.full_like(self.k, 7.0), torch.full_like(self.v, 7.0)
        y.yocopp_compose_append(*self.raw, ALPHA, LAM, y.make_cache(k2, v2, self.table), self.pos, cu_new=self.cu)
        assert torch.equal(self.v, v2)
        written = torch.zeros(self.k.shape, dtype=torch.bool, device="cuda")
        for t, page, slot in self.cells():
            got = self.k[page, :, slot].double()
            assert bool(((got - want[t]).abs() <= tol[t] * 1.001 + half * want[t].abs() + 1e-38).all()), t
            written[page, :, slot] = True
        assert bool((self.k[~written] == 7).all())
        wq, tq = self.turn(self.q.double(), torch.zeros_like(self.q, dtype=torch.float64))
        assert bool(((self.q_out.double() - wq).abs() <= tq * 1.001 + half * wq.abs() + 1e-38).all())


TYPES = [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)]


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [None, 0.5, "odd", 2])
def test_pairs_and_layouts(y, dtype, d, interleaved, rotary):
    rotary = {None: d, 0.5: d // 2, "odd": d // 2 + 6, 2: 2}[rotary]
    Case(y, dtype=dtype, d=d, rotary=rotary, interleaved=interleaved, axes=min(3, rotary // 2), seed=1).run(y).check(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("block", [0, 16, 256])
def test_axes_and_caches(y, dtype, axes, block):
    Case(y, dtype=dtype, axes=axes, block=block, rows=(1, 40, 0, 7), start=(3, 0, 2, 11), seed=2).run(y).check(y)


def test_axes_in_any_order(y):
    Case(y, axes=4, axis=[(c * 7) % 4 for c in range(64)], seed=3).run(y).check(y)


@pytest.mark.parametrize("far", [1, 2 ** 31 - 1])
def test_near_and_far_positions(y, far):
    Case(y, dtype="f32", far=far, seed=4).run(y).check(y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(y, dtype):
    Case(y, dtype=dtype, rows=(3001, 17), start=(5, 0), hkv=3, hq=3, block=64, seed=5).run(y).check(y)


def test_position_zero_keeps_the_composition(y):
    c = Case(y, seed=6)
    c.positions.zero_()
    c.run(y)
    k2, v2 = torch.full_like(c.k, 7.0), torch.full_like(c.v, 7.0)
    y.yocopp_compose_append(*c.raw, ALPHA, LAM, y.make_cache(k2, v2, c.table), c.pos, cu_new=c.cu)
    torch.cuda.synchronize()
    # composed in fp32 and rounded once: within an ulp of the exact composition's rounding
    assert bool(((c.k.double() - k2.double()).abs() <= 2.0 ** -7 * k2.double().abs()).all())
    assert torch.equal(c.q_out, c.q)


def test_queries_alone_and_in_place(y):
    c = Case(y, seed=7).run(y)
    want = c.q_out.clone()
    before = c.k.clone()
    q = c.q.clone()
    y.yocopp_rope_compose_append(None, None, None, None, None, 0.0, c.rope, c.positions, c.cache, None, q=q, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(c.k, before)
    c2 = Case(y, seed=7)
    y.yocopp_rope_compose_append(*c2.raw, ALPHA, LAM, c2.rope, c2.positions, c2.cache, c2.pos, cu_new=c2.cu)
    torch.cuda.synchronize()
    assert torch.equal(c2.k, c.k)


def test_uniform_rows(y):
    c = Case(y, rows=(6, 6), start=(1, 20), seed=8)
    c.cu = None
    c.q_out = torch.empty_like(c.q)
    y.yocopp_rope_compose_append(*c.raw, ALPHA, LAM, c.rope, c.positions, c.cache, c.pos, q=c.q, q_out=c.q_out,
                                 n_uniform=6)
    c.cu = torch.tensor([0, 6, 12], dtype=torch.int32, device="cuda")
    c.check(y)


def test_rows_without_a_place_are_skipped(y):
    c = Case(y, rows=(5, 3), start=(0, 9), block=16, seed=9)
    good = Case(y, rows=(5, 3), start=(0, 9), block=16, seed=9).run(y)
    c.table[0, 0] = c.k.shape[0]
    c.run(y)
    torch.cuda.synchronize()
    assert y.yocopp_get_device_status(reset=True) == y.YOCOPP_EDEVICE_CHECK
    blk = int(good.table[0, 0])
    assert bool((c.k[blk] == 7).all()) and torch.equal(c.q_out, good.q_out)
    blk = int(good.table[1, 0])
    assert torch.equal(c.k[blk], good.k[blk])
    for p in (-1, 10 ** 6, 2 ** 31 - 2):
        c.pos[1] = p
        c.run(y)
        torch.cuda.synchronize()
        assert y.yocopp_get_device_status(reset=True) in (y.YOCOPP_ECAPACITY, y.YOCOPP_EDEVICE_CHECK)


def test_graph_replay(y):
    c = Case(y, seed=10).run(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(y)
    for x in c.raw + [c.q]:
        x.copy_(x.roll(1, 0))
    c.positions.add_(5)
    g.replay()
    c.check(y)


def test_offsets_past_32_bits(y):
    c = Case(y, hkv=8, block=64, rows=(5, 70), start=(0, 9), seed=11)
    blocks = (5 << 30) // (8 * 64 * 128 * 2)
    k = torch.empty((blocks, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    big = c.table + (blocks - c.k.shape[0])
    k[blocks - c.k.shape[0]:], v[blocks - c.k.shape[0]:] = 7.0, 7.0
    c.cache = y.make_cache(k, v, big)
    c.run(y)
    torch.cuda.synchronize()
    c.k.copy_(k[blocks - c.k.shape[0]:])
    c.v.copy_(v[blocks - c.v.shape[0]:])
    c.check(y)
