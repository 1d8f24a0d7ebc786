"""Argument checks of the chunk attention, the rotary append and the page
operators, without a GPU: status codes of the C ABI and errors of the binding."""
import ctypes

import pytest
import torch

import decode_attention_yocopp_b200 as y


def _cache(**kw):
    c = y.yocopp_cache()
    c.k, c.v = 0x1000, 0x2000
    c.dtype, c.batch, c.num_kv_heads, c.head_dim, c.capacity = y.YOCOPP_BF16, 2, 8, 128, 64
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _paged(**kw):
    return _cache(**{**dict(block_table=0x3000, block_size=32, max_blocks_per_seq=2, num_blocks=4), **kw})


def _chunk(c=None, q=0x10, pos=0x10, cu=None, n=4, total=8, max_q=0, tree=None, window=0, out=0x20, hq=32, scale=0.0,
           ws=0x100, nbytes=1 << 40):
    return y.load().yocopp_chunk_attn(q, ctypes.byref(c or _cache()), pos, cu, n, total, max_q, tree, window, out, hq,
                                      scale, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(hq=12), dict(hq=0), dict(hq=-8), dict(q=None), dict(q=0x18), dict(out=None), dict(out=0x28), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(total=-1), dict(total=9), dict(n=-1), dict(n=65, total=130),
    dict(cu=0x20, max_q=-1), dict(cu=0x20, max_q=65), dict(window=-1), dict(tree=0x20, window=5),
    dict(tree=0x24), dict(c=_cache(head_dim=96)), dict(c=_cache(k=0x1008)), dict(c=_paged(block_size=48)),
    dict(c=_cache(capacity=1 << 28)), dict(tree=0x20, c=_cache(capacity=256), n=65, total=130),
    dict(c=_cache(capacity=1 << 20), hq=8 << 12, n=1 << 19, total=1 << 20),
])
def test_chunk_refusals(kw):
    assert _chunk(**kw) == y.YOCOPP_EINVAL


def test_chunk_dtype_and_size():
    assert _chunk(c=_cache(dtype=5)) == y.YOCOPP_EDTYPE
    lib = y.load()
    assert lib.yocopp_chunk_attn_workspace_size(ctypes.byref(_cache()), 12) == y.YOCOPP_EINVAL
    assert lib.yocopp_chunk_attn_workspace_size(ctypes.byref(_cache(batch=0)), 8) == y.YOCOPP_EINVAL
    assert lib.yocopp_chunk_attn_workspace_size(None, 8) == y.YOCOPP_EINVAL


def _rope_call(rope, c=None, raw=(0x10, 0x10, 0x10, 0x10), alpha=(0.1, 0.2, 0.3, 0.4), lam=35.0, positions=0x10, pos=0x10,
               q=0x20, qo=0x30, hq=8, cu=None, n=1, total=2):
    a = None if alpha is None else (ctypes.c_float * 4)(*alpha)
    return y.load().yocopp_rope_compose_append(*raw, a, lam, ctypes.byref(rope) if rope is not None else None, positions,
                                               ctypes.byref(c or _cache()), pos, q, qo, hq, cu, n, total, None)


def _bad_rope(**kw):
    r = y.make_rope(128, sections=[32, 16, 16])
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(r, k)[v[0]] = v[1]
        else:
            setattr(r, k, v)
    return r


@pytest.mark.parametrize("rope", [
    None, _bad_rope(rotary_dim=0), _bad_rope(rotary_dim=7), _bad_rope(rotary_dim=130), _bad_rope(interleaved=2),
    _bad_rope(num_axes=0), _bad_rope(num_axes=5), _bad_rope(num_axes=2), _bad_rope(axis=(3, -1)),
    _bad_rope(inv_freq=(63, float("nan")))])
def test_rope_descriptor_refusals(rope):
    assert _rope_call(rope) == y.YOCOPP_EINVAL


@pytest.mark.parametrize("kw", [
    dict(raw=(None, 0x10, 0x10, 0x10)), dict(raw=(0x10, 0x10, 0x10, None)), dict(raw=(0x10, 0x18, 0x10, 0x10)),
    dict(alpha=None), dict(alpha=(float("inf"), 0, 0, 0)), dict(lam=float("nan")), dict(positions=None), dict(pos=None),
    dict(q=None), dict(qo=None), dict(q=0x28), dict(qo=0x38), dict(hq=0), dict(hq=(1 << 20) + 1), dict(n=2), dict(total=-1), dict(total=1 << 31),
    dict(raw=(None,) * 4, q=None, qo=None), dict(c=_cache(head_dim=64))])
def test_rope_refusals(kw):
    assert _rope_call(_bad_rope(), **kw) == y.YOCOPP_EINVAL


def test_rope_nothing_to_do():
    assert _rope_call(_bad_rope(), n=0, total=0) == y.YOCOPP_OK
    assert _rope_call(_bad_rope(), c=_cache(dtype=9)) == y.YOCOPP_EDTYPE


def test_make_rope():
    r = y.make_rope(20, base=100.0, sections=[4, 3, 3], interleaved=True)
    assert (r.rotary_dim, r.interleaved, r.num_axes) == (20, 1, 3)
    assert list(r.axis[:10]) == [0] * 4 + [1] * 3 + [2] * 3
    assert r.inv_freq[5] == pytest.approx(0.1, rel=1e-15) and r.inv_freq[0] == 1.0
    r = y.make_rope(8, axis=[1, 0, 1, 0], inv_freq=[1, 2, 3, 4])
    assert r.num_axes == 2 and list(r.axis[:4]) == [1, 0, 1, 0] and r.inv_freq[3] == 4.0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=130), dict(rotary_dim=8, sections=[3]),
                dict(rotary_dim=8, inv_freq=[1.0]), dict(rotary_dim=8, sections=[4], axis=[0] * 4)):
        with pytest.raises(ValueError):
            y.make_rope(**bad)


def _pages(caches=None, count=None, refs=0x10, a=0x10, lens=0x10, n=1, held=0x10, ws=0x100, nbytes=1 << 40):
    c = y.cache_list(caches or [_paged(), _paged()])
    return y.load().yocopp_pages_resize(c, len(c) if count is None else count, refs, a, lens, n, held, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(caches=[_cache()]), dict(count=0), dict(caches=[_paged()] * 129), dict(caches=[_paged(), _paged(num_blocks=5)]),
    dict(caches=[_paged(), _paged(num_kv_heads=4)]), dict(caches=[_paged(), _paged(block_table=0x3010)]),
    dict(caches=[_paged(), _paged(dtype=1)]), dict(caches=[_paged(block_table=0x3002)]), dict(refs=None), dict(a=None),
    dict(lens=None), dict(held=None), dict(n=-1), dict(n=3)])
def test_pages_refusals(kw):
    assert _pages(**kw) == y.YOCOPP_EINVAL


def test_pages_workspace_and_others():
    need = y.yocopp_pages_workspace_size(y.cache_list([_paged()]))
    assert need > 0
    for ws, nbytes in ((None, need), (0x180, need), (0x100, need - 1)):
        assert _pages(caches=[_paged()], ws=ws, nbytes=nbytes) == y.YOCOPP_EWORKSPACE
    assert _pages(n=0, a=None, lens=None, held=None) == y.YOCOPP_OK
    lib, c = y.load(), y.cache_list([_paged()])
    assert lib.yocopp_pages_fork(c, 1, 0x10, 0x10, 0x10, 0x10, 1, 2, 0x10, 0x100, need, None) == y.YOCOPP_EINVAL
    assert lib.yocopp_pages_fork(c, 1, 0x10, 0x10, None, 0x10, 1, 0, 0x10, 0x100, need, None) == y.YOCOPP_EINVAL
    assert lib.yocopp_pages_fork(c, 1, 0x10, 0x10, 0x10, 0x10, 1, 0, 0x10, 0x100, need - 1, None) == y.YOCOPP_EWORKSPACE
    assert lib.yocopp_pages_compact(c, 1, None, 0x10, 0x100, need, None) == y.YOCOPP_EINVAL
    assert lib.yocopp_pages_compact(c, 1, 0x10, None, 0x100, need, None) == y.YOCOPP_EINVAL


def test_binding_refuses_tensors_that_do_not_fit():
    c = _cache()
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    ok = dict(pos=torch.zeros(2, dtype=torch.int32), n_uniform=1)
    for bad_q, kw in ((q.float(), {}), (q[:, :, :64], {}), (q.transpose(0, 1), {}), (q, dict(pos=torch.zeros(2))),
                      (q, dict(tree_mask=torch.zeros(2, dtype=torch.int32)))):
        with pytest.raises(TypeError):
            y.yocopp_chunk_attn(bad_q, c, torch.zeros_like(bad_q), None, **{**ok, **kw})
    with pytest.raises(TypeError):
        y.yocopp_chunk_attn(q, c, torch.zeros((2, 16, 128), dtype=torch.bfloat16), None, **ok)
    r = y.make_rope(128, sections=[40, 24])
    with pytest.raises(TypeError):  # one axis of positions for two
        y.yocopp_rope_compose_append(q, q, q, q, (0, 1, 0, 1), 1.0, r, torch.zeros((1, 2), dtype=torch.int32), c,
                                     torch.zeros(2, dtype=torch.int32), n_uniform=1)
    with pytest.raises(TypeError):  # host tensors
        y.yocopp_chunk_attn(q, c, torch.zeros_like(q), None, **ok)
    caches = y.cache_list([_paged()])
    i = torch.zeros(1, dtype=torch.int32)
    for refs, lens in ((torch.zeros(3, dtype=torch.int32), i), (torch.zeros(4), i),
                       (torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(TypeError):
            y.yocopp_pages_resize(caches, refs, i, lens, i, i)
