"""Bad calls of the serving operators are refused before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

from long_context_decoding_saga_b200 import build as build_mod
from long_context_decoding_saga_b200 import saga

FAKE = 0x100000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return saga.load()


def _shape(**kw):
    base = dict(batch=1, h_q=8, h_k=1, h_v=8, d=64, l_cap=1024)
    base.update(kw)
    return saga.SagaShape.of(**base)


def _cache(fmt=1, **kw):
    base = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, format=fmt)
    base.update(kw)
    return saga._Cache(*(base[n] for n in ("k", "v", "k_scale", "v_scale", "format")))


def _rows(heads, d=64, **kw):
    base = dict(data=FAKE, batch_stride=0, token_stride=heads * d, head_stride=d)
    base.update(kw)
    return saga._Rows(base["data"], base["batch_stride"], base["token_stride"], base["head_stride"])


def _op(**kw):
    base = dict(norm=1, eps=1e-6, q_weight=FAKE, k_weight=FAKE, inv_freq=FAKE, rot_dim=64, interleaved=0)
    base.update(kw)
    return saga._NormRope(*(base[n] for n in ("norm", "eps", "q_weight", "k_weight", "inv_freq", "rot_dim", "interleaved")))


def _append(lib, shape=None, tokens=2, q=None, k=None, v=None, op=None, starts=FAKE, q_out=FAKE, cache=None):
    ref = ctypes.byref
    return lib.saga_norm_rope_append(ref(shape or _shape()), tokens, ref(q or _rows(8)), ref(k or _rows(1)),
                                     ref(v or _rows(8)), ref(op or _op()), starts, None, None, q_out,
                                     ref(cache or _cache()), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(shape=_shape(d=96)), saga.SAGA_ERR_UNSUPPORTED),
    (dict(shape=_shape(h_q=6, h_k=4)), saga.SAGA_ERR_ARG),
    (dict(tokens=0), saga.SAGA_ERR_ARG),
    (dict(tokens=1025), saga.SAGA_ERR_ARG),
    (dict(q=_rows(8, data=None)), saga.SAGA_ERR_ARG),
    (dict(q=_rows(8, data=FAKE + 8)), saga.SAGA_ERR_ARG),
    (dict(q=_rows(8, head_stride=60)), saga.SAGA_ERR_ARG),
    (dict(k=_rows(1, token_stride=68)), saga.SAGA_ERR_ARG),
    (dict(v=_rows(8, batch_stride=-8)), saga.SAGA_ERR_ARG),
    (dict(op=_op(rot_dim=0)), saga.SAGA_ERR_ARG),
    (dict(op=_op(rot_dim=24)), saga.SAGA_ERR_ARG),
    (dict(op=_op(rot_dim=80)), saga.SAGA_ERR_ARG),
    (dict(op=_op(eps=-1.0)), saga.SAGA_ERR_ARG),
    (dict(op=_op(eps=float("nan"))), saga.SAGA_ERR_ARG),
    (dict(op=_op(q_weight=FAKE + 2)), saga.SAGA_ERR_ARG),
    (dict(starts=None), saga.SAGA_ERR_ARG),
    (dict(q_out=None), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(k=None)), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(v=FAKE + 8)), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(fmt=2)), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(k_scale=None)), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(v_scale=FAKE + 2)), saga.SAGA_ERR_ARG),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code
    assert lib.saga_last_error()


@pytest.mark.parametrize("q", [_rows(8, head_stride=128, token_stride=1024), _rows(8, token_stride=640)])
def test_in_place_needs_dense_queries(lib, q):
    assert _append(lib, q=q) == saga.SAGA_ERR_ARG
    assert b"dense" in lib.saga_last_error()


def test_status_must_be_aligned(lib):
    ref = ctypes.byref
    assert lib.saga_kv_store(ref(_shape()), 2, ref(_rows(1)), ref(_rows(8)), FAKE, None, ref(_cache()), FAKE + 2,
                             None) == saga.SAGA_ERR_ARG
    assert b"status" in lib.saga_last_error()


def test_load_refusals(lib):
    ref, s = ctypes.byref, _shape()
    call = lambda cache=_cache(), start=0, rows=4, ko=FAKE, vo=FAKE: lib.saga_kv_load(ref(s), ref(cache), start, rows, None, ko, vo, None)
    for kw in (dict(cache=_cache(fmt=0)), dict(start=-1), dict(rows=0), dict(start=1021), dict(ko=None, vo=None),
               dict(ko=FAKE + 8)):
        assert call(**kw) == saga.SAGA_ERR_ARG, kw
        assert lib.saga_last_error()
    assert lib.saga_kv_load(ref(_shape(batch=8192)), ref(_cache()), 0, 4, None, FAKE, FAKE, None) == saga.SAGA_ERR_UNSUPPORTED


def _tree(lib, shape=None, tokens=4, q=FAKE, cache=None, prefix=FAKE, out=FAKE, dtype=0, ws=FAKE, ws_bytes=1 << 40):
    ref = ctypes.byref
    return lib.saga_tree_attn(ref(shape or _shape()), tokens, q, ref(cache or _cache()), prefix, None, None, None, out,
                              dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(shape=_shape(d=32)), saga.SAGA_ERR_UNSUPPORTED),
    (dict(shape=_shape(batch=0)), saga.SAGA_ERR_ARG),
    (dict(tokens=0), saga.SAGA_ERR_ARG),
    (dict(tokens=65), saga.SAGA_ERR_ARG),
    (dict(shape=_shape(l_cap=3)), saga.SAGA_ERR_ARG),
    (dict(q=None), saga.SAGA_ERR_ARG),
    (dict(q=FAKE + 8), saga.SAGA_ERR_ARG),
    (dict(out=FAKE + 4), saga.SAGA_ERR_ARG),
    (dict(prefix=None), saga.SAGA_ERR_ARG),
    (dict(dtype=5), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(fmt=7)), saga.SAGA_ERR_ARG),
    (dict(cache=_cache(v_scale=None)), saga.SAGA_ERR_ARG),
])
def test_tree_refusals(lib, kw, code):
    assert _tree(lib, **kw) == code
    assert lib.saga_last_error()


def test_tree_workspace_refusals(lib):
    assert _tree(lib, ws=None) == saga.SAGA_ERR_WORKSPACE
    assert _tree(lib, ws=FAKE + 16) == saga.SAGA_ERR_WORKSPACE
    assert lib.saga_tree_workspace_bytes(ctypes.byref(_shape()), 0) == 0
    assert lib.saga_tree_workspace_bytes(ctypes.byref(_shape(d=96)), 1) == 0


def test_binding_refusals(lib):
    s = _shape()
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        saga.alloc_cache(s, saga.SAGA_CACHE_E4M3, device="cpu")
    with pytest.raises(ValueError):
        saga.KVCache(bf(1, 1, 4, 64), bf(1, 8, 4, 64))
    with pytest.raises(ValueError):  # one scale of two
        saga.KVCache(bf(1, 1, 4, 64), bf(1, 8, 4, 64), torch.zeros(1, 1, 4), None)
    with pytest.raises(ValueError):
        saga.KVCache(bf(1, 4, 64), bf(1, 8, 4, 64))
    with pytest.raises(ValueError):
        saga.alloc_cache(s, 9, device="cpu")
    with pytest.raises(TypeError):  # caches are described by a KVCache
        saga.saga_kv_store(s, bf(1, 2, 1, 64), bf(1, 2, 8, 64), (bf(1, 1, 4, 64), bf(1, 8, 4, 64)), None)


@pytest.mark.gpu
def test_binding_refusals_of_cuda_tensors():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s = saga.SagaShape.of(2, 8, 1, 8, 64, 32)
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
    cache = saga.alloc_cache(s, saga.SAGA_CACHE_E4M3)
    starts, q = z(2, dtype=torch.int32), z(2, 3, 8, 64)
    k, v = z(2, 3, 1, 64), z(2, 3, 8, 64)
    saga.saga_kv_store(s, k, v, cache, starts)  # in order
    ws = saga.alloc_tree_workspace(s, 3)
    saga.saga_tree_attn(s, q, cache, starts, torch.empty_like(q), ws)
    store = lambda **kw: saga.saga_kv_store(kw.pop("s", s), kw.pop("k", k), kw.pop("v", v), kw.pop("cache", cache),
                                            kw.pop("starts", starts), **kw)
    tree = lambda **kw: saga.saga_tree_attn(s, kw.pop("q", q), cache, kw.pop("pl", starts),
                                            kw.pop("out", torch.empty_like(q)), kw.pop("ws", ws), **kw)
    with pytest.raises(ValueError):  # another shape's cache
        store(s=saga.SagaShape.of(2, 8, 1, 8, 64, 33))
    with pytest.raises(TypeError):
        store(k=k.float())
    with pytest.raises(ValueError):
        store(k=k.cpu())
    with pytest.raises(ValueError):
        store(k=z(2, 3, 2, 64))
    with pytest.raises(ValueError):  # elements of a head not dense
        store(k=z(2, 3, 64, 2).transpose(2, 3)[:, :, :1])
    with pytest.raises(TypeError):
        store(starts=starts.long())
    with pytest.raises(ValueError):
        store(starts=None)
    with pytest.raises(ValueError):
        store(counts=z(3, dtype=torch.int32))
    with pytest.raises(saga.SagaError):  # more tokens than rows
        store(k=z(2, 33, 1, 64), v=z(2, 33, 8, 64))
    with pytest.raises(saga.SagaError):  # strides of 4 elements
        store(k=torch.zeros(2 * 3 * 68, dtype=torch.bfloat16, device="cuda").as_strided((2, 3, 1, 64), (204, 68, 64, 1)))
    with pytest.raises(TypeError):
        tree(out=q.half())
    with pytest.raises(ValueError):
        tree(out=torch.empty((2, 3, 8, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        tree(q=z(2, 3, 16, 64)[:, :, ::2])
    with pytest.raises(TypeError):
        tree(tree_mask=z(2, 3, dtype=torch.int32))
    with pytest.raises(TypeError):
        tree(tau=z(2, 8))
    with pytest.raises(saga.SagaError):
        tree(ws=ws[:256])
    with pytest.raises(saga.SagaError):
        saga.saga_kv_load(s, saga.alloc_cache(s), 0, 4, z(2, 1, 4, 64))  # a bf16 cache
    with pytest.raises(ValueError):
        saga.saga_norm_rope_append(s, q, k, v, cache, starts, q.clone(), q_weight=z(64))  # a weight, no norm
    torch.cuda.synchronize()
    assert saga.saga_get_status(ws) == 0


def test_packed_structures_are_the_headers():
    """The binding's packed strings have the layout of the C structures."""
    import struct
    rows = saga._Rows.from_buffer_copy(saga._pack_rows(FAKE, 1 << 40, 8, 64))
    assert struct.calcsize("@Pqqq") == ctypes.sizeof(saga._Rows)
    assert (rows.data, rows.batch_stride, rows.token_stride, rows.head_stride) == (FAKE, 1 << 40, 8, 64)
    op = saga._NormRope.from_buffer_copy(saga._pack_norm_rope(1, 0.5, FAKE, 0, FAKE + 16, 64, 1))
    assert struct.calcsize("@ifPPPii") == ctypes.sizeof(saga._NormRope)
    assert (op.norm, op.eps, op.q_weight, op.k_weight, op.inv_freq, op.rot_dim, op.interleaved) == \
        (1, 0.5, FAKE, None, FAKE + 16, 64, 1)
