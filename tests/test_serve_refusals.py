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
    cpu_cache = saga.alloc_cache(s, saga.SAGA_CACHE_E4M3, device="cpu")
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        saga.saga_kv_store(s, bf(1, 2, 1, 64), bf(1, 2, 8, 64), cpu_cache, i32)
    with pytest.raises(TypeError):
        saga.saga_kv_store(s, torch.zeros(1, 2, 1, 64), bf(1, 2, 8, 64), cpu_cache, i32)
    with pytest.raises(ValueError):
        saga.saga_kv_store(s, bf(1, 2, 64), bf(1, 2, 8, 64), cpu_cache, i32)
    with pytest.raises(ValueError):
        saga.KVCache(bf(1, 1, 4, 64), bf(1, 8, 4, 64), torch.zeros(1, 1, 4), None)
    with pytest.raises(ValueError):
        saga.alloc_cache(s, 9, device="cpu")
