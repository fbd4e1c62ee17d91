"""Norm, rotation, append, 8-bit store and load on the GPU against float64.

Bounds, element by element.  Norm: the sum of squares has at most D / 8 + 5 roundings of 2^-24 (half of it through
the root), the reciprocal root and the two products 6 more: under 17 * 2^-24.  Rotation: a turn's fraction is
rounded to fp32 (2 pi 2^-25), its sine and cosine are good to 2^-22, the products and the sum add 2 * 2^-24.  All of
it is under 2^-19 (|a| + |b|) for the pair (a, b), and one rounding to bf16 adds 2^-8 of the value.  The 8-bit
scale inherits 2 * 2^-19 (|a| + |b| is at most twice the row's largest rotated element), so a stored value is off by
half a code step, 2^-4 of it or 2^-10 scales, and by 2^-17 of the row's largest.  Rows that are neither normed nor
rotated are exact: the scale and the code are single fp32 operations that numpy repeats.
"""
import numpy as np
import pytest
import torch

from long_context_decoding_saga_b200 import saga
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decoding_saga_b200 import build
    build.build()
    saga.load()


def _cache(shape, fmt, g):
    """A cache full of junk that must survive outside the appended rows."""
    c = saga.alloc_cache(shape, fmt)
    for t in c._tensors():
        if t is not None:
            t.view(torch.uint8).copy_(torch.randint(0, 120, t.view(torch.uint8).shape, generator=g).to(torch.uint8))
    return c


def _bytes(c):
    return [None if t is None else t.view(torch.uint8).cpu().numpy().copy() for t in c._tensors()]


def _quantise_exactly(x):
    """fp32 scale and code values of rows x (float64 values of bf16), with the library's single fp32 operations."""
    amax = np.maximum(np.abs(x).max(-1), so.AMAX_FLOOR).astype(np.float32)
    up = np.float32(448) / amax
    y = x.astype(np.float32) * up[..., None]
    codes = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    return codes, amax / np.float32(448)


def _positions(B, T, g, far):
    return torch.randint(0, far, (B, T), generator=g, dtype=torch.int32)


def _check(B, T, heads, fmt, rot, interleaved, norm, weights, counts, packed, seed, far=200000, eps=1e-6, starts=None,
           default_positions=False, in_place=False):
    h_q, h_k, h_v, d = heads
    l_cap = T + 37
    shape = saga.SagaShape.of(B, h_q, h_k, h_v, d, l_cap)
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, T, h_q + h_k + h_v, d), generator=g) *
         torch.exp(2 * torch.randn((B, T, h_q + h_k + h_v, 1), generator=g))).to(torch.bfloat16)
    xg = x.cuda()
    q, k, v = xg[:, :, :h_q], xg[:, :, h_q:h_q + h_k], xg[:, :, h_q + h_k:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    starts = torch.randint(0, l_cap - T + 1, (B,), generator=g, dtype=torch.int32) if starts is None else starts
    pos = _positions(B, T, g, far)
    inv = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None
    qw = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16) if weights else None
    kw = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16) if weights else None
    cache = _cache(shape, fmt, g)
    before = _bytes(cache)
    q_out = q if in_place else torch.full((B, T, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cd = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    saga.saga_norm_rope_append(shape, q, k, v, cache, starts.cuda(), q_out,
                               positions=None if default_positions else pos.cuda(), counts=cd, norm=norm,
                               q_weight=None if qw is None else qw.cuda(), k_weight=None if kw is None else kw.cuda(),
                               eps=eps, inv_freq=None if inv is None else inv.cuda(), interleaved=interleaved,
                               status=status)
    torch.cuda.synchronize()
    after = _bytes(cache)
    xe = x.double().numpy()
    n = [T] * B if counts is None else [min(max(c, 0), T) for c in counts]
    clamped = False
    touched = [np.zeros((B, h, l_cap), bool) for h in (h_k, h_v)]
    for b in range(B):
        rows = np.arange(n[b]) + int(starts[b])
        p = rows if default_positions else pos[b, :n[b]].numpy()
        here = (rows >= 0) & (rows < l_cap)
        clamped |= bool((~here).any())
        for name, lo, h, w in (("q", 0, h_q, qw), ("k", h_q, h_k, kw), ("v", h_q + h_k, h_v, None)):
            a = xe[b, :n[b], lo:lo + h]
            pair = np.zeros_like(a)
            if name != "v":
                if norm:
                    a = so.norm(a, None if w is None else w.double().numpy(), eps)
                if inv is not None:
                    fr = inv.double().numpy()
                    i = np.arange(rot // 2)
                    f, s = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                    pair[..., f], pair[..., s] = a[..., s], a[..., f]
                    e = 2.0 ** -19 * (np.abs(a) + np.abs(pair))
                    a = so.rotate(a, p, fr, interleaved)
                else:
                    e = 2.0 ** -19 * np.abs(a)
            else:
                e = np.zeros_like(a)
            if name == "q":
                got = q_out[b, :n[b]].double().cpu().numpy()
                assert (np.abs(got - a) <= 2.0 ** -8 * (np.abs(a) + e) + e).all()
                continue
            ci = 0 if name == "k" else 1
            touched[ci][b][:, rows[here]] = True
            a, e = a[here].transpose(1, 0, 2), e[here].transpose(1, 0, 2)  # [h, rows, d]
            stored = cache._tensors()[ci][b][:, rows[here]].double().cpu().numpy()
            if fmt == saga.SAGA_CACHE_BF16:
                assert (np.abs(stored - a) <= 2.0 ** -8 * (np.abs(a) + e) + e).all()
                if name == "v":
                    assert np.array_equal(stored, a)
                continue
            scale = cache._tensors()[2 + ci][b][:, rows[here]].cpu().numpy()
            if name == "v" or not (norm or rot):
                codes, exact_scale = _quantise_exactly(a)
                assert np.array_equal(scale, exact_scale) and np.array_equal(stored, codes)
            exact = so.row_scale(a)
            assert (np.abs(scale - exact) <= 2.0 ** -17 * exact).all()
            step = np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * exact[..., None])
            assert (np.abs(stored * scale[..., None].astype(np.float64) - a) <=
                    step + 2.0 ** -16 * 448 * exact[..., None]).all()
        absent = q_out[b, n[b]:].double().cpu().numpy()
        kept = x[b, n[b]:, :h_q].double().numpy() if in_place else np.full_like(absent, 7.0)
        assert np.array_equal(absent, kept)
    for i, (old, new) in enumerate(zip(before, after)):
        if old is None:
            continue
        mask = touched[i % 2]
        old, new = old.reshape(mask.shape + (-1,)), new.reshape(mask.shape + (-1,))
        assert np.array_equal(old[~mask], new[~mask]), "a row that no token owns changed"
    assert saga.saga_get_status(status) == (saga.SAGA_STATUS_LEN_CLAMPED if clamped else 0)


HEADS = [(8, 1, 8, 64), (12, 1, 4, 128), (32, 2, 8, 64), (16, 4, 2, 64), (3, 3, 1, 128), (1, 1, 1, 64)]
FMTS = [saga.SAGA_CACHE_BF16, saga.SAGA_CACHE_E4M3]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("B,T", [(1, 1), (3, 5), (2, 130)])
def test_norm_and_rotation(heads, fmt, B, T):
    _check(B, T, heads, fmt, heads[3], False, True, True, None, False, 10 * T + heads[0])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 112])
def test_partial_rotation(rot, interleaved, fmt):
    _check(2, 7, (12, 1, 4, 128), fmt, rot, interleaved, False, False, None, True, 77 + rot)


@pytest.mark.parametrize("norm,weights", [(True, False), (True, True), (False, False)])
def test_norm_with_and_without_weights(norm, weights):
    _check(2, 9, (32, 4, 8, 64), saga.SAGA_CACHE_BF16, 64, True, norm, weights, None, True, 5, eps=0.5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[0, 3, 9, 20, -4], [9, 9, 9, 9, 9], [0, 0, 0, 0, 0]])
def test_ragged_batches(counts, fmt):
    _check(5, 9, (12, 1, 4, 128), fmt, 128, False, True, True, counts, True, 6)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_outside_the_cache_are_dropped_and_flagged(fmt):
    starts = torch.tensor([-3, 40, 2 ** 31 - 2, 41, -2 ** 31], dtype=torch.int32)
    _check(5, 6, (8, 1, 8, 64), fmt, 64, False, True, True, None, False, 8, starts=starts)


def test_positions_default_to_the_cache_row():
    _check(2, 11, (32, 2, 8, 64), saga.SAGA_CACHE_BF16, 64, False, False, False, None, True, 9, default_positions=True)


def test_far_positions():
    _check(1, 33, (12, 1, 4, 128), saga.SAGA_CACHE_BF16, 128, False, False, False, None, False, 10, far=2 ** 31 - 1)


@pytest.mark.parametrize("counts", [None, [3, 0]])
def test_in_place(counts):
    _check(2, 6, (32, 2, 8, 64), saga.SAGA_CACHE_BF16, 64, False, True, True, counts, False, 11, in_place=True)


@pytest.mark.parametrize("tokens", [4099, 9001])
def test_many_tokens(tokens):
    _check(1, tokens, (2, 1, 1, 64), saga.SAGA_CACHE_E4M3, 64, False, True, True, None, True, 12)


def _store_case(B, T, heads, fmt, values, counts=None):
    h_q, h_k, h_v, d = heads
    l_cap = T + 5
    shape = saga.SagaShape.of(B, h_q, h_k, h_v, d, l_cap)
    cache = _cache(shape, fmt, torch.Generator().manual_seed(1))
    k, v = values(B, T, h_k, d), values(B, T, h_v, d)
    starts = torch.arange(B, dtype=torch.int32) % 5
    cd = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    saga.saga_kv_store(shape, k.cuda(), v.cuda(), cache, starts.cuda(), counts=cd)
    torch.cuda.synchronize()
    return shape, cache, k, v, starts


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("B,T", [(1, 1), (4, 3), (2, 257)])
def test_store_and_load(heads, B, T):
    g = torch.Generator().manual_seed(T)
    values = lambda B, T, h, d: (torch.randn((B, T, h, d), generator=g) *
                                 torch.exp(4 * torch.randn((B, T, h, 1), generator=g))).to(torch.bfloat16)
    shape, cache, k, v, starts = _store_case(B, T, heads, saga.SAGA_CACHE_E4M3, values)
    for ci, x in enumerate((k, v)):
        codes, scale = _quantise_exactly(x.double().numpy())
        for b in range(B):
            lo = int(starts[b])
            got = cache._tensors()[ci][b, :, lo:lo + T].double().cpu().numpy()
            assert np.array_equal(got, codes[b].transpose(1, 0, 2))
            assert np.array_equal(cache._tensors()[2 + ci][b, :, lo:lo + T].cpu().numpy(), scale[b].T)
    l_cap = shape.l_cap
    for start, rows in ((0, l_cap), (3, T), (l_cap - 1, 1)):
        h_k, h_v, d = heads[1:]
        ko = torch.full((B, h_k, rows, d), 3.0, dtype=torch.bfloat16, device="cuda")
        vo = torch.full((B, h_v, rows, d), 3.0, dtype=torch.bfloat16, device="cuda")
        lens = torch.tensor([(b * T) // 2 + start for b in range(B)], dtype=torch.int32)
        saga.saga_kv_load(shape, cache, start, rows, ko, vo, lens=lens.cuda())
        only = torch.empty_like(vo)
        saga.saga_kv_load(shape, cache, start, rows, v_out=only)
        for ci, o in enumerate((ko, vo)):
            codes = cache._tensors()[ci][:, :, start:start + rows].float().cpu().numpy()
            scale = cache._tensors()[2 + ci][:, :, start:start + rows].cpu().numpy()
            want = torch.from_numpy(codes * scale[..., None]).to(torch.bfloat16)  # one fp32 product, one rounding
            for b in range(B):
                n = max(0, min(rows, int(lens[b]) - start))
                assert torch.equal(o[b, :, :n].cpu(), want[b, :, :n])
                assert (o[b, :, n:] == 3.0).all()
            if ci == 1:
                assert torch.equal(only.cpu(), want)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -120, 2.0 ** -100, 1.5, 3.0e38, -2.0 ** 100])
def test_store_of_constant_rows(value):
    """Rows of zeros, of magnitudes below the floor and of the largest ones: finite codes, exact where the largest
    magnitude is every element's."""
    fill = lambda B, T, h, d: torch.full((B, T, h, d), value).to(torch.bfloat16)
    shape, cache, k, v, starts = _store_case(1, 3, (8, 1, 8, 64), saga.SAGA_CACHE_E4M3, fill)
    x = k.double().numpy()
    codes, scale = _quantise_exactly(x)
    got = cache.k[0, :, :3].double().cpu().numpy()
    assert np.isfinite(got).all() and np.array_equal(got, codes[0].transpose(1, 0, 2))
    assert np.isfinite(cache.k_scale[0, :, :3].cpu().numpy()).all()
    if abs(x.flat[0]) >= so.AMAX_FLOOR:
        back = got * cache.k_scale[0, :, :3, None].double().cpu().numpy()
        assert (np.abs(back - x[0].transpose(1, 0, 2)) <= 2.0 ** -22 * np.abs(x.flat[0])).all()


def test_store_into_bf16_matches_the_one_token_append():
    heads = (32, 2, 8, 64)
    g = torch.Generator().manual_seed(3)
    values = lambda B, T, h, d: torch.randn((B, T, h, d), generator=g).to(torch.bfloat16)
    shape, cache, k, v, starts = _store_case(2, 1, heads, saga.SAGA_CACHE_BF16, values)
    for b in range(2):
        one = saga.SagaShape.of(1, *heads, shape.l_cap)
        c = saga.alloc_cache(one)
        saga.saga_kv_append(one, c.k, c.v, k[b:b + 1, 0].cuda().contiguous(), v[b:b + 1, 0].cuda().contiguous(),
                            int(starts[b]))
        assert torch.equal(c.k[0, :, int(starts[b])], cache.k[b, :, int(starts[b])])
        assert torch.equal(c.v[0, :, int(starts[b])], cache.v[b, :, int(starts[b])])


def test_captured_append_follows_device_lengths():
    heads, T = (12, 1, 4, 128), 3
    shape = saga.SagaShape.of(2, *heads, 64)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((2, T, 17, 128), generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :, :12], x[:, :, 12:13], x[:, :, 13:]
    inv = (10000.0 ** (-torch.arange(0, 128, 2) / 128)).float().cuda()
    q_out = torch.zeros((2, T, 12, 128), dtype=torch.bfloat16, device="cuda")
    cache, starts, counts = saga.alloc_cache(shape, saga.SAGA_CACHE_E4M3), torch.zeros(2, dtype=torch.int32).cuda(), \
        torch.full((2,), T, dtype=torch.int32).cuda()
    call = lambda c, qo: saga.saga_norm_rope_append(shape, q, k, v, c, starts, qo, counts=counts, norm=True, inv_freq=inv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache, q_out)
    for step in range(4):
        starts.copy_(torch.tensor([step * 5, 60 - step], dtype=torch.int32))
        counts.copy_(torch.tensor([step, 1], dtype=torch.int32))
        cache2 = saga.KVCache(*[t.clone() for t in cache._tensors()])
        out2 = q_out.clone()
        graph.replay()
        call(cache2, out2)
        torch.cuda.synchronize()
        assert torch.equal(q_out, out2)
        for a, b in zip(cache._tensors(), cache2._tensors()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
