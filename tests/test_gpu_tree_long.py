"""Attention of drafted tokens on the GPU at lengths where one lost row would drown in the tolerance, unless the rows
stand out: keys that resemble the queries sit at the first row, the last row and inside of every tile of 128 cache
rows, wherever the work is cut, and their values mark one element each.  The bounds are those of tests/test_gpu_tree.py;
each test first shows, on the exact outputs, that leaving out any one of these rows would exceed them.  And the precision
of 8-bit caches where it is lowest: queries with an outlier, and a long tail below one dominant row."""
import numpy as np
import pytest
import torch

from long_context_decoding_saga_b200 import saga
from tests import test_gpu_tree as tree

pytestmark = pytest.mark.gpu

BF16, E4M3 = saga.SAGA_CACHE_BF16, saga.SAGA_CACHE_E4M3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decoding_saga_b200 import build
    build.build()
    saga.load()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _marked_rows(P, per_tile, g):
    rows = set()
    for lo in range(0, P, 128):
        hi = min(lo + 128, P) - 1
        inside = int(torch.randint(lo, hi + 1, (1,), generator=g))
        rows |= set([lo, hi, inside][:per_tile])
    return sorted(rows)


def _inputs(heads, prefixes, T, per_tile, g):
    """Keys, values, queries (fp32) with marked rows, and the marked rows of each batch row."""
    h_q, h_k, h_v, d = heads
    B, l_cap = len(prefixes), max(prefixes) + T + 5
    u = torch.randn((B, h_k, 1, d), generator=g)
    u = u / u.square().mean(-1, keepdim=True).sqrt()
    k = 0.5 * torch.randn((B, h_k, l_cap, d), generator=g)
    v = 0.01 * torch.randn((B, h_v, l_cap, d), generator=g)
    marked = []
    for b, P in enumerate(prefixes):
        rows = _marked_rows(P, per_tile, g)
        marked.append(rows)
        if not rows:
            continue
        # their weights together are about four times those of all others: a score ln(4 others / marked) above
        gain = np.log(max(4.0 * P / len(rows), 2.0)) / np.sqrt(d)
        k[b][:, rows] = gain * u[b] + 0.05 * torch.randn((h_k, len(rows), d), generator=g)
        v[b][:, rows, torch.arange(len(rows)) % d] += 4.0
    q = u[:, torch.arange(h_q) * h_k // h_q, 0][:, None] + 0.1 * torch.randn((B, T, h_q, d), generator=g)
    return k, v, q.to(torch.bfloat16), marked


def _cached(shape, fmt, k, v):
    """The cache that holds k and v, and what it stands for, in float64."""
    c = saga.alloc_cache(shape, fmt)
    values = []
    for i, x in enumerate((k, v)):
        if fmt == BF16:
            x = x.to(torch.bfloat16)
            c._tensors()[i].copy_(x)
            values.append(x.double().numpy())
        else:
            scale = x.abs().amax(-1) / 448
            codes = (x / scale[..., None]).to(torch.float8_e4m3fn)
            c._tensors()[i].view(torch.uint8).copy_(codes.view(torch.uint8))
            c._tensors()[2 + i].copy_(scale)
            values.append(codes.double().numpy() * scale.double().numpy()[..., None])
    return c, values[0], values[1]


def _exact(q, K, V, P, T, fmt, marked):
    """Outputs of a chain of T tokens after P rows, their bounds, and for each marked row whether leaving it out would
    exceed the bounds somewhere.  q [T, h_q, d], K [h_k, cap, d], V [h_v, cap, d]."""
    h_q, d = q.shape[1:]
    h_k, h_v, L = K.shape[0], V.shape[0], P + T
    hidden = np.arange(L)[None] > P + np.arange(T)[:, None]
    out, bound = np.zeros((T, h_q, d)), np.zeros((T, h_q, d))
    weights = np.zeros((T, h_q, L))
    dots = 0.0
    for j in range(h_q):
        keys = K[j * h_k // h_q, :L]
        a = q[:, j] @ keys.T / np.sqrt(d)
        dots = max(dots, float((np.abs(q[:, j]) @ np.abs(keys).T).max()))
        a[hidden] = -np.inf
        w = np.exp(a - a.max(-1, keepdims=True))
        weights[:, j] = w / w.sum(-1, keepdims=True)
        out[:, j] = weights[:, j] @ V[j * h_v // h_q, :L]
        bound[:, j] = weights[:, j] @ np.abs(V[j * h_v // h_q, :L])
    es = ((d + 64) * 2.0 ** -23 + 2.0 ** -21) * dots / np.sqrt(d)
    if fmt == E4M3:
        es += 2.0 ** -17 * np.abs(q).max() * np.abs(K[:, :L]).sum(-1).max() / np.sqrt(d)
    rel = (2.0 ** -7 + 2.0 ** -14 if fmt == BF16 else 2.0 ** -9 + 2.0 ** -10) + np.expm1(2 * es) + 2.0 ** -20 + L * 2.0 ** -23
    bound = bound * rel + (L * 2.0 ** -27 * np.abs(V[:, :L]).max() if fmt == E4M3 else 0.0)
    shows = []
    for row in marked:
        w = weights[..., row, None]
        rest = (out - w * V[np.arange(h_q) * h_v // h_q, row][None]) / (1 - w)
        shows.append(bool((np.abs(rest - out) > 2 * bound).any()))
    return out, bound, shows


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", [((8, 1, 8, 64), 1), ((12, 1, 4, 128), 2), ((32, 2, 8, 64), 8), ((8, 1, 1, 128), 16)])
@pytest.mark.parametrize("prefixes,per_tile", [([33000], 1), ([20001, 4097, 0, 131, 9000], 3), ([2500] * 7, 3)])
def test_every_tile_counts(prefixes, per_tile, heads, T, fmt):
    g = torch.Generator().manual_seed(60 + T + len(prefixes))
    k, v, q, marked = _inputs(heads, prefixes, T, per_tile, g)
    B = len(prefixes)
    shape = saga.SagaShape.of(B, *heads, k.shape[2])
    cache, K, V = _cached(shape, fmt, k, v)
    out = torch.empty((B, T, heads[0], heads[3]), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    saga.saga_tree_attn(shape, q.cuda(), cache, _i32(prefixes), out, ws)
    for b, P in enumerate(prefixes):
        exact, bound, shows = _exact(q[b].double().numpy(), K[b], V[b], P, T, fmt, marked[b])
        assert all(shows), "a marked row of this test would not be missed"
        off = np.abs(out[b].double().cpu().numpy() - exact)
        assert (off <= bound).all(), (b, float((off - bound).max()))
    assert saga.saga_get_status(ws) == 0


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,B,T", [((8, 1, 8, 128), 40, 1), ((8, 1, 1, 128), 256, 16)])
def test_every_tile_counts_beyond_32_bits_of_elements(heads, B, T, fmt):
    """The last batch row of a cache of more than 2^31 elements."""
    P = 65000
    g = torch.Generator().manual_seed(70 + T)
    k, v, q, marked = _inputs(heads, [P], T, 1, g)
    shape = saga.SagaShape.of(B, *heads, 66000)
    assert B * heads[2] * 66000 * heads[3] > 2 ** 31
    small, K, V = _cached(saga.SagaShape.of(1, *heads, k.shape[2]), fmt, k, v)
    cache = saga.alloc_cache(shape, fmt)
    for a, b in zip(cache._tensors(), small._tensors()):
        if a is not None:
            a[B - 1:, :, :b.shape[2]].view(torch.uint8).copy_(b.view(torch.uint8))
    qs = torch.zeros((B,) + tuple(q.shape[1:]), dtype=torch.bfloat16)
    qs[B - 1] = q[0]
    lens, counts = [0] * B, [0] * B
    lens[B - 1], counts[B - 1] = P, T
    out = torch.zeros((B, T, heads[0], heads[3]), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    saga.saga_tree_attn(shape, qs.cuda(), cache, _i32(lens), out, ws, counts=_i32(counts))
    exact, bound, shows = _exact(q[0].double().numpy(), K[0], V[0], P, T, fmt, marked[0])
    assert all(shows), "a marked row of this test would not be missed"
    off = np.abs(out[B - 1].double().cpu().numpy() - exact)
    assert (off <= bound).all(), float((off - bound).max())
    assert saga.saga_get_status(ws) == 0


@pytest.mark.parametrize("heads,T", [((12, 1, 4, 128), 2), ((8, 1, 8, 64), 1), ((32, 2, 8, 64), 8)])
def test_queries_with_an_outlier(heads, T):
    """8-bit caches take q as two e4m3 numbers: elements far below a row's largest are off by up to 2^-17 of it."""
    g = torch.Generator().manual_seed(80 + T)
    shape = saga.SagaShape.of(1, *heads, 700)
    cache, K, V = tree._fill(shape, E4M3, g)
    q = 0.3 * torch.randn((1, T, heads[0], heads[3]), generator=g)
    q[..., 3] = 60.0
    q[:, :, 1::2, 3] = -200.0
    q = q.to(torch.bfloat16)
    out = torch.empty((1, T, heads[0], heads[3]), device="cuda")
    saga.saga_tree_attn(shape, q.cuda(), cache, _i32([600]), out, saga.alloc_tree_workspace(shape, T))
    exact, bound, _ = _exact(q[0].double().numpy(), K[0], V[0], 600, T, E4M3, [])
    assert (np.abs(out[0].double().cpu().numpy() - exact) <= bound).all()


@pytest.mark.parametrize("below", [10, 16, 22, 26, 28])
def test_a_long_tail_below_one_row(below):
    """8-bit caches, an item in one CTA: one dominant row and 16383 rows 2^-below under it, whose values are another
    element's.  Down to 2^-16 the tail keeps its 9 bits; below, each row is off by up to 2^-27 of the dominant one."""
    B, L = 140, 16384
    shape = saga.SagaShape.of(B, 1, 1, 1, 64, L)
    k = torch.zeros((1, 1, L, 64))
    k[..., 0] = 1.0
    k[:, :, 77, 0] = -1.0
    v = torch.zeros((1, 1, L, 64))
    v[..., 1] = 1.0
    v[:, :, 77] = 0.0
    v[:, :, 77, 0] = 1.0
    q = torch.zeros((1, 1, 1, 64))
    q[..., 0] = -below * np.log(2.0) * 8 / 2  # scores 0.5 * below * ln 2 and minus that
    q = q.to(torch.bfloat16)
    one, K, V = _cached(saga.SagaShape.of(1, 1, 1, 1, 64, L), E4M3, k, v)
    cache = saga.KVCache(*[t.expand((B,) + tuple(t.shape[1:])).contiguous() for t in one._tensors()])
    out = torch.empty((B, 1, 1, 64), device="cuda")
    saga.saga_tree_attn(shape, q.expand(B, 1, 1, 64).contiguous().cuda(), cache, _i32([L - 1] * B), out,
                        saga.alloc_tree_workspace(shape, 1))
    exact, bound, _ = _exact(q[0].double().numpy(), K[0], V[0], L - 1, 1, E4M3, [])
    if below <= 16:
        bound = bound - L * 2.0 ** -27 * np.abs(V).max()
    got = out[:, 0].double().cpu().numpy()
    assert (np.abs(got - exact) <= bound).all(), (got[0, 0, :2], exact[0, 0, :2])


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_thresholds_of_the_refresh_over_drafted_tokens(fmt):
    """Rows normed, rotated and appended after a stored history, the thresholds of the library's own refresh on the
    first token, and the tree's attention under them: each head's threshold is moved into the widest gap near it among
    all tokens' scores, so that no score is within rounding of it."""
    from oracle import serve_oracle as so
    heads, P, T, n_top = (12, 1, 4, 128), 700, 5, 64
    h_q, h_k, h_v, d = heads
    shape = saga.SagaShape.of(1, *heads, 800)
    g = torch.Generator().manual_seed(90)
    cache = saga.alloc_cache(shape, fmt)
    pl = _i32([P])
    hist = torch.randn((1, P, h_k + h_v, d), generator=g).to(torch.bfloat16).cuda()
    saga.saga_kv_store(shape, hist[:, :, :h_k], hist[:, :, h_k:], cache, _i32([0]))
    x = torch.randn((1, T, h_q + h_k + h_v, d), generator=g).to(torch.bfloat16).cuda()
    masks = [[0b1, 0b11, 0b101, 0b1011, 0b10000]]
    inv = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().cuda()
    q_out = torch.empty((1, T, h_q, d), dtype=torch.bfloat16, device="cuda")
    saga.saga_norm_rope_append(shape, x[:, :, :h_q], x[:, :, h_q:h_q + h_k], x[:, :, h_q + h_k:], cache, pl, q_out,
                               norm=True, inv_freq=inv)
    keys = cache.k
    if fmt == E4M3:
        keys = torch.zeros((1, h_k, 800, d), dtype=torch.bfloat16, device="cuda")
        saga.saga_kv_load(shape, cache, 0, 800, k_out=keys)
    tau = torch.zeros((1, h_q), device="cuda")
    saga.atopn_refresh_threshold(shape, q_out[:, 0].contiguous(), keys, P + 1, n_top, tau, saga.alloc_workspace(shape))
    K, V = cache.k[0].double().cpu().numpy(), cache.v[0].double().cpu().numpy()
    if fmt == E4M3:
        K = K * cache.k_scale[0].double().cpu().numpy()[..., None]
        V = V * cache.v_scale[0].double().cpu().numpy()[..., None]
    qe = q_out[0].double().cpu().numpy()
    moved = np.zeros((1, h_q), np.float32)
    for j in range(h_q):
        a = qe[:, j] @ K[0, :P + T].T / np.sqrt(d)
        given = float(tau[0, j])
        first = np.sort(a[0, :P + 1])[::-1]
        # the refresh's keys are bf16: of an 8-bit cache, each off by 2^-8 of itself at most
        near = 2.0 ** -8 * float((np.abs(qe[0, j]) @ np.abs(K[0, :P + 1]).T).max()) / np.sqrt(d) if fmt == E4M3 else 1e-3
        assert first[n_top - 1] - near <= given <= first[n_top - 1] + near
        s = np.sort(a.ravel())
        i = int(np.searchsorted(s, given))
        lo, hi = max(0, i - 20), min(len(s) - 1, i + 20)
        at = lo + int((s[lo + 1:hi + 1] - s[lo:hi]).argmax())
        moved[0, j] = 0.5 * (s[at] + s[at + 1])
    out = torch.empty((1, T, h_q, d), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    saga.saga_tree_attn(shape, q_out, cache, pl, out, ws, tree_mask=tree._words(masks).cuda(),
                        tau=torch.from_numpy(moved).cuda())
    exact, bound, border, es = tree._bounds(qe, K, V, P, T, masks[0], moved[0].astype(np.float64), d, fmt)
    assert border > es, "a threshold of this test is too near a score"
    dense, _ = so.attend(qe, K, V, P, T, masks[0], None)
    assert (np.abs(dense - exact) > 2 * bound).any(axis=(1, 2)).all(), "the thresholds drop too little to be seen"
    assert (np.abs(out[0].double().cpu().numpy() - exact) <= bound).all()
    assert saga.saga_get_status(ws) == 0
