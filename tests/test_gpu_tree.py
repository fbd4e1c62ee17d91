"""Attention of drafted tokens on the GPU against float64.

Bound, element by element, with w the exact softmax weights: a score is off by at most
  es = ((D + 64) 2^-23 + 2^-21) sum |q_c k_c| / sqrt(d)
(fp32 sums in any order with truncating tensor-core steps, the products with the scales), which changes weights by
a factor of at most e^(2 es).  bf16 caches: the weights are rounded to bf16, w' = w (1 + d) with |d| <= 2^-8, and
divided by the sum of the rounded ones, so sum w' v / sum w' is off by at most sum w |v| (2^-8 + 2^-8) to first order
(2^-14 covers the second).  8-bit caches: a weight is the sum of three e5m2 numbers, each off by at most 2^-3 of what
is left (2^-9), taken in half precision (2^-11), and divided by the exact sum; what is below half of e5m2's smallest
number, 2^-17 where the largest weight is 2^10 or more, is 2^-27 of that for each of L rows.  q is two e4m3 numbers
there, with elements below 2^-14 of the row's largest off by up to 2^-17 of it, which es includes.  The exponential and
the fp32 sums over L rows add 2^-20 + L 2^-23, and a bf16 output 2^-8 of the value:
  |out - exact| <= sum w |v| ([bf16] 2^-7 + 2^-14, [8-bit] 2^-9 + 2^-10, + e^(2 es) - 1 + 2^-20 + L 2^-23)
                   + [8-bit] L 2^-27 max |v|  (+ 2^-8 |exact| for bf16).
Thresholds are placed so that every score is more than es from them: a score that is off by at most es is then on
the same side of its threshold.
"""
import numpy as np
import pytest
import torch

from long_context_decoding_saga_b200 import saga
from oracle import serve_oracle as so

pytestmark = pytest.mark.gpu

BF16, E4M3 = saga.SAGA_CACHE_BF16, saga.SAGA_CACHE_E4M3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decoding_saga_b200 import build
    build.build()
    saga.load()


def _fill(shape, fmt, g, spread=1.0, row_spread=0.0):
    """Caches with every row finite; returns the cache and its values in float64."""
    B, h_q, h_k, h_v, d, l_cap = shape.astuple()
    c = saga.alloc_cache(shape, fmt)
    vals = []
    for i, h in enumerate((h_k, h_v)):
        x = torch.randn((B, h, l_cap, d), generator=g) * spread
        if row_spread:
            x = x * torch.exp(row_spread * torch.randn((B, h, l_cap, 1), generator=g))
        if fmt == BF16:
            x = x.to(torch.bfloat16)
            c._tensors()[i].copy_(x)
            vals.append(x.double().numpy())
        else:
            scale = x.abs().amax(-1) / 448
            codes = (x / scale[..., None]).to(torch.float8_e4m3fn)
            c._tensors()[i].view(torch.uint8).copy_(codes.view(torch.uint8))
            c._tensors()[2 + i].copy_(scale)
            vals.append(codes.double().numpy() * scale.double().numpy()[..., None])
    return c, vals[0], vals[1]


def _trees(B, T, g, bits=None):
    masks = []
    for _ in range(B):
        row = []
        for t in range(T):
            parent = t - 1 - int(torch.randint(0, 4, (1,), generator=g))
            row.append((row[parent] if parent >= 0 else 0) | 1 << t)
        masks.append(row)
    return masks


def _words(masks):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64)


def _bounds(q, K, V, prefix, n, masks, tau, D, fmt):
    """exact outputs, and their bounds for an fp32 output, of one batch row."""
    exact, border = so.attend(q, K, V, prefix, n, masks, tau)
    spread, _ = so.attend(q, K, np.abs(V), prefix, n, masks, tau)
    T, h_q, d = q.shape
    L = prefix + n
    if L == 0 or n == 0:
        return exact, np.zeros_like(exact), border, 0.0
    dots = max(float((np.abs(q[:n, j]) @ np.abs(K[j * K.shape[0] // h_q, :L]).T).max()) for j in range(h_q))
    es = ((D + 64) * 2.0 ** -23 + 2.0 ** -21) * dots / np.sqrt(d)
    if fmt == E4M3:
        es += 2.0 ** -17 * np.abs(q[:n]).max() * np.abs(K[:, :L]).sum(-1).max() / np.sqrt(d)
    rel = (2.0 ** -7 + 2.0 ** -14 if fmt == BF16 else 2.0 ** -9 + 2.0 ** -10) + np.expm1(2 * es) + 2.0 ** -20 + L * 2.0 ** -23
    lost = L * 2.0 ** -27 * np.abs(V[:, :L]).max() if fmt == E4M3 else 0.0
    return exact, spread * rel + lost, border, es


def _check(heads, fmt, prefixes, T, masks=None, counts=None, tau_n=0, out_dtype=torch.float32, seed=0, l_cap=None,
           spread=1.0, row_spread=0.0, q_scale=1.0, poison=False, tau_value=None, tau_rank=0):
    h_q, h_k, h_v, d = heads
    B = len(prefixes)
    l_cap = max(prefixes) + T + 3 if l_cap is None else l_cap
    shape = saga.SagaShape.of(B, *heads, l_cap)
    g = torch.Generator().manual_seed(1000 + seed)
    cache, K, V = _fill(shape, fmt, g, spread, row_spread)
    q = (torch.randn((B, T, h_q, d), generator=g) * q_scale).to(torch.bfloat16)
    if masks == "tree":
        masks = _trees(B, T, g)
    n = [T] * B if counts is None else [min(max(c, 0), T) for c in counts]
    qe = q.double().numpy()
    tau = None
    if tau_value is not None:
        tau = np.full((B, h_q), tau_value, np.float32)
    elif tau_n or tau_rank:
        tau = np.zeros((B, h_q), np.float32)
        for b in range(B):
            for j in range(h_q):
                a = np.sort((K[b, j * h_k // h_q, :prefixes[b] + n[b]] @ qe[b, :max(n[b], 1), j].T).ravel() / np.sqrt(d))[::-1]
                m = min(tau_rank or tau_n * max(n[b], 1), len(a) - 2)
                lo, hi = max(0, m - 20), min(len(a) - 1, m + 20)
                gaps = a[lo:hi] - a[lo + 1:hi + 1]
                i = lo + int(gaps.argmax())
                tau[b, j] = 0.5 * (a[i] + a[i + 1])
    if poison:  # rows that nobody sees: past the last token, and drafted rows outside every mask
        for b in range(B):
            seen = 0
            for t in range(n[b]):
                seen |= (1 << (t + 1)) - 1 if masks is None else masks[b][t]
            rows = [prefixes[b] + u for u in range(n[b]) if not seen >> u & 1] + list(range(prefixes[b] + n[b], l_cap))
            for t in cache._tensors()[:2]:
                t[b].view(torch.uint8)[:, rows] = 0x7F if fmt == E4M3 else 0xFF
            for t in cache._tensors()[2:]:
                if t is not None:
                    t[b][:, rows] = float("nan")
    out = torch.full((B, T, h_q, d), 7.0, dtype=out_dtype, device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    args = dict(tree_mask=None if masks is None else _words(masks).cuda(),
                counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda(),
                tau=None if tau is None else torch.from_numpy(tau).cuda())
    pl = torch.tensor(prefixes, dtype=torch.int32).cuda()
    saga.saga_tree_attn(shape, q.cuda(), cache, pl, out, ws, **args)
    again = torch.full_like(out, 7.0)
    saga.saga_tree_attn(shape, q.cuda(), cache, pl, again, ws, **args)
    torch.cuda.synchronize()
    assert saga.saga_get_status(ws) == 0
    assert torch.equal(out, again), "a second call on the workspace differs"
    for b in range(B):
        exact, bound, border, es = _bounds(qe[b], K[b], V[b], prefixes[b], n[b], None if masks is None else masks[b],
                                           None if tau is None else tau[b].astype(np.float64), d, fmt)
        if tau_n or tau_rank:
            assert border > es, "the thresholds of this test are too near a score"
        got = out[b, :n[b]].double().cpu().numpy()
        if out_dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(exact) + bound)
        off = np.abs(got - exact)
        assert (off <= bound).all(), (b, float((off - bound).max()), float(off.max()))
        assert (out[b, n[b]:] == 7.0).all()


HEADS = [(8, 1, 8, 64), (12, 1, 4, 128), (32, 2, 8, 64), (32, 8, 8, 64), (16, 4, 2, 64), (3, 3, 1, 128), (1, 1, 1, 64),
         (32, 1, 32, 64), (32, 1, 1, 128), (64, 1, 8, 64), (16, 2, 4, 128), (40, 2, 10, 64)]


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("T", [1, 5])
def test_head_layouts(heads, fmt, T):
    _check(heads, fmt, [300], T, masks="tree", seed=T)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("prefix", [0, 1, 63, 127, 128, 129, 255, 1000, 2500])
@pytest.mark.parametrize("T", [1, 3])
def test_prefix_lengths(prefix, fmt, T):
    _check((12, 1, 4, 128), fmt, [prefix], T, seed=prefix)
    _check((32, 2, 8, 64), fmt, [prefix], T, masks="tree", seed=prefix + 1)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 16, 31, 33, 48, 63, 64])
@pytest.mark.parametrize("heads", [(32, 2, 8, 64), (12, 1, 4, 128), (4, 4, 4, 64)])
def test_token_counts(heads, T, fmt):
    _check(heads, fmt, [200], T, masks="tree", seed=T, out_dtype=torch.bfloat16)
    _check(heads, fmt, [64], T, seed=T)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_ragged_batch(fmt):
    prefixes = [0, 1, 700, 128, 3, 1500, 64, 129, 0, 256]
    counts = [6, 0, 1, 4, 9, -2, 5, 6, 0, 3]
    _check((32, 2, 8, 64), fmt, prefixes, 6, masks="tree", counts=counts, seed=3)
    _check((12, 1, 4, 128), fmt, prefixes, 6, counts=counts, seed=4, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_rows_that_see_nothing_give_zero(fmt):
    _check((32, 2, 8, 64), fmt, [0, 0], 4, masks=[[0, 2, 3, 0], [0, 0, 0, 0]], seed=5)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads", [(32, 2, 8, 64), (12, 1, 4, 128)])
def test_rows_that_nobody_sees_may_hold_nan(heads, fmt):
    _check(heads, fmt, [100, 0, 126, 250], 7, masks=[[0b1, 0b101, 0b101, 0, 0, 0b10101, 0]] * 4, counts=[7, 3, 7, 6],
           seed=6, poison=True)
    _check(heads, fmt, [100, 0, 126], 3, seed=7, poison=True, l_cap=400)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads", [(32, 2, 8, 64), (12, 1, 4, 128), (8, 1, 8, 64)])
@pytest.mark.parametrize("tau_n", [1, 16, 200])
def test_thresholds(heads, tau_n, fmt):
    _check(heads, fmt, [900], 4, masks="tree", tau_n=tau_n, seed=tau_n)


@pytest.mark.parametrize("value", [float("-inf"), float("inf"), float("nan")])
def test_threshold_that_keeps_all_or_nothing(value):
    _check((32, 2, 8, 64), BF16, [300], 3, tau_value=value, seed=8)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("q_scale,spread,row_spread", [(12.0, 4.0, 0.0), (1e-3, 1.0, 0.0), (1.0, 1.0, 2.0),
                                                       (2.0 ** 40, 2.0 ** -40, 0.0), (2.0 ** -40, 2.0 ** 40, 0.0)])
def test_magnitudes(q_scale, spread, row_spread, fmt):
    """Sharp and flat softmaxes, rows of very different magnitudes, and magnitudes far from one."""
    _check((12, 1, 4, 128), fmt, [600], 3, seed=9, q_scale=q_scale, spread=spread, row_spread=row_spread)
    _check((32, 2, 8, 64), fmt, [600], 3, seed=9, q_scale=q_scale, spread=spread, row_spread=row_spread)


def test_rising_scores():
    """Every block's scores exceed all before it, so the running maximum moves at every step."""
    heads, P = (12, 1, 4, 128), 2000
    shape = saga.SagaShape.of(1, *heads, P + 1)
    for fmt in (BF16, E4M3):
        k = torch.zeros((1, 1, P + 1, 128))
        k[0, 0, :, 0] = torch.arange(P + 1) / 2.0
        v = torch.randn((1, 4, P + 1, 128), generator=torch.Generator().manual_seed(1))
        cache = saga.alloc_cache(shape, fmt)
        saga.saga_kv_store(shape, k.transpose(1, 2).to(torch.bfloat16).cuda(), v.transpose(1, 2).to(torch.bfloat16).cuda(),
                           cache, torch.zeros(1, dtype=torch.int32).cuda())
        K, V = cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy()
        if fmt == E4M3:
            K, V = K * cache.k_scale.double().cpu().numpy()[..., None], V * cache.v_scale.double().cpu().numpy()[..., None]
        q = torch.zeros((1, 1, 12, 128))
        q[..., 0] = torch.linspace(-40, 40, 12)
        q = q.to(torch.bfloat16)
        out = torch.empty((1, 1, 12, 128), device="cuda")
        ws = saga.alloc_tree_workspace(shape, 1)
        saga.saga_tree_attn(shape, q.cuda(), cache, torch.tensor([P], dtype=torch.int32).cuda(), out, ws)
        exact, bound, _, _ = _bounds(q[0].double().numpy(), K[0], V[0], P, 1, None, None, 128, fmt)
        assert (np.abs(out[0].double().cpu().numpy() - exact) <= bound).all()


def test_a_bad_prefix_is_clamped_and_flagged():
    heads = (8, 1, 8, 64)
    shape = saga.SagaShape.of(2, *heads, 100)
    g = torch.Generator().manual_seed(2)
    cache, K, V = _fill(shape, BF16, g)
    q = torch.randn((2, 3, 8, 64), generator=g).to(torch.bfloat16)
    out = torch.empty((2, 3, 8, 64), device="cuda")
    ws = saga.alloc_tree_workspace(shape, 3)
    saga.saga_tree_attn(shape, q.cuda(), cache, torch.tensor([-5, 98], dtype=torch.int32).cuda(), out, ws)
    assert saga.saga_get_status(ws) == saga.SAGA_STATUS_LEN_CLAMPED
    for b, P in enumerate((0, 97)):
        exact, bound, _, _ = _bounds(q[b].double().numpy(), K[b], V[b], P, 3, None, None, 64, BF16)
        assert (np.abs(out[b].double().cpu().numpy() - exact) <= bound).all()


def test_one_token_matches_the_dense_decode_call():
    heads = (32, 8, 8, 64)
    shape = saga.SagaShape.of(1, *heads, 1200)
    g = torch.Generator().manual_seed(3)
    cache, K, V = _fill(shape, BF16, g)
    q = torch.randn((1, 1, 32, 64), generator=g).to(torch.bfloat16).cuda()
    out, ref = torch.empty((1, 1, 32, 64), device="cuda"), torch.empty((1, 32, 64), device="cuda")
    saga.saga_tree_attn(shape, q, cache, torch.tensor([1000], dtype=torch.int32).cuda(), out,
                        saga.alloc_tree_workspace(shape, 1))
    tau = torch.empty((1, 32), device="cuda")
    saga.saga_decode_attn(shape, q[:, 0].contiguous(), cache.k, cache.v, 1001, 1200, 1, 0, tau, ref,
                          saga.alloc_workspace(shape))
    exact, bound, _, _ = _bounds(q[0].double().cpu().numpy(), K[0], V[0], 1000, 1, None, None, 64, BF16)
    assert (np.abs(out[0, 0].double().cpu().numpy() - ref[0].double().cpu().numpy()) <= 2 * bound[0]).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_captured_call_follows_device_lengths(fmt):
    heads, T = (32, 2, 8, 64), 4
    shape = saga.SagaShape.of(2, *heads, 900)
    g = torch.Generator().manual_seed(4)
    cache, K, V = _fill(shape, fmt, g)
    q = torch.randn((2, T, 32, 64), generator=g).to(torch.bfloat16).cuda()
    out = torch.zeros((2, T, 32, 64), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    pl = torch.tensor([5, 5], dtype=torch.int32).cuda()
    cn = torch.tensor([T, T], dtype=torch.int32).cuda()
    mask = _words(_trees(2, T, g)).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saga.saga_tree_attn(shape, q, cache, pl, out, ws, tree_mask=mask, counts=cn)
    for prefixes, counts in (([0, 896], [4, 4]), ([500, 10], [1, 3]), ([128, 0], [0, 4])):
        pl.copy_(torch.tensor(prefixes, dtype=torch.int32))
        cn.copy_(torch.tensor(counts, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        want = torch.full_like(out, 7.0)
        saga.saga_tree_attn(shape, q, cache, pl, want, saga.alloc_tree_workspace(shape, T), tree_mask=mask, counts=cn)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert saga.saga_get_status(ws) == 0


def test_two_streams_with_workspaces_of_their_own():
    heads, T = (12, 1, 4, 128), 3
    shape = saga.SagaShape.of(1, *heads, 3000)
    g = torch.Generator().manual_seed(5)
    cache, K, V = _fill(shape, BF16, g)
    pl = torch.tensor([2900], dtype=torch.int32).cuda()
    qs = [torch.randn((1, T, 12, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    wss = [saga.alloc_tree_workspace(shape, T) for _ in range(2)]
    want = [torch.empty((1, T, 12, 128), device="cuda") for _ in range(2)]
    for i in range(2):
        saga.saga_tree_attn(shape, qs[i], cache, pl, want[i], wss[i])
    got = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            saga.saga_tree_attn(shape, qs[i], cache, pl, got[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_a_served_step(fmt):
    """Rows of a projection, normed, rotated and appended as drafted tokens after a stored history; the tree's
    attention over them; and, on the 8-bit cache, the thresholds from keys read back."""
    heads, P, T = (12, 1, 4, 128), 700, 5
    h_q, h_k, h_v, d = heads
    shape = saga.SagaShape.of(1, *heads, 800)
    g = torch.Generator().manual_seed(6)
    cache = saga.alloc_cache(shape, fmt)
    hist = torch.randn((1, P, h_k + h_v, d), generator=g).to(torch.bfloat16).cuda()
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    saga.saga_kv_store(shape, hist[:, :, :h_k], hist[:, :, h_k:], cache, zero)
    x = torch.randn((1, T, h_q + h_k + h_v, d), generator=g).to(torch.bfloat16).cuda()
    masks = [[0b1, 0b11, 0b101, 0b1011, 0b10000]]
    depth = torch.tensor([[0, 1, 1, 2, 0]], dtype=torch.int32)
    pl = torch.tensor([P], dtype=torch.int32).cuda()
    inv = (10000.0 ** (-torch.arange(0, d, 2) / d)).float()
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    q_out = torch.empty((1, T, h_q, d), dtype=torch.bfloat16, device="cuda")
    saga.saga_norm_rope_append(shape, x[:, :, :h_q], x[:, :, h_q:h_q + h_k], x[:, :, h_q + h_k:], cache, pl, q_out,
                               positions=(P + depth).cuda(), norm=True, q_weight=w.cuda(), k_weight=w.cuda(),
                               inv_freq=inv.cuda())
    tau = torch.zeros((1, h_q), device="cuda")
    keys = cache.k
    if fmt == E4M3:
        keys = torch.zeros((1, h_k, 800, d), dtype=torch.bfloat16, device="cuda")
        saga.saga_kv_load(shape, cache, 0, 800, k_out=keys)
    saga.atopn_refresh_threshold(shape, q_out[:, 0].contiguous(), keys, P + 1, 64, tau, saga.alloc_workspace(shape))
    tau -= 0.01  # off the scores themselves
    ws = saga.alloc_tree_workspace(shape, T)
    outs = {}
    for name, th in (("dense", None), ("kept", tau)):
        outs[name] = torch.empty((1, T, h_q, d), device="cuda")
        saga.saga_tree_attn(shape, q_out, cache, pl, outs[name], ws, tree_mask=_words(masks).cuda(), tau=th)
    assert saga.saga_get_status(ws) == 0
    # from the projection's rows on, in float64
    K, V = cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy()
    if fmt == E4M3:
        K, V = K * cache.k_scale.double().cpu().numpy()[..., None], V * cache.v_scale.double().cpu().numpy()[..., None]
    xe = x[0].double().cpu().numpy()
    qn = so.rotate(so.norm(xe[:, :h_q], w.double().numpy(), 1e-6), (P + depth[0]).numpy(), inv.double().numpy(), False)
    qg = q_out[0].double().cpu().numpy()
    assert np.abs(qg - qn).max() <= 2.0 ** -8 * np.abs(qn).max() * 1.01
    exact, bound, _, _ = _bounds(qg, K[0], V[0], P, T, masks[0], None, d, fmt)
    assert (np.abs(outs["dense"][0].double().cpu().numpy() - exact) <= bound).all()
    te = tau[0].double().cpu().numpy()
    exact, bound, border, es = _bounds(qg, K[0], V[0], P, T, masks[0], te, d, fmt)
    if border > es:
        assert (np.abs(outs["kept"][0].double().cpu().numpy() - exact) <= bound).all()
    counts = (K[0, 0, :P + 1] @ qg[0].T / np.sqrt(d) >= te).sum(axis=0)
    assert (counts >= 64).all()


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads", [(8, 1, 8, 128), (16, 1, 16, 64), (16, 1, 16, 128)])
@pytest.mark.parametrize("T,prefix", [(1, 9000), (16, 9000), (16, 8953), (3, 40)])
def test_more_value_heads_than_tiles_in_flight(heads, T, prefix, fmt):
    """Value heads of a chunk that do not fit the ring of tiles at once, with the drafted rows in a last tile that
    has others before it (long runs), or in the last two; rows that nobody sees hold NaN."""
    masks = [[0b1 if t == 0 else 1 << t | 1 for t in range(T)]]
    if T > 2:
        masks[0][2] = 0
        masks[0][T - 1] &= ~4
    _check(heads, fmt, [prefix] * 4, T, masks=masks * 4, seed=T, poison=True)


@pytest.mark.parametrize("heads,T", [((8, 1, 8, 64), 4), ((8, 1, 8, 128), 1), ((12, 1, 4, 128), 2), ((32, 2, 8, 64), 2)])
def test_few_columns_lose_nothing_to_bf16_weights(heads, T):
    """Up to 8 columns of a value head: a weight is two bf16 numbers, off by 2^-8 of 2^-8 of it, and so is the sum it is
    divided by: 2^-15 in place of 2^-7 in the bound."""
    h_q, h_k, h_v, d = heads
    assert h_q // h_v * T <= 8
    P = 900
    shape = saga.SagaShape.of(1, *heads, P + T)
    g = torch.Generator().manual_seed(19)
    cache, K, V = _fill(shape, BF16, g)
    q = torch.randn((1, T, h_q, d), generator=g).to(torch.bfloat16)
    out = torch.empty((1, T, h_q, d), device="cuda")
    saga.saga_tree_attn(shape, q.cuda(), cache, torch.tensor([P], dtype=torch.int32).cuda(), out,
                        saga.alloc_tree_workspace(shape, T))
    exact, bound, _, _ = _bounds(q[0].double().numpy(), K[0], V[0], P, T, None, None, d, BF16)
    spread, _ = so.attend(q[0].double().numpy(), K[0], np.abs(V[0]), P, T, None, None)
    bound = bound - spread * (2.0 ** -7 + 2.0 ** -14 - 2.0 ** -15 - 2.0 ** -28)
    assert (np.abs(out[0].double().cpu().numpy() - exact) <= bound).all()


# ---- chunks of many query rows: the other of the two kernels (see the rule in the source) for both formats
MANY = [((32, 2, 8, 64), 12), ((12, 1, 4, 128), 40), ((32, 1, 32, 64), 33), ((64, 1, 8, 64), 16), ((3, 3, 1, 128), 64)]


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", MANY)
@pytest.mark.parametrize("rank", [4, 200])
def test_thresholds_of_many_rows(heads, T, rank, fmt):
    """Thresholds at a rank among all scores of a head (with so many scores, those of higher ranks lie closer together
    than es): some drafted tokens keep nothing, others several rows."""
    _check(heads, fmt, [700], T, masks="tree", tau_rank=rank, seed=T + rank)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", MANY)
def test_many_rows_and_rows_that_nobody_sees(heads, T, fmt):
    """Unseen rows hold NaN; some drafted tokens see a few rows, some none, and batch rows hold fewer tokens."""
    masks = [[0 if t % 5 == 3 else 1 << t | (1 << (t // 2)) for t in range(T)] for _ in range(4)]
    for row in masks:  # token 1's row is seen by nobody
        for t in range(T):
            row[t] &= ~2
    _check(heads, fmt, [0, 126, 500, 1], T, masks=masks, counts=[T, T - 3, 5, T], seed=T, poison=True)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", MANY[:3])
@pytest.mark.parametrize("q_scale,spread,row_spread", [(12.0, 4.0, 0.0), (1e-3, 1.0, 0.0), (1.0, 1.0, 2.0),
                                                       (2.0 ** 40, 2.0 ** -40, 0.0)])
def test_magnitudes_of_many_rows(heads, T, q_scale, spread, row_spread, fmt):
    _check(heads, fmt, [600], T, seed=11, q_scale=q_scale, spread=spread, row_spread=row_spread)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("T", [2, 20])
def test_batch_rows_beyond_a_warp(T, fmt):
    """More batch rows than a warp has lanes, many of them empty, of very different lengths."""
    g = torch.Generator().manual_seed(12)
    prefixes = [int(x) ** 2 // 40 for x in torch.randint(0, 200, (75,), generator=g)]
    counts = [int(x) for x in torch.randint(-2, T + 1, (75,), generator=g)]
    counts[:33] = [0] * 33
    counts[-1] = T
    _check((16, 2, 4, 128), fmt, prefixes, T, masks="tree", counts=counts, seed=13, l_cap=max(prefixes) + T)


@pytest.mark.parametrize("value", [float("-inf"), float("inf"), float("nan")])
@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_threshold_that_keeps_all_or_nothing_of_many_rows(fmt, value):
    _check((32, 2, 8, 64), fmt, [300], 12, tau_value=value, seed=14)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("T", [1, 16])
def test_rows_beyond_32_bits_of_elements(T, fmt):
    """The last batch row of a cache of more than 2^31 elements."""
    heads, B, l_cap, P = (8, 1, 8, 128), 40, 66000, 65000
    h_q, h_k, h_v, d = heads
    assert B * h_v * l_cap * d > 2 ** 31
    shape = saga.SagaShape.of(B, *heads, l_cap)
    one = saga.SagaShape.of(1, *heads, l_cap)
    g = torch.Generator().manual_seed(15)
    small, K, V = _fill(one, fmt, g)
    cache = saga.alloc_cache(shape, fmt)
    for a, b in zip(cache._tensors(), small._tensors()):
        if a is not None:
            a[B - 1:].view(torch.uint8).copy_(b.view(torch.uint8))
    q = torch.randn((B, T, h_q, d), generator=g).to(torch.bfloat16)
    pl = torch.zeros(B, dtype=torch.int32)
    pl[B - 1] = P
    counts = torch.zeros(B, dtype=torch.int32)
    counts[B - 1] = T
    out = torch.zeros((B, T, h_q, d), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    saga.saga_tree_attn(shape, q.cuda(), cache, pl.cuda(), out, ws, counts=counts.cuda())
    exact, bound, _, _ = _bounds(q[B - 1].double().numpy(), K[0], V[0], P, T, None, None, d, fmt)
    assert (np.abs(out[B - 1].double().cpu().numpy() - exact) <= bound).all()
    assert saga.saga_get_status(ws) == 0
    # and its rows stored and read back there
    x = torch.randn((B, 3, h_k + h_v, d), generator=g).to(torch.bfloat16).cuda()
    starts = torch.full((B,), l_cap - 3, dtype=torch.int32).cuda()
    saga.saga_kv_store(shape, x[:, :, :h_k], x[:, :, h_k:], cache, starts)
    saga.saga_kv_store(one, x[B - 1:, :, :h_k], x[B - 1:, :, h_k:], small, starts[:1])
    for a, b in zip(cache._tensors(), small._tensors()):
        if a is not None:
            assert torch.equal(a[B - 1:].view(torch.uint8), b.view(torch.uint8))
    if fmt == E4M3:
        outs = [torch.empty((s.batch, h_v, 1000, d), dtype=torch.bfloat16, device="cuda") for s in (shape, one)]
        saga.saga_kv_load(shape, cache, l_cap - 1000, 1000, v_out=outs[0])
        saga.saga_kv_load(one, small, l_cap - 1000, 1000, v_out=outs[1])
        assert torch.equal(outs[0][B - 1:], outs[1])


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_a_workspace_serves_fewer_tokens(fmt):
    """A workspace for 64 tokens, reused from call to call, gives what a fresh one gives."""
    heads = (32, 2, 8, 64)
    shape = saga.SagaShape.of(2, *heads, 700)
    g = torch.Generator().manual_seed(16)
    cache, _, _ = _fill(shape, fmt, g)
    pl = torch.tensor([600, 31], dtype=torch.int32).cuda()
    ws = saga.alloc_tree_workspace(shape, 64)
    for T in (64, 1, 33, 2, 5, 17, 6, 64, 9, 3):
        q = torch.randn((2, T, 32, 64), generator=g).to(torch.bfloat16).cuda()
        got, want = (torch.empty((2, T, 32, 64), device="cuda") for _ in range(2))
        saga.saga_tree_attn(shape, q, cache, pl, got, ws)
        saga.saga_tree_attn(shape, q, cache, pl, want, saga.alloc_tree_workspace(shape, T))
        assert torch.equal(got, want)
    assert saga.saga_get_status(ws) == 0
    sizes = [saga.saga_tree_workspace_bytes(shape, t) for t in range(1, 65)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("fmt", [BF16, E4M3])
def test_two_graphs_on_one_workspace(fmt):
    """Captured calls of both kernels that share a workspace, replayed in turn at other lengths."""
    heads = (32, 2, 8, 64)
    shape = saga.SagaShape.of(1, *heads, 2000)
    g = torch.Generator().manual_seed(17)
    cache, _, _ = _fill(shape, fmt, g)
    pl = torch.zeros(1, dtype=torch.int32).cuda()
    ws = saga.alloc_tree_workspace(shape, 16)
    calls = []
    for T in (2, 16):
        q = torch.randn((1, T, 32, 64), generator=g).to(torch.bfloat16).cuda()
        out = torch.zeros((1, T, 32, 64), device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            saga.saga_tree_attn(shape, q, cache, pl, out, ws)
        calls.append((T, q, out, graph))
    for P in (0, 1900, 130):
        pl.fill_(P)
        for _, _, _, graph in calls + calls:
            graph.replay()
        for T, q, out, _ in calls:
            want = torch.empty_like(out)
            saga.saga_tree_attn(shape, q, cache, pl, want, saga.alloc_tree_workspace(shape, T))
            assert torch.equal(out, want)


def test_rows_of_a_bf16_cache_as_tokens():
    """A bf16 cache's rows, token and head dimensions exchanged, quantised into an 8-bit cache: the same codes as from
    dense rows; and rows that several heads or tokens share (strides of zero)."""
    heads, L = (8, 2, 8, 128), 300
    shape = saga.SagaShape.of(2, *heads, L)
    src, _, _ = _fill(shape, BF16, torch.Generator().manual_seed(18))
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    a, b, c = (saga.alloc_cache(shape, E4M3) for _ in range(3))
    k, v = src.k.transpose(1, 2), src.v.transpose(1, 2)
    saga.saga_kv_store(shape, k, v, a, zero)
    saga.saga_kv_store(shape, k.contiguous(), v.contiguous(), b, zero)
    for x, y in zip(a._tensors(), b._tensors()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    one = k[:1, :1, :1]
    saga.saga_kv_store(shape, one.expand(2, L, 2, 128), one.expand(2, L, 8, 128), c, zero)
    for x, y in ((c.k, a.k), (c.v, a.k), (c.k_scale, a.k_scale), (c.v_scale, a.k_scale)):
        assert (x.view(torch.uint8) == y[:1, :1, :1].view(torch.uint8)).all() if x.dim() == 4 else (x == y[0, 0, 0]).all()
