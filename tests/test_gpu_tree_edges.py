"""Attention of drafted tokens on the GPU where unseen or bad numbers could get into the results.  Bounds as in
tests/test_gpu_tree.py."""
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


# bit patterns of a bf16 element, of an e4m3 code (all ones but the sign: its only NaN) and of a scale
POISON = {"inf": (0x7F80, 0x7F, float("inf")), "-inf": (-0x80, 0xFF, float("-inf")), "nan": (-1, 0xFF, float("nan")),
          "largest": (0x7F7F, 0x7E, 3.4e38)}


@pytest.mark.parametrize("poison", sorted(POISON))
@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", [((12, 1, 4, 128), 4), ((8, 1, 8, 64), 4), ((32, 2, 8, 64), 16)])
@pytest.mark.parametrize("q_scale,spread", [(1.0, 1.0), (12.0, 4.0)])
def test_rows_that_nobody_sees_may_hold_anything(q_scale, spread, heads, T, fmt, poison):
    """Drafted rows outside every mask and rows past the last token, with an empty prefix (they share their warp with
    every row that is seen), at a tile's end and inside one; scores near zero and far from it."""
    prefixes, l_cap = [0, 125, 300], 400
    shape = saga.SagaShape.of(3, *heads, l_cap)
    g = torch.Generator().manual_seed(40 + T)
    cache, K, V = tree._fill(shape, fmt, g, spread)
    # token 1's row is seen by nobody, not by itself either; token 2 sees nothing of the drafted rows
    masks = [[0 if t == 2 else (1 << t | 1) & ~2 for t in range(T)]] * 3
    bits, code, scale = POISON[poison]
    for b, P in enumerate(prefixes):
        rows = [P + 1, P + 2] + list(range(P + T, l_cap))
        for t in cache._tensors()[:2]:
            (t.view(torch.uint8) if fmt == E4M3 else t.view(torch.int16))[b, :, rows] = code if fmt == E4M3 else bits
        for t in cache._tensors()[2:]:
            if t is not None:
                t[b][:, rows] = scale
    q = (q_scale * torch.randn((3, T, heads[0], heads[3]), generator=g)).to(torch.bfloat16)
    out = torch.empty((3, T, heads[0], heads[3]), device="cuda")
    ws = saga.alloc_tree_workspace(shape, T)
    saga.saga_tree_attn(shape, q.cuda(), cache, _i32(prefixes), out, ws, tree_mask=tree._words(masks).cuda())
    for b, P in enumerate(prefixes):
        exact, bound, _, _ = tree._bounds(q[b].double().numpy(), K[b], V[b], P, T, masks[b], None, heads[3], fmt)
        got = out[b].double().cpu().numpy()
        assert np.isfinite(got).all(), (b, "not finite")
        off = np.abs(got - exact)
        assert (off <= bound).all(), (b, float((off - bound).max()))
    assert saga.saga_get_status(ws) == 0


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", [((12, 1, 4, 128), 2), ((8, 1, 8, 64), 2), ((32, 2, 8, 64), 16), ((8, 1, 1, 128), 16)])
@pytest.mark.parametrize("what,row", [("k", 0), ("k", 130), ("k", 2999), ("v", 131)])
@pytest.mark.parametrize("thresholds", [False, True])
def test_a_nan_that_is_seen_shows(thresholds, heads, T, fmt, what, row):
    """Seen rows have to be finite; a NaN among them makes the outputs that it belongs to NaN, never finite numbers,
    where one CTA holds the item (a batch row of few tiles) and where several do."""
    h_q, h_k, h_v, d = heads
    prefixes = [3000, 200] if row < 200 else [3000, 3000]
    shape = saga.SagaShape.of(2, *heads, 3000 + T)
    g = torch.Generator().manual_seed(50 + T)
    cache, K, V = tree._fill(shape, fmt, g)
    q = torch.randn((2, T, h_q, d), generator=g).to(torch.bfloat16)
    # thresholds below every score
    tau = torch.full((2, h_q), -1e4, device="cuda") if thresholds else None
    calls = []
    for b in range(2):  # the batch row that holds the NaN
        c = saga.KVCache(*[t.clone() for t in cache._tensors() if t is not None])
        t = c.k if what == "k" else c.v
        if fmt == E4M3:
            t.view(torch.uint8)[b, 0, row, 5] = 0x7F
        else:
            t[b, 0, row, 5] = float("nan")
        out = torch.zeros((2, T, h_q, d), device="cuda")
        ws = saga.alloc_tree_workspace(shape, T)
        saga.saga_tree_attn(shape, q.cuda(), c, _i32(prefixes), out, ws, tau=tau)
        assert saga.saga_get_status(ws) == 0
        calls.append(out.cpu())
    clean = torch.zeros((2, T, h_q, d), device="cuda")
    saga.saga_tree_attn(shape, q.cuda(), cache, _i32(prefixes), clean, saga.alloc_tree_workspace(shape, T), tau=tau)
    clean = clean.cpu()
    assert torch.isfinite(clean).all()
    for b, out in enumerate(calls):
        hit = torch.zeros((2, T, h_q, d), dtype=torch.bool)
        if what == "k":
            hit[b, :, :h_q // h_k] = True  # every output of the key head's queries
        else:
            hit[b, :, :h_q // h_v, 5] = True
        assert torch.isnan(out[hit]).all(), (b, int(torch.isfinite(out[hit]).sum()))
        assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("fmt", [BF16, E4M3])
@pytest.mark.parametrize("heads,T", [((12, 1, 4, 128), 2), ((8, 1, 8, 64), 2), ((32, 2, 8, 64), 16), ((8, 1, 1, 128), 16)])
def test_a_wait_that_runs_out_is_flagged_and_the_context_stays_usable(heads, T, fmt):
    """The products of every CTA with tiles wait in vain for 2 ms; the CTA gives up and unwinds: the call returns, the
    status word says so, and the next calls, on the same workspace and on a fresh one, are right."""
    h_q, h_k, h_v, d = heads
    shape = saga.SagaShape.of(2, *heads, 3000 + T)
    g = torch.Generator().manual_seed(60 + T)
    cache, K, V = tree._fill(shape, fmt, g)
    q = torch.randn((2, T, h_q, d), generator=g).to(torch.bfloat16)
    prefixes = [3000, 200]
    ws = saga.alloc_tree_workspace(shape, T)
    args = (shape, q.cuda(), cache, _i32(prefixes))
    saga.saga_test_expire_next_wait(2_000_000)
    saga.saga_tree_attn(*args, torch.empty((2, T, h_q, d), device="cuda"), ws)
    torch.cuda.synchronize()
    assert saga.saga_get_status(ws) == saga.SAGA_STATUS_TIMEOUT
    ws2 = saga.alloc_tree_workspace(shape, T)
    outs = []
    for w in (ws, ws2):
        outs.append(torch.empty((2, T, h_q, d), device="cuda"))
        saga.saga_tree_attn(*args, outs[-1], w)
    assert saga.saga_get_status(ws2) == 0
    assert torch.equal(outs[0], outs[1])
    for b, P in enumerate(prefixes):
        exact, bound, _, _ = tree._bounds(q[b].double().numpy(), K[b], V[b], P, T, None, None, d, fmt)
        assert (np.abs(outs[0][b].double().cpu().numpy() - exact) <= bound).all()
