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
