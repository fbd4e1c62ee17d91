"""Cases and plain forms of the operators around a served SAGA cache: per-head norm and position rotation of a
projection's rows with the append to the cache, the 8-bit (e4m3) cache's store and load, and attention of drafted
tokens (a tree, a chain or a single token) over either cache.

With `own` false, run() computes the operators from elementary torch operations in 32 bits; with `own` true it
makes the library's calls.  Layouts: rows q [B, T, h_q, d], k [B, T, h_k, d], v [B, T, h_v, d]; caches
[B, h, l_cap, d] with one fp32 scale per (batch, head, row) in the 8-bit format.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100

# (h_q, h_k, h_v, d) of the synthetic configurations, the sweep and a few others of the library's range
HEADS = {
    "tiny": (8, 1, 8, 64),
    "llama_saga": (32, 2, 8, 64),
    "qwen_saga": (12, 1, 4, 128),
    "llama_hk1": (32, 1, 8, 64),
    "llama_hk4": (32, 4, 8, 64),
    "llama_gqa": (32, 8, 8, 64),
    "fewer_values": (16, 4, 2, 64),
    "wide": (16, 2, 4, 128),
}


def listed():
    return [
        # one new token of one sequence: the latency of a decode step's rotation and append
        _norm_rope("norm_rope_decode1_qwen", "qwen_saga", 1, 1, 1024, "bf16", norm=True),
        # a batch of drafted trees, ragged, quantised as it is written
        _norm_rope("norm_rope_tree_b16_e4m3", "llama_saga", 16, 8, 640, "e4m3", norm=True, ragged=True),
        # a prompt straight from a packed projection
        _norm_rope("norm_rope_prompt_8k", "llama_saga", 1, 8191, 8200, "bf16", norm=True, packed=True),
        # two prompts, half of each head rotated in neighbouring pairs, no norm, quantised as they are written
        _norm_rope("norm_rope_prompt_e4m3_partial", "qwen_saga", 2, 4097, 4224, "e4m3", rot=64, interleaved=True,
                   ragged=True),
        # a whole 128K history quantised at once
        _store("store_history_128k", "qwen_saga", 1, 131072, 131072),
        # ragged histories read back (an exact threshold refresh reads bf16 keys)
        _load("load_history_b4_32k", "llama_saga", 4, 32767, 32768, ragged=True),
        # a short chain of drafted tokens over a short cache
        _tree("tree_chain_tiny_1k", "tiny", 1, 4, 1019, 1024, "bf16", chain=True),
        # a drafted tree over a 32K cache
        _tree("tree_llama_saga_32k", "llama_saga", 1, 8, 32768, 32832, "bf16"),
        # one token over a 128K cache in 8 bits: a decode step on the quantised cache
        _tree("tree_one_token_qwen_128k_e4m3", "qwen_saga", 1, 1, 131071, 131072, "e4m3", chain=True),
        # a drafted tree over a 128K cache in 8 bits
        _tree("tree_qwen_128k_e4m3", "qwen_saga", 1, 16, 131072, 131136, "e4m3"),
        # drafted tokens under the stale Atop-N thresholds, as a reuse step of the decode call selects
        _tree("tree_qwen_128k_atopn", "qwen_saga", 1, 4, 131072, 131136, "bf16", n_top=512),
        # wide trees over ragged dense caches
        _tree("tree_dense_gqa_b8_ragged", "llama_gqa", 8, 64, 16384, 16448, "bf16", ragged=True),
    ]


def _norm_rope(name, heads, batch, tokens, l_cap, fmt, norm=False, rot=0, interleaved=False, packed=False,
               ragged=False):
    d = HEADS[heads][3]
    return {"name": name, "op": "norm_rope", "heads": heads, "batch": batch, "tokens": tokens, "l_cap": l_cap,
            "format": fmt, "norm": norm, "rot": rot or d, "interleaved": interleaved, "packed": packed,
            "ragged": ragged}


def _store(name, heads, batch, tokens, l_cap, ragged=False):
    return {"name": name, "op": "store", "heads": heads, "batch": batch, "tokens": tokens, "l_cap": l_cap,
            "format": "e4m3", "ragged": ragged}


def _load(name, heads, batch, tokens, l_cap, ragged=False):
    return {"name": name, "op": "load", "heads": heads, "batch": batch, "tokens": tokens, "l_cap": l_cap,
            "format": "e4m3", "ragged": ragged}


def _tree(name, heads, batch, tokens, prefix, l_cap, fmt, chain=False, n_top=0, ragged=False):
    return {"name": name, "op": "tree", "heads": heads, "batch": batch, "tokens": tokens, "prefix": prefix,
            "l_cap": l_cap, "format": fmt, "chain": chain, "n_top": n_top, "ragged": ragged}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "store", "load", "tree", "tree", "tree"])
    heads = rng.choice(sorted(HEADS))
    h_q, h_k, h_v, d = HEADS[heads]
    batch = _log_int(rng, 1, 16)
    fmt = rng.choice(["bf16", "e4m3"])
    ragged = rng.random() < 0.5
    if op == "norm_rope":
        tokens = _log_int(rng, 1, 8191)
        while batch > 1 and batch * tokens * (h_q + h_k + h_v) * d > 8191 * 42 * 64:
            batch = batch // 2
        c = _norm_rope("", heads, batch, tokens, tokens + _log_int(rng, 1, 256), fmt, norm=rng.random() < 0.6,
                       rot=rng.choice([0, d // 2, d // 4]), interleaved=rng.random() < 0.4,
                       packed=rng.random() < 0.5, ragged=ragged)
    elif op in ("store", "load"):
        tokens = _log_int(rng, 1, 131072)
        batch = max(1, min(batch, 131072 * 5 * 128 // (tokens * (h_k + h_v) * d)))
        tokens = min(tokens, 131072 * 5 * 128 // (batch * (h_k + h_v) * d))
        c = (_store if op == "store" else _load)("", heads, batch, tokens, tokens + rng.randrange(0, 64), ragged)
    else:
        tokens = _log_int(rng, 1, 64)
        prefix = _log_int(rng, 1, 131072)
        # within the largest listed cases: cached elements, and scores
        prefix = min(prefix, 131072 * 5 * 128 // ((h_k + h_v) * d))
        batch = max(1, min(batch, 131072 * 5 * 128 // (prefix * (h_k + h_v) * d)))
        most = 8 * 64 * 32 * 16384 * 64 // 2
        batch = max(1, min(batch, most // (prefix * tokens * h_q * d)))
        tokens = max(1, min(tokens, most // (prefix * batch * h_q * d)))
        chain = rng.random() < 0.3
        n_top = rng.choice([0, 0, 64, 256]) if prefix >= 1024 else 0
        c = _tree("", heads, batch, tokens, prefix, prefix + tokens + rng.randrange(0, 64), fmt, chain, n_top, ragged)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _counts(case):
    """Valid tokens of each batch row (norm_rope, store, load, tree)."""
    B, T = case["batch"], case["tokens"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T - (b * 5 * T) // (8 * B)) for b in range(B)]


def _prefixes(case):
    B, P = case["batch"], case["prefix"]
    if not case["ragged"]:
        return [P] * B
    return [max(0, P - (b * 7 * P) // (8 * B)) for b in range(B)]


def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _empty_cache(case):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, cap = case["batch"], case["l_cap"]
    if case["format"] == "bf16":
        return {"k": torch.zeros((B, h_k, cap, d), dtype=torch.bfloat16, device="cuda"),
                "v": torch.zeros((B, h_v, cap, d), dtype=torch.bfloat16, device="cuda")}
    return {"k": torch.zeros((B, h_k, cap, d), dtype=torch.float8_e4m3fn, device="cuda"),
            "v": torch.zeros((B, h_v, cap, d), dtype=torch.float8_e4m3fn, device="cuda"),
            "k_scale": torch.zeros((B, h_k, cap), dtype=torch.float32, device="cuda"),
            "v_scale": torch.zeros((B, h_v, cap), dtype=torch.float32, device="cuda")}


def _rows(case, g):
    """New rows q, k, v of every token: slices of one packed projection, or tensors of their own."""
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T = case["batch"], case["tokens"]
    # magnitudes differ from token to token and from head to head, as projections' outputs do
    packed = _randn(g, B, T, (h_q + h_k + h_v), d) * torch.exp(0.5 * _randn(g, B, T, 1, 1)) * \
        torch.exp(0.5 * _randn(g, 1, 1, h_q + h_k + h_v, 1))
    packed = packed.to(torch.bfloat16)
    q, k, v = packed[:, :, :h_q], packed[:, :, h_q:h_q + h_k], packed[:, :, h_q + h_k:]
    if not case.get("packed"):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v


def prepare(case, seed):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T, cap, op = case["batch"], case["tokens"], case["l_cap"], case["op"]
    g = _gen(seed)
    s = {"case": case, "counts": _ints(_counts(case)) if case["ragged"] else None}
    if op == "norm_rope":
        s["q"], s["k"], s["v"] = _rows(case, g)
        starts = torch.randint(0, cap - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["starts"] = starts
        # drafted tokens sit at their depth in the tree, a prompt's tokens one after the other; sequences that
        # were cut from the front keep far positions
        depth = torch.arange(T, device="cuda", dtype=torch.int32)
        if T <= 64:
            depth = torch.minimum(depth, torch.randint(0, T, (T,), generator=g, device="cuda", dtype=torch.int32))
        far = torch.randint(0, 131072, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = (starts[:, None] + far + depth[None]).contiguous()
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
                                      / case["rot"])).float()
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.2 * _randn(g, d)).to(torch.bfloat16)
            s["k_weight"] = (1 + 0.2 * _randn(g, d)).to(torch.bfloat16)
        s["cache"] = _empty_cache(case)
        s["q_out"] = torch.zeros((B, T, h_q, d), dtype=torch.bfloat16, device="cuda")
    elif op == "store":
        _, s["k"], s["v"] = _rows(case, g)
        s["starts"] = torch.randint(0, cap - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["cache"] = _empty_cache(case)
    elif op == "load":
        s["cache"] = _filled(case, g)[0]
        s["k_out"] = torch.zeros((B, h_k, T, d), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros((B, h_v, T, d), dtype=torch.bfloat16, device="cuda")
    else:
        s["prefix"] = _ints(_prefixes(case))
        s["cache"], keys = _filled(case, g)
        s["q"] = _queries(case, g, keys, s["prefix"])
        s["mask"] = None if case["chain"] else _trees(case, g)
        s["tau"] = _thresholds(case, s) if case["n_top"] else None
        s["out"] = torch.zeros((B, T, h_q, d), dtype=torch.bfloat16, device="cuda")
    if own:
        _handles(s)
    return s


def _filled(case, g):
    """A cache with every row written (rows past the valid ones hold what an earlier sequence left there), and its
    keys before any quantisation."""
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, cap = case["batch"], case["l_cap"]
    u = _randn(g, B, h_k, 1, d)
    k = _randn(g, B, h_k, cap, d)
    # one key in a hundred resembles its head's queries
    like = torch.rand((B, h_k, cap, 1), generator=g, device="cuda") < 0.01
    k = torch.where(like, 0.7 * u + 0.3 * k, k)
    v = _randn(g, B, h_v, cap, d)
    cache = _empty_cache(case)
    if case["format"] == "bf16":
        cache["k"].copy_(k)
        cache["v"].copy_(v)
    else:
        for name, x in (("k", k), ("v", v)):
            codes, scale = _quantised(x.to(torch.bfloat16).float())
            cache[name].copy_(codes)
            cache[name + "_scale"].copy_(scale)
    return cache, (k, u)


def _queries(case, g, keys, prefix):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T = case["batch"], case["tokens"]
    k, u = keys
    # each query head: the mean of 16 cached keys and the head's direction, with a token's own noise
    pick = (torch.rand((B, h_q, 16), generator=g, device="cuda") * prefix.clamp(min=1)[:, None, None]).long()
    group = torch.arange(h_q, device="cuda") * h_k // h_q
    src = k[torch.arange(B, device="cuda")[:, None, None], group[None, :, None], pick]
    base = 0.7 * src.mean(dim=2) + 0.3 * u[:, group, 0]
    return (base[:, None] + 0.3 * _randn(g, B, T, h_q, d)).to(torch.bfloat16)


def _trees(case, g):
    """Random trees: token t's parent is one of the four tokens before it, or the cache's end; the mask of a token
    holds itself and its ancestors."""
    B, T = case["batch"], case["tokens"]
    back = torch.randint(1, 5, (B, T), generator=g, device="cuda").cpu().tolist()
    masks = []
    for b in range(B):
        row = []
        for t in range(T):
            parent = t - back[b][t]
            row.append((row[parent] if parent >= 0 else 0) | (1 << t))
        masks.append([m - (1 << 64) if m >= 1 << 63 else m for m in row])
    return torch.tensor(masks, dtype=torch.int64).cuda()


def _thresholds(case, s):
    """One threshold per (batch, query head), shared by the drafted tokens: midway in the widest gap near the score
    of rank n_top * T of theirs."""
    h_q = HEADS[case["heads"]][0]
    B, T = case["batch"], case["tokens"]
    scores = _scores(s, torch.float32)  # [B, T, h_q, cap], -inf where hidden
    flat = scores.permute(0, 2, 1, 3).reshape(B * h_q, -1)
    n = min(case["n_top"] * T, flat.shape[1] - 40)
    top = flat.topk(min(n + 32, flat.shape[1]), dim=1).values
    window = top[:, max(0, n - 32):]
    window = torch.where(torch.isfinite(window), window, window[:, :1])
    gap = window[:, :-1] - window[:, 1:]
    at = gap.argmax(dim=1, keepdim=True)
    return (0.5 * (window.gather(1, at) + window.gather(1, at + 1))).reshape(B, h_q).contiguous()


# ------------------------------------------------------------------------------------------------ the library's calls
def _handles(s):
    from long_context_decoding_saga_b200 import saga
    case = s["case"]
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    s["saga"] = saga
    s["shape"] = saga.SagaShape.of(case["batch"], h_q, h_k, h_v, d, case["l_cap"])
    c = s["cache"]
    s["kv"] = saga.KVCache(c["k"], c["v"], c.get("k_scale"), c.get("v_scale"))
    if case["op"] == "tree":
        s["workspace"] = saga.alloc_tree_workspace(s["shape"], case["tokens"])


def _run_own(s):
    saga, case = s["saga"], s["case"]
    op, shape, kv = case["op"], s["shape"], s["kv"]
    if op == "norm_rope":
        saga.saga_norm_rope_append(shape, s["q"], s["k"], s["v"], kv, s["starts"], s["q_out"],
                                   positions=s["positions"], counts=s["counts"], norm=case["norm"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                   inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        return [s["q_out"], s["cache"]]
    if op == "store":
        saga.saga_kv_store(shape, s["k"], s["v"], kv, s["starts"], counts=s["counts"])
        return s["cache"]
    if op == "load":
        saga.saga_kv_load(shape, kv, 0, case["tokens"], s["k_out"], s["v_out"], lens=s["counts"])
        return [s["k_out"], s["v_out"]]
    saga.saga_tree_attn(shape, s["q"], kv, s["prefix"], s["out"], s["workspace"], tree_mask=s["mask"],
                        counts=s["counts"], tau=s["tau"])
    return s["out"]


# ------------------------------------------------------------------------------------------------ plain forms
def _valid(case, s, T):
    """[B, T]: tokens that are there."""
    t = torch.arange(T, device="cuda")[None]
    n = s["counts"].long()[:, None] if s["counts"] is not None else case["tokens"]
    return (t < n).expand(case["batch"], T)


def _rotated(x, s, interleaved, rot):
    """The position rotation of the first `rot` elements of each head; x [B, T, h, d] in the working type."""
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _normed(x, weight):
    return x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * weight.to(x.dtype)


def _quantised(x):
    """e4m3 codes and fp32 scales, one scale per row of d elements."""
    amax = x.abs().amax(dim=-1, keepdim=True).clamp(min=AMAX_FLOOR)
    codes = (x * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, (amax / E4M3_MAX)[..., 0]


def _append(case, s, k, v):
    """Rows k, v [B, T, h, d] (32 bits) into the cache at starts[b] + t; rows of missing tokens are kept."""
    B, T = case["batch"], case["tokens"]
    valid = _valid(case, s, T)
    b = torch.arange(B, device="cuda")[:, None]
    at = s["starts"].long()[:, None] + torch.arange(T, device="cuda")[None]
    cache = s["cache"]
    _append_one(case, cache, "k", k, b, at, valid)
    _append_one(case, cache, "v", v, b, at, valid)


def _append_one(case, cache, name, x, b, at, valid):
    x = x.float()
    if case["format"] == "bf16":
        old = cache[name].transpose(1, 2)[b, at]
        cache[name].transpose(1, 2)[b, at] = torch.where(valid[..., None, None], x.to(torch.bfloat16), old)
        return
    codes, scale = _quantised(x)
    as_bytes = cache[name].view(torch.uint8).transpose(1, 2)
    as_bytes[b, at] = torch.where(valid[..., None, None], codes.view(torch.uint8), as_bytes[b, at])
    scales = cache[name + "_scale"].transpose(1, 2)
    scales[b, at] = torch.where(valid[..., None], scale, scales[b, at])


def _values(cache, name, dtype):
    x = cache[name].to(dtype)
    return x * cache[name + "_scale"].to(dtype)[..., None] if name + "_scale" in cache else x


def _visible(case, s):
    """[B, T, cap]: the cache rows that a drafted token attends to: the prefix, and what its tree mask holds."""
    T, cap = case["tokens"], case["l_cap"]
    row = torch.arange(cap, device="cuda")[None, None]
    prefix = s["prefix"].long()[:, None, None]
    u = row - prefix
    n = s["counts"].long()[:, None, None] if s["counts"] is not None else T
    if s["mask"] is None:
        seen = u <= torch.arange(T, device="cuda")[None, :, None]
    else:
        seen = ((s["mask"][:, :, None] >> u.clamp(0, 63)) & 1).bool()
    return (u < 0) | ((u < n) & seen)


def _scores(s, dtype):
    """[B, T, h_q, cap] scaled scores, -inf where a token does not attend."""
    case = s["case"]
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T, cap = case["batch"], case["tokens"], case["l_cap"]
    G = h_q // h_k
    q = s["q"].to(dtype).reshape(B, T, h_k, G, d).permute(0, 2, 1, 3, 4).reshape(B, h_k, T * G, d)
    scores = (q @ _values(s["cache"], "k", dtype).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    scores = scores.reshape(B, h_k, T, G, cap).permute(0, 2, 1, 3, 4).reshape(B, T, h_q, cap)
    return scores.masked_fill(~_visible(case, s)[:, :, None], -math.inf)


def _attend(s, dtype):
    case = s["case"]
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T, cap = case["batch"], case["tokens"], case["l_cap"]
    scores = _scores(s, dtype)
    if s["tau"] is not None:
        scores = scores.masked_fill(~(scores >= s["tau"].to(dtype)[:, None, :, None]), -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    H = h_q // h_v
    p = p.reshape(B, T, h_v, H, cap).permute(0, 2, 1, 3, 4).reshape(B, h_v, T * H, cap)
    o = p @ _values(s["cache"], "v", dtype)
    return o.reshape(B, h_v, T, H, d).permute(0, 2, 1, 3, 4).reshape(B, T, h_q, d)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        q, k = s["q"].float(), s["k"].float()
        if case["norm"]:
            q, k = _normed(q, s["q_weight"]), _normed(k, s["k_weight"])
        q = _rotated(q, s, case["interleaved"], case["rot"])
        k = _rotated(k, s, case["interleaved"], case["rot"])
        there = _valid(case, s, case["tokens"])[..., None, None]
        s["q_out"].copy_(torch.where(there, q.to(torch.bfloat16), s["q_out"]))
        _append(case, s, k, s["v"])
        return [s["q_out"], s["cache"]]
    if op == "store":
        _append(case, s, s["k"], s["v"])
        return s["cache"]
    T = case["tokens"]
    there = _valid(case, s, T)
    if op == "load":
        k = _values({n: x[:, :, :T] for n, x in s["cache"].items()}, "k", torch.float32)
        v = _values({n: x[:, :, :T] for n, x in s["cache"].items()}, "v", torch.float32)
        there = there[:, None, :, None]
        s["k_out"].copy_(torch.where(there, k.to(torch.bfloat16), s["k_out"]))
        s["v_out"].copy_(torch.where(there, v.to(torch.bfloat16), s["v_out"]))
        return [s["k_out"], s["v_out"]]
    o = _attend(s, torch.float32)
    s["out"].copy_(torch.where(there[..., None, None], o.to(torch.bfloat16), s["out"]))
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    counts = _counts(case)
    n = sum(counts)
    h = h_k + h_v
    eight = case["format"] == "e4m3"
    row = d + 4 if eight else 2 * d  # bytes of one cached row of one head
    if case["op"] == "norm_rope":
        return {"bytes": n * (2 * d * (2 * h_q + h) + h * row + 4) + 2 * case["rot"] + 4 * case["batch"],
                "flops": n * d * (8 * (h_q + h_k) + 2 * h)}
    if case["op"] in ("store", "load"):
        return {"bytes": n * h * (2 * d + row) + 4 * case["batch"], "flops": 2 * n * h * d}
    prefixes = _prefixes(case)
    keys = sum(p + c for p, c in zip(prefixes, counts))
    # under a threshold only kept value rows count: at most n_top for each query head and token
    values = sum(h_v * (p + c) if not case["n_top"] else min(h_v * (p + c), c * h_q * case["n_top"])
                 for p, c in zip(prefixes, counts))
    pairs = sum(c * (p + c) for p, c in zip(prefixes, counts))
    kept = sum(c * (p + c if not case["n_top"] else min(p + c, case["n_top"])) for p, c in zip(prefixes, counts))
    return {"bytes": (h_k * keys + values) * row + n * h_q * d * 4 + 8 * n + 4 * case["batch"],
            "flops": 2 * h_q * d * (pairs + kept)}


# ------------------------------------------------------------------------------------------------ exact values
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one batch row (and one key head) at a time."""
    s = prepare(case, seed)
    h_q, h_k, h_v, d = HEADS[case["heads"]]
    B, T, cap, op = case["batch"], case["tokens"], case["l_cap"], case["op"]
    counts = _counts(case)
    f64 = {"dtype": torch.float64, "device": "cuda"}
    if op in ("norm_rope", "store"):
        out = {"k": torch.zeros((B, h_k, cap, d), **f64), "v": torch.zeros((B, h_v, cap, d), **f64)}
        if case["format"] == "e4m3":
            out["k_scale"] = torch.zeros((B, h_k, cap), **f64)
            out["v_scale"] = torch.zeros((B, h_v, cap), **f64)
        q_out = torch.zeros((B, T, h_q, d), **f64)
        starts = s["starts"].tolist()
        for b in range(B):
            n, lo = counts[b], starts[b]
            rows = {"k": s["k"][b, :n].double(), "v": s["v"][b, :n].double()}
            if op == "norm_rope":
                turn = _exact_turn(s["positions"][b, :n], s["inv_freq"], case["interleaved"], case["rot"], d)
                both = {"q": s["q"][b, :n].double(), "k": rows["k"]}
                for name in ("q", "k"):
                    x = both[name]
                    if case["norm"]:
                        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * s[name + "_weight"].double()
                    both[name] = turn(x)
                q_out[b, :n] = both["q"]
                rows["k"] = both["k"]
            for name in ("k", "v"):
                x = rows[name].transpose(0, 1)  # [h, n, d]
                if case["format"] == "e4m3":
                    big = torch.maximum(x.max(-1).values, -x.min(-1).values).clamp(min=AMAX_FLOOR)
                    out[name + "_scale"][b, :, lo:lo + n] = big / E4M3_MAX
                    x = x * E4M3_MAX / big[..., None]
                out[name][b, :, lo:lo + n] = x
        return [q_out, out] if op == "norm_rope" else out
    cache = s["cache"]
    if op == "load":
        outs = [torch.zeros((B, h, T, d), **f64) for h in (h_k, h_v)]
        for b in range(B):
            n = counts[b]
            for o, name in zip(outs, ("k", "v")):
                o[b, :, :n] = cache[name][b, :, :n].double() * cache[name + "_scale"][b, :, :n, None].double()
        return outs
    out = torch.zeros((B, T, h_q, d), **f64)
    prefixes = _prefixes(case)
    masks = s["mask"].cpu().numpy().view(np.uint64) if s["mask"] is not None else None
    for b in range(B):
        P, n = prefixes[b], counts[b]
        L = P + n
        seen = torch.ones((n, L), dtype=torch.bool)
        for t in range(n):
            word = int(masks[b, t]) if masks is not None else (1 << (t + 1)) - 1
            seen[t, P:] = torch.tensor([bool(word >> u & 1) for u in range(n)])
        seen = seen.cuda()
        for j in range(h_q):
            keys, vals = cache["k"][b, j * h_k // h_q, :L].double(), cache["v"][b, j * h_v // h_q, :L].double()
            if case["format"] == "e4m3":
                keys = keys * cache["k_scale"][b, j * h_k // h_q, :L, None].double()
                vals = vals * cache["v_scale"][b, j * h_v // h_q, :L, None].double()
            a = torch.einsum("td,ld->tl", s["q"][b, :n, j].double(), keys) / math.sqrt(d)
            keep = seen if s["tau"] is None else seen & (a >= s["tau"][b, j].double())
            a = torch.where(keep, a, -math.inf)
            lse = torch.logsumexp(a, dim=1, keepdim=True)
            weights = torch.where(keep, torch.exp(a - torch.where(torch.isfinite(lse), lse, 0.0)), 0.0)
            out[b, :n, j] = torch.einsum("tl,ld->td", weights, vals)
    return out


def _exact_turn(positions, inv_freq, interleaved, rot, d):
    """The rotation as complex products: pair i turns by exp(1j * position * inv_freq[i])."""
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(positions.shape[0], rot // 2).contiguous(),
                    positions.double()[:, None] * inv_freq.double()[None])[:, None]
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)

    def turn(x):
        y = x.clone()
        w = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y
    return turn
