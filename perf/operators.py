"""Cases, inputs and plain forms of the serving operators: add_rmsnorm, linear_w4, paged_append, paged_attention.

The four make up a serving step of the local-MQA block: the residual's addition with the norm (bf16 or 8-bit
output), the projections with 4-bit weights, the rotation and the append to an 8-bit paged cache, and the
attention over that cache.  Definitions:

  add_rmsnorm      h = bf16(x + r);  y = h * rsqrt(mean(h^2) + eps) * w; y in bf16, or in e4m3 with one scale for
                   each group of channels, the smallest power of two 2^e, e in [-100, 120], with amax <= 448 * 2^e.
  linear_w4        out[m, n] = sum_k s[n, k // g] * (q[n, k] - 8) * x[m, k] + b[n]; q in 0..15, two to a byte, the
                   even k in the low half; x in bf16, or in e4m3 with a scale for each group of 128 channels.
  paged_append     token t of sequence i has position ctx_len[i] + t: q and k are rotated there, q is rounded to
                   bf16, k and v are written in e4m3 into slot position % page_size of page
                   block_table[i, position // page_size]; one scale for each page and key/value head, as above; a
                   page entered past its first slot keeps a scale that is not smaller than the one it had, and its
                   older values are rounded to the new scale.
  paged_attention  out = softmax(q.k / sqrt(D)) v over the cached positions p with pos - window < p <= pos.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0
FULL = 1 << 30  # a window that reaches every position
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the norm of a decode step: four tokens of the 2B width, 8-bit output for the projections
        {"name": "norm_decode_e4m3", "op": "add_rmsnorm", "M": 4, "N": 2560, "group": 128},
        # the norm of a prefill: 8 sequences of 4096 tokens, bf16 output
        {"name": "norm_prefill_bf16", "op": "add_rmsnorm", "M": 32768, "N": 2560, "group": 0},
        # a ragged packed batch of the 9B width, 8-bit output with finer scales
        {"name": "norm_ragged_e4m3", "op": "add_rmsnorm", "M": 4099, "N": 4096, "group": 64},
        # out_proj of one token
        {"name": "w4_one_token", "op": "linear_w4", "M": 1, "N": 2560, "K": 2560, "group": 128, "act8": False},
        # the MLP's up projection of a small decode batch, 8-bit activations
        {"name": "w4_batch_act8", "op": "linear_w4", "M": 8, "N": 7680, "K": 2560, "group": 128, "act8": True},
        # a larger batch at the 9B width with finer groups, an odd number of rows and of outputs
        {"name": "w4_wide_batch", "op": "linear_w4", "M": 37, "N": 12289, "K": 4096, "group": 32, "act8": False},
        # one token for each of 256 sequences: latency counts
        {"name": "append_decode", "op": "paged_append", "S": 256, "new": 1, "ragged": False, "ctx": 8192, "H": 10,
         "Hkv": 1, "D": 256, "page": 64, "window": 2048},
        # prompts of up to 4096 tokens, the first of their documents
        {"name": "append_prompts", "op": "paged_append", "S": 8, "new": 4096, "ragged": True, "ctx": 0, "H": 10,
         "Hkv": 1, "D": 256, "page": 64, "window": 2048},
        # chunks of several lengths that begin and end inside pages, four key/value heads
        {"name": "append_chunks_gqa", "op": "paged_append", "S": 37, "new": 300, "ragged": True, "ctx": 5000, "H": 16,
         "Hkv": 4, "D": 128, "page": 16, "window": 2048},
        # a decode batch of the 2B layout: 256 sequences inside the 2048-token window
        {"name": "attend_decode_batch", "op": "paged_attention", "S": 256, "new": 1, "ragged": False, "ctx": 16384,
         "H": 10, "Hkv": 1, "D": 256, "page": 64, "window": 2048},
        # one token of one sequence over a long cache without a window
        {"name": "attend_one_long", "op": "paged_attention", "S": 1, "new": 1, "ragged": False, "ctx": 131072, "H": 10,
         "Hkv": 1, "D": 256, "page": 64, "window": FULL},
        # chunks of prompts after a cached context, ragged, inside the window
        {"name": "attend_chunks", "op": "paged_attention", "S": 5, "new": 256, "ragged": True, "ctx": 8192, "H": 10,
         "Hkv": 1, "D": 256, "page": 32, "window": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_rmsnorm", "linear_w4", "paged_append", "paged_attention"])
    if op == "add_rmsnorm":
        group = rng.choice([0, 0, 32, 64, 128])
        M, N = _log(rng, 1, 32768), 128 * rng.randint(4, 40)
        if group == 0:
            N += 8 * rng.randint(0, 15)
        M = max(1, min(M, 32768 * 2560 // N))
        return {"op": op, "M": M, "N": N, "group": group}
    if op == "linear_w4":
        group = rng.choice([32, 64, 128])
        return {"op": op, "M": _log(rng, 1, 64), "N": _log(rng, 200, 12288), "K": 128 * rng.randint(4, 40),
                "group": group, "act8": rng.random() < 0.5}
    D = rng.choice([128, 256])
    Hkv = rng.choice([1, 1, 2, 4])
    G = rng.choice([1, 2, 4, 5, 8, 10])
    page = rng.choice([16, 32, 64, 128])
    if op == "paged_append":
        S = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 65536 // (S * Hkv * (G + 2))))
        return {"op": op, "S": S, "new": new, "ragged": rng.random() < 0.7, "ctx": rng.choice([0, _log(rng, 10, 16384)]),
                "H": G * Hkv, "Hkv": Hkv, "D": D, "page": page, "window": 2048}
    S = _log(rng, 1, 192)
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 200)])
    keys = max(64, min(131072, (1 << 18) // (S * Hkv)))
    window = rng.choice([FULL, 2048, _log(rng, 17, 4000)])
    ctx = _log(rng, 20, 65536) if window < FULL else _log(rng, 20, keys)
    new = max(1, min(new, 4096 // S))
    if window < FULL:
        window = max(17, min(window, keys))
    return {"op": op, "S": S, "new": new, "ragged": rng.random() < 0.7, "ctx": ctx, "H": G * Hkv, "Hkv": Hkv, "D": D,
            "page": page, "window": window}


def _lengths(case):
    """Cached and new lengths of each sequence: fixed by the case, so that its work is."""
    r = np.random.default_rng(case["S"] * 7919 + case["new"] * 31 + case["ctx"])
    S = case["S"]
    ctx = r.integers(case["ctx"] // 2, case["ctx"] + 1, S) if S > 1 else np.array([case["ctx"]])
    if case["ragged"]:
        new = r.integers(0 if case["new"] > 1 else 1, case["new"] + 1, S)
        new[r.integers(0, S)] = case["new"]
    else:
        new = np.full(S, case["new"])
    return ctx.astype(np.int64), new.astype(np.int64)


# ------------------------------------------------------------------------------------------------------ the inputs
def _batch(case, g, window):
    """The packed batch that a scheduler hands to both cache operators: pages in no order, those that lie wholly
    before the window given back (-1 in the table)."""
    ctx, new = _lengths(case)
    S, ps = case["S"], case["page"]
    total = ctx + new
    pages = -(-total // ps)
    first = np.maximum(ctx - window + 1, 0) // ps
    r = np.random.default_rng(g)
    held = np.maximum(pages - first, 0)
    P = int(held.sum()) + 3
    order = r.permutation(P).astype(np.int32)
    table = np.full((S, int(max(1, pages.max()))), -1, np.int32)
    at = 0
    for i in range(S):
        table[i, first[i]:pages[i]] = order[at:at + held[i]]
        at += int(held[i])
    pad = 3 if case["ragged"] else 0  # rows behind the last sequence
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return {"cu": torch.from_numpy(cu).cuda(), "ctx": torch.from_numpy(ctx.astype(np.int32)).cuda(),
            "table": torch.from_numpy(table).cuda(), "rows": int(cu[-1]) + pad, "pages": P, "spare": int(order[-1]),
            "max_new": int(new.max()), "max_total": int(total.max())}


def _exponent(amax):
    """The smallest e in [-100, 120] with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.full_like(e, -100)).clamp(-100, 120)


def _filled(shape, gen):
    """A cache that earlier steps wrote: codes, and their scales a page and head, pages of different sizes."""
    codes = torch.empty(shape, dtype=E4M3, device="cuda")
    scale = torch.empty(shape[:2], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 25) // (shape[1] * shape[2] * shape[3]))
    for a in range(0, shape[0], step):
        n = min(step, shape[0] - a)
        x = torch.randn((n,) + shape[1:], generator=gen, device="cuda")
        x = x * torch.exp(0.5 * torch.randn((n, shape[1], 1, 1), generator=gen, device="cuda"))
        s = torch.exp2(_exponent(x.abs().amax((2, 3))).float())
        scale[a:a + n] = s
        codes[a:a + n] = (x / s[:, :, None, None]).to(E4M3)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    s = {"case": dict(case), "op": case["op"]}

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "add_rmsnorm":
        M, N = case["M"], case["N"]
        s["x"] = randn(M, N).bfloat16()
        s["r"] = (3 * randn(M, N)).bfloat16()
        s["w"] = 1 + 0.1 * randn(N)
        s["h"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        if case["group"]:
            s["out"] = torch.zeros(M, N, dtype=E4M3, device="cuda")
            s["scale"] = torch.zeros(M, N // case["group"], device="cuda")
        else:
            s["out"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "linear_w4":
        M, N, K = case["M"], case["N"], case["K"]
        s["W"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["ws"] = ((0.5 + torch.rand(N, K // case["group"], generator=gen, device="cuda")) / 4 / math.sqrt(K)).bfloat16()
        s["b"] = 0.1 * randn(N)
        x = randn(M, K)
        if case["act8"]:
            s["xs"] = torch.exp2(_exponent(x.reshape(M, K // 128, 128).abs().amax(2)).float())
            s["x"] = (x.reshape(M, K // 128, 128) / s["xs"][:, :, None]).reshape(M, K).to(E4M3)
        else:
            s["x"], s["xs"] = x.bfloat16(), None
        s["out"] = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        return s
    window = case["window"]
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    s["batch"] = b = _batch(case, int(seed), window)
    shape = (b["pages"], Hkv, case["page"], D)
    s["kc"], s["ks"] = _filled(shape, gen)
    s["vc"], s["vs"] = _filled(shape, gen)
    if case["op"] == "paged_append":
        s["qkv"] = (1.5 * randn(b["rows"], (H + 2 * Hkv) * D)).bfloat16()
        s["q"] = torch.zeros(b["rows"], H * D, dtype=torch.bfloat16, device="cuda")
        s["workspace"] = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    else:
        s["q"] = randn(b["rows"], H * D).bfloat16()
        s["out"] = torch.zeros(b["rows"], H * D, dtype=torch.bfloat16, device="cuda")
        s["workspace"] = torch.zeros(24 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------- the plain forms
def _plain_add_rmsnorm(s):
    group = s["case"]["group"]
    h = (s["x"].float() + s["r"].float()).bfloat16()
    x = h.float()
    y = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["w"]
    if not group:
        return {"h": h, "out": y.bfloat16()}
    y = y.reshape(y.shape[0], -1, group)
    scale = torch.exp2(_exponent(y.abs().amax(2)).float())
    return {"h": h, "out": (y / scale[:, :, None]).reshape(h.shape).to(E4M3), "scale": scale}


def _plain_linear_w4(s):
    W = torch.stack([s["W"] & 15, s["W"] >> 4], 2).reshape(s["W"].shape[0], -1).float() - 8
    W = (W.reshape(W.shape[0], s["ws"].shape[1], -1) * s["ws"].float()[:, :, None]).reshape(W.shape)
    x = s["x"].float()
    if s["xs"] is not None:
        x = (x.reshape(x.shape[0], -1, 128) * s["xs"][:, :, None]).reshape(x.shape)
    return {"out": (x @ W.t() + s["b"]).bfloat16()}


def _rotate(x, pos):
    """x [rows, heads, D] at positions [rows], the pairs (x[i], x[i + D/2])."""
    half = x.shape[2] // 2
    inv = ROPE_BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) * 2 / x.shape[2])
    a = pos.double()[:, None] * inv
    c, sn = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    x1, x2 = x[:, :, :half], x[:, :, half:]
    return torch.cat([x1 * c - x2 * sn, x2 * c + x1 * sn], 2)


def _append_pool(codes, scales, x, page, slot, entered):
    """x [rows, Hkv, D] into (page, slot) of the pool; entered [S]: the page that each sequence's run begins in."""
    P, Hkv, ps, D = codes.shape
    amax = torch.zeros(P, Hkv, device=x.device).scatter_reduce_(0, page[:, None].expand(-1, Hkv), x.abs().amax(2), "amax")
    first = torch.full((P,), ps, device=x.device).scatter_reduce_(0, page, slot, "amin")  # the first slot written
    need = torch.exp2(_exponent(amax).float())
    new = torch.where((first == 0)[:, None], need, torch.maximum(need, scales))
    new = torch.where((first < ps)[:, None], new, scales)
    first = torch.where(first < ps, first, 0)[entered]
    older = (torch.arange(ps, device=x.device) < first[:, None])[:, None, :, None]
    was = codes.view(torch.uint8)[entered]
    again = (was.view(E4M3).float() * (scales / new)[entered][:, :, None, None]).to(E4M3).view(torch.uint8)
    codes.view(torch.uint8)[entered] = torch.where(older, again, was)
    scales.copy_(new)
    codes.view(torch.uint8)[page, :, slot] = (x / new[page][:, :, None]).to(E4M3).view(torch.uint8)


def _plain_paged_append(s):
    b, c = s["batch"], s["case"]
    H, Hkv, D, ps = c["H"], c["Hkv"], c["D"], c["page"]
    rows = torch.arange(b["rows"], device="cuda")
    n = b["cu"][-1]
    at = torch.where(rows < n, rows, 0)  # rows behind the last sequence: the first one's writes again
    seq = torch.searchsorted(b["cu"][1:], at.int(), right=True)
    pos = b["ctx"][seq].long() + at - b["cu"][seq].long()
    x = s["qkv"][at].float().reshape(-1, H + 2 * Hkv, D)
    qk = _rotate(x[:, :H + Hkv], pos)
    page, slot = b["table"][seq, pos // ps].long(), pos % ps
    last = b["table"].shape[1] - 1
    entered = b["table"].gather(1, (b["ctx"].long() // ps).clamp(max=last)[:, None])[:, 0].long()
    entered = torch.where(b["cu"][1:] > b["cu"][:-1], entered, b["spare"])
    _append_pool(s["kc"], s["ks"], qk[:, H:], page, slot, entered)
    _append_pool(s["vc"], s["vs"], x[:, H + Hkv:], page, slot, entered)
    s["q"].copy_(torch.where((rows < n)[:, None], qk[:, :H].reshape(-1, H * D).bfloat16(), s["q"]))
    return {"q": s["q"], "k": s["kc"], "k_scale": s["ks"], "v": s["vc"], "v_scale": s["vs"]}


def _plain_paged_attention(s):
    b, c = s["batch"], s["case"]
    S, H, Hkv, D, ps, window = c["S"], c["H"], c["Hkv"], c["D"], c["page"], c["window"]
    T = b["max_new"]
    span = min(b["max_total"], window + T - 1)
    cu, ctx = b["cu"].long(), b["ctx"].long()
    n = cu[1:] - cu[:-1]
    p = (ctx - window + 1).clamp(min=0)[:, None] + torch.arange(span, device="cuda")       # [S, span]
    inside = p < (ctx + n)[:, None]
    p = torch.where(inside, p, ctx.clamp(min=1)[:, None] - 1)
    page = b["table"][torch.arange(S, device="cuda")[:, None], p // ps].long().clamp(min=0)
    k = s["kc"].view(torch.uint8)[page, :, p % ps].view(E4M3).float() * s["ks"][page][..., None]  # [S, span, Hkv, D]
    v = s["vc"].view(torch.uint8)[page, :, p % ps].view(E4M3).float() * s["vs"][page][..., None]
    t = torch.arange(T, device="cuda")
    row = torch.where(t < n[:, None], cu[:-1, None] + t, b["rows"])                         # [S, T]
    q = s["q"][row.clamp(max=b["rows"] - 1)].float().reshape(S, T, Hkv, H // Hkv, D)
    pos = (ctx[:, None] + t)[:, :, None]                                                    # [S, T, 1]
    see = inside[:, None] & (p[:, None] <= pos) & (p[:, None] > pos - window)               # [S, T, span]
    q = q.permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)
    sc = (q @ k.permute(0, 2, 3, 1) / math.sqrt(D)).reshape(S, Hkv, T, H // Hkv, span)
    sc = torch.where(see[:, None, :, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(sc - m)
    o = (e / e.sum(-1, keepdim=True).clamp(min=1e-30)).reshape(S, Hkv, -1, span) @ v.permute(0, 2, 1, 3)
    o = o.reshape(S, Hkv, T, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(S * T, H * D)
    out = torch.zeros(b["rows"] + 1, H * D, device="cuda")
    out[row.reshape(-1)] = o
    return {"out": out[:-1].bfloat16()}


# -------------------------------------------------------------------------------------------------------- one pass
def _own(s):
    from lm_causal_depthwise_b200 import api
    c = s["case"]
    if s["op"] == "add_rmsnorm":
        if not c["group"]:
            out, h = api.add_rmsnorm(s["x"], s["r"], s["w"], EPS, out=s["out"], residual_out=s["h"])
            return {"h": h, "out": out}
        out, scale, h = api.add_rmsnorm_e4m3(s["x"], s["r"], s["w"], EPS, group=c["group"], out=s["out"],
                                             scale=s["scale"], residual_out=s["h"])
        return {"h": h, "out": out, "scale": scale}
    if s["op"] == "linear_w4":
        return {"out": api.linear_w4(s["x"], s["W"], s["ws"], s["b"], A_scale=s["xs"], out=s["out"])}
    b = s["batch"]
    batch = api.PagedBatch(b["cu"], b["ctx"], b["table"], b["max_new"], b["max_total"])
    cache = api.PagedCache(s["kc"], s["ks"], s["vc"], s["vs"])
    if s["op"] == "paged_append":
        q = api.paged_append(s["qkv"], batch, cache, rope_base=ROPE_BASE, q_out=s["q"], workspace=s["workspace"])
        return {"q": q, "k": cache.k, "k_scale": cache.k_scale, "v": cache.v, "v_scale": cache.v_scale}
    return {"out": api.paged_attention(s["q"], batch, cache, window=c["window"], out=s["out"], workspace=s["workspace"])}


def run(state):
    if own:
        return _own(state)
    return {"add_rmsnorm": _plain_add_rmsnorm, "linear_w4": _plain_linear_w4, "paged_append": _plain_paged_append,
            "paged_attention": _plain_paged_attention}[state["op"]](state)


# -------------------------------------------------------------------------------------------------------- the work
def work(case):
    if case["op"] == "add_rmsnorm":
        M, N, g = case["M"], case["N"], case["group"]
        return {"bytes": M * N * (6 + (1 if g else 2)) + (4 * M * (N // g) if g else 0) + 4 * N, "flops": 6 * M * N}
    if case["op"] == "linear_w4":
        M, N, K, g = case["M"], case["N"], case["K"], case["group"]
        x = M * K * (1 if case["act8"] else 2) + (4 * M * (K // 128) if case["act8"] else 0)
        return {"bytes": N * K // 2 + 2 * N * (K // g) + x + 4 * N + 2 * M * N, "flops": 2 * M * N * K}
    ctx, new = _lengths(case)
    H, Hkv, D, ps = case["H"], case["Hkv"], case["D"], case["page"]
    n, S = int(new.sum()), case["S"]
    if case["op"] == "paged_append":
        pages = int((-(-(ctx + new) // ps) - ctx // ps)[new > 0].sum())
        return {"bytes": n * D * (2 * (H + 2 * Hkv) + 2 * H + 2 * Hkv) + pages * (4 + 8 * Hkv) + 8 * S,
                "flops": n * D * (3 * H + 6 * Hkv)}
    window = case["window"]
    seen = sum(int(np.minimum(np.arange(c, c + m) + 1, window).sum()) for c, m in zip(ctx, new))
    first = np.maximum(ctx - window + 1, 0)
    keys = int((ctx + new - first)[new > 0].sum())
    return {"bytes": keys * Hkv * 2 * D + 8 * Hkv * (keys // ps + S) + 4 * n * H * D + 8 * S,
            "flops": 4 * D * H * seen}


# ------------------------------------------------------------------------------------- what 64 bits give, by itself
def _pow2(amax):
    """2^e, e the smallest in [-100, 120] with amax <= 448 * 2^e, from log2 and one correction."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(-100, 120)
    e = torch.where((amax <= 448 * torch.exp2(e - 1)) & (e > -100), e - 1, e)
    return torch.exp2(torch.where((amax > 448 * torch.exp2(e)) & (e < 120), e + 1, e))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "add_rmsnorm":
        h = s["x"].double() + s["r"].double()
        x = h.bfloat16().double()
        y = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / case["N"] + EPS) * s["w"].double()
        if not case["group"]:
            return {"h": h, "out": y}
        y = y.unflatten(1, (-1, case["group"]))
        sc = _pow2(y.abs().amax(2))
        return {"h": h, "out": (y / sc.unsqueeze(2)).flatten(1), "scale": sc}
    if case["op"] == "linear_w4":
        K = case["K"]
        W = torch.empty(case["N"], K, dtype=torch.float64, device="cuda")
        W[:, 0::2] = (s["W"] % 16).double()
        W[:, 1::2] = (s["W"] // 16).double()
        W = (W - 8) * s["ws"].double().repeat_interleave(case["group"], 1)
        x = s["x"].double()
        if case["act8"]:
            x = x * s["xs"].double().repeat_interleave(128, 1)
        return {"out": torch.matmul(x, W.T) + s["b"].double()}
    b = s["batch"]
    cu, ctx, table = b["cu"].tolist(), b["ctx"].tolist(), b["table"].long()
    H, Hkv, D, ps = case["H"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "paged_attention":
        out = torch.zeros(b["rows"], H * D, dtype=torch.float64, device="cuda")
        for i in range(case["S"]):
            n = cu[i + 1] - cu[i]
            if n == 0:
                continue
            lo, hi = max(0, ctx[i] - case["window"] + 1), ctx[i] + n
            p = torch.arange(lo, hi, device="cuda")
            g = table[i][p // ps]
            q = s["q"][cu[i]:cu[i] + n].double().reshape(n, Hkv, H // Hkv, D)
            at = torch.arange(ctx[i], hi, device="cuda")[:, None]
            hide = (p > at) | (p <= at - case["window"])
            for j in range(Hkv):
                k = s["kc"].view(torch.uint8)[g, j, p % ps].view(E4M3).double() * s["ks"][g, j].double()[:, None]
                v = s["vc"].view(torch.uint8)[g, j, p % ps].view(E4M3).double() * s["vs"][g, j].double()[:, None]
                z = torch.einsum("tgd,pd->tgp", q[:, j], k) / D ** 0.5
                z = z.masked_fill(hide[:, None], -math.inf).softmax(-1)
                o = torch.einsum("tgp,pd->tgd", z, v)
                out.view(-1, Hkv, H // Hkv, D)[cu[i]:cu[i] + n, j] = o
        return {"out": out}
    got = {"q": s["q"].double(), "k": s["kc"].double(), "k_scale": s["ks"].double(), "v": s["vc"].double(),
           "v_scale": s["vs"].double()}
    freq = torch.exp(torch.arange(D // 2, device="cuda", dtype=torch.float64) * (-2 / D * math.log(ROPE_BASE)))
    for i in range(case["S"]):
        n = cu[i + 1] - cu[i]
        if n == 0:
            continue
        x = s["qkv"][cu[i]:cu[i + 1]].double().reshape(n, H + 2 * Hkv, D)
        pos = torch.arange(ctx[i], ctx[i] + n, device="cuda")
        turn = torch.polar(torch.ones(n, 1, D // 2, dtype=torch.float64, device="cuda"), (pos.double()[:, None] * freq)[:, None])
        z = torch.complex(x[:, :H + Hkv, :D // 2].contiguous(), x[:, :H + Hkv, D // 2:].contiguous()) * turn
        qk = torch.cat([z.real, z.imag], 2)
        got["q"][cu[i]:cu[i + 1]] = qk[:, :H].reshape(n, H * D)
        slots = -(-(ctx[i] + n) // ps) * ps - ctx[i] // ps * ps  # those of the pages that are touched
        off = ctx[i] % ps
        pages = table[i, ctx[i] // ps:ctx[i] // ps + slots // ps]
        for name, y in (("k", qk[:, H:]), ("v", x[:, H + Hkv:])):
            for j in range(Hkv):
                full = torch.zeros(slots, D, dtype=torch.float64, device="cuda")
                full[off:off + n] = y[:, j]
                sc = _pow2(full.reshape(-1, ps, D).abs().amax((1, 2)))
                c = got[name][pages, j]
                if off:
                    old = got[name + "_scale"][pages[0], j]
                    sc[0] = torch.maximum(sc[0], old)
                    c[0, :off] *= old / sc[0]
                c.reshape(-1, D)[off:off + n] = (full.reshape(-1, ps, D) / sc[:, None, None]).reshape(-1, D)[off:off + n]
                got[name][pages, j] = c
                got[name + "_scale"][pages, j] = sc
    return got
