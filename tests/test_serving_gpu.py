"""GPU parity of the serving operators (rglru_add_rmsnorm, rglru_add_rmsnorm_e4m3, rglru_linear_w4,
rglru_paged_append, rglru_paged_attention) against the float64 oracle (oracle/serving.py).

Bars, from the arithmetic.  A rounding is off by at most half a step: bf16 2^-8 relative, f16 2^-11, e4m3
2^-4 relative or 2^-10 of its scale below the normal range.  On top of it comes the fp32 arithmetic before it:
  norm       the sum of squares has at most 64 sequential roundings of 2^-24 per thread and reduction, then a
             square root, a division and two products: 2^-17 of the value, taken as 2^-16.
  linear_w4  operands exact; at most K / 16 + 64 sequential additions, each off by 2^-23 of the largest partial sum
             (a tensor core may truncate), which sum |s q x| bounds.
  append     the angle is a turn in fp32 (2^-25 of it, times 2 pi) and its sine and cosine 2^-23; three
             roundings of 2^-24 follow: 1e-6 (|x1| + |x2|) holds them.  Values are copies: codes of v exact.
  attention  scores: head_dim / 16 + 8 sequential additions off by 2^-23 of sum |q k| scale each; q enters exactly, as
             f16 after a power of two (it has 8 bits), or, in calls with more than 32 rows a sequence and key head, as
             two e4m3 terms, exact down to 2^-9 of the row's largest value and off by 2^-17 of that below: of normal
             values fewer than one in a hundred, so at most 2^-17 * 4 / 100 of sum |q k| * 3, far inside the additions'
             2^-18 and more; k enters exactly; the exponential and its argument 2^-18; a probability enters the second
             product as f16 (2^-11), and the sums are fp32: relative to sum p |v|.
A scale is a power of two: it may differ only where the largest magnitude is within those errors of the border.
"""
import numpy as np
import pytest
import torch

from lm_causal_depthwise_b200 import api
from oracle import serving as O

pytestmark = pytest.mark.gpu

dev = "cuda"
bf = torch.bfloat16
E4 = torch.float8_e4m3fn


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(bf)


def _within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.nanmax(err / tol):.3g} of the bar"


# ------------------------------------------------------------------------------------------------- add_rmsnorm
def _check_norm(x, r, w, eps, group, in_place=None):
    N = x.shape[-1]
    h32 = x.float() if r is None else x.float() + r.float()
    h = h32.to(bf)
    want = O.add_rmsnorm(_np(h), _np(w), eps)
    xd, rd = x.to(dev), None if r is None else r.to(dev)
    ro = {"x": xd, "r": rd, None: None}[in_place]
    if group == 0:
        out, ho = api.add_rmsnorm(xd, rd, w.to(dev), eps, residual_out=ro)
        _within(_np(out), want, (2.0 ** -8 + 2.0 ** -16) * np.abs(want) + 1e-38, f"norm N={N}")
    else:
        out, sc, ho = api.add_rmsnorm_e4m3(xd, rd, w.to(dev), eps, group=group, residual_out=ro)
        g = want.reshape(*want.shape[:-1], N // group, group)
        amax = np.abs(g).max(-1)
        s = _np(sc)
        near = (O.scale_of(amax * (1 - 2.0 ** -16)) == s) | (O.scale_of(amax * (1 + 2.0 ** -16)) == s)
        assert near.all(), "scale"
        got = _np(out).reshape(g.shape) * s[..., None]
        tol = np.maximum(2.0 ** -4 * np.abs(g), 2.0 ** -10 * s[..., None]) + 2.0 ** -16 * np.abs(g)
        _within(got, g, tol, f"norm e4m3 N={N} group={group}")
    assert torch.equal(ho.cpu(), h)
    assert ho.data_ptr() == (xd if r is None else ho if ro is None else ro).data_ptr()


@pytest.mark.parametrize("M,N,group", [(1, 8, 0), (1, 2560, 0), (3, 2560, 128), (5, 32, 32), (7, 4096, 64), (300, 520, 0),
                                       (33, 4608, 256), (2, 16384, 128), (3, 16376, 0), (9, 96, 32), (1000, 256, 256),
                                       (2, 8200, 0), (4, 12288, 32), (150, 1056, 32), (2500, 2560, 128)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_add_rmsnorm(M, N, group, with_residual):
    rng = np.random.default_rng(M * 7 + N)
    x, w = _bf16(rng, M, N), torch.from_numpy((1 + 0.2 * rng.standard_normal(N)).astype(np.float32))
    _check_norm(x, _bf16(rng, M, N, scale=4) if with_residual else None, w, 1e-6, group)


@pytest.mark.parametrize("in_place", ["x", "r"])
@pytest.mark.parametrize("group", [0, 32])
def test_add_rmsnorm_in_place_and_leading_dims(in_place, group):
    rng = np.random.default_rng(1)
    x, r = _bf16(rng, 2, 3, 5, 640), _bf16(rng, 2, 3, 5, 640)
    _check_norm(x, r, torch.ones(640), 1e-5, group, in_place)


def test_add_rmsnorm_extremes():
    """A zero row, huge rows (the sum of squares stays finite), rows below eps, a weight of both signs and zero."""
    rng = np.random.default_rng(2)
    x = _bf16(rng, 6, 512)
    x[1] = 0
    x[2] *= 1e16
    x[3] *= 1e-20
    w = torch.from_numpy(rng.standard_normal(512).astype(np.float32))
    w[:32] = 0
    for group in (0, 32):
        _check_norm(x, None, w, 1e-6, group)
        r = torch.zeros_like(x)
        r[1] = -x[1]
        r[4] = -x[4]                                  # cancels to a zero row
        _check_norm(x, r, w, 1e-6, group)


def test_add_rmsnorm_nan_and_inf_stay_in_their_row():
    rng = np.random.default_rng(3)
    x = _bf16(rng, 5, 256).to(dev)
    x[1, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(256, device=dev)
    clean = x.clone()
    clean[1], clean[3] = 0, 0
    out, _ = api.add_rmsnorm(x, None, w)
    ref, _ = api.add_rmsnorm(clean, None, w)
    q, s, _ = api.add_rmsnorm_e4m3(x, None, w, group=64)
    qr, sr, _ = api.add_rmsnorm_e4m3(clean, None, w, group=64)
    for i in (0, 2, 4):
        assert torch.equal(out[i], ref[i]) and torch.equal(s[i], sr[i])
        assert torch.equal(q[i].view(torch.uint8), qr[i].view(torch.uint8))
    assert out[1].isnan().all() and q[1].float().isnan().all()
    assert out[3, 9].isnan() and (out[3, :9] == 0).all()          # inf * 0
    assert torch.isfinite(s).all()


# --------------------------------------------------------------------------------------------------- linear_w4
def _w4_case(rng, M, N, K, group, a_group, bias=True):
    W = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8))
    s = torch.from_numpy((0.01 + 0.05 * rng.random((N, K // group))).astype(np.float32)).to(bf)
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)) if bias else None
    if a_group:
        A = torch.from_numpy(O.round_e4m3(rng.standard_normal((M, K)) * 100).astype(np.float32)).to(E4)
        sa = torch.from_numpy(np.exp2(rng.integers(-9, -3, (M, K // a_group))).astype(np.float32))
        x = _np(A) * np.repeat(_np(sa), a_group, 1)
    else:
        A, sa = _bf16(rng, M, K), None
        x = _np(A)
    return A, sa, W, s, b, x


def _check_w4(rng, M, N, K, group, a_group=0, bias=True):
    A, sa, W, s, b, x = _w4_case(rng, M, N, K, group, a_group, bias)
    want, size = O.linear_w4(x, W.numpy(), _np(s), None if b is None else _np(b))
    buf = torch.full((M * N + 64,), 77.0, dtype=bf, device=dev)      # a guard behind the output
    out = buf[:M * N].view(M, N)
    got = api.linear_w4(A.to(dev), W.to(dev), s.to(dev), None if b is None else b.to(dev),
                        None if sa is None else sa.to(dev), out=out)
    assert got.data_ptr() == out.data_ptr() and (buf[M * N:] == 77).all()
    tol = 2.0 ** -8 * np.abs(want) + (K / 16 + 64) * 2.0 ** -23 * size + 1e-30
    _within(_np(got), want, tol, f"w4 M={M} N={N} K={K} group={group} a_group={a_group}")


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 31, 33, 48, 49, 64])
@pytest.mark.parametrize("N,K,group,a_group", [(64, 256, 128, 0), (100, 288, 32, 0), (33, 640, 64, 64), (17, 2560, 128, 128)])
def test_linear_w4(M, N, K, group, a_group):
    _check_w4(np.random.default_rng(M * 100 + N), M, N, K, group, a_group)


@pytest.mark.parametrize("M,N,K,group,a_group,bias", [
    (1, 1, 32, 32, 0, False), (1, 1, 32, 32, 32, True), (3, 15, 96, 32, 32, False), (64, 16, 128, 128, 0, True),
    (1, 2560, 2560, 128, 0, True), (8, 769, 7680, 128, 128, True), (37, 1001, 4096, 32, 256, False),
    (64, 300, 5120, 64, 256, True), (2, 4099, 160, 32, 32, True), (20, 40, 20480, 128, 128, True), (4, 9, 192, 64, 32, True)])
def test_linear_w4_sizes(M, N, K, group, a_group, bias):
    _check_w4(np.random.default_rng(N + K), M, N, K, group, a_group, bias)


@pytest.mark.parametrize("M,N,K,group,a_group", [
    (64, 70, 20480, 128, 128), (20, 20001, 128, 128, 0), (48, 20001, 288, 32, 32), (64, 20001, 1280, 64, 0),
    (64, 4300, 12320, 32, 0), (16, 9000, 288, 32, 0), (1, 40, 20480, 64, 128)])
def test_linear_w4_rounds_and_passes(M, N, K, group, a_group):
    """More outputs than the clusters take at once, more of x than shared memory holds, long sums for few rows."""
    _check_w4(np.random.default_rng(M + N + K), M, N, K, group, a_group)


def test_linear_w4_repeats_beside_another_stream():
    """Sums over a cluster in rank order: the same bits each time, also with other projections on a second stream."""
    rng = np.random.default_rng(7)
    cases = []
    for M, N, K in ((40, 1000, 2560), (64, 3000, 384), (20, 500, 5120)):
        A, _, W, s, b, _ = (t if t is None or isinstance(t, np.ndarray) else t.to(dev) for t in _w4_case(rng, M, N, K, 128, 0))
        cases.append((A, W, s, b))
    ref = [api.linear_w4(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append([api.linear_w4(*c) for c in cases])
    torch.cuda.synchronize()
    for o in outs:
        for a, r in zip(o, ref):
            assert torch.equal(a, r)


def test_linear_w4_every_code_at_every_place():
    """One-hot rows read single weights back: the packing order, all 16 codes, every position of a group."""
    N, K, group = 48, 256, 32
    rng = np.random.default_rng(5)
    W = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8))
    s = torch.from_numpy(np.exp2(rng.integers(-3, 3, (N, K // group))).astype(np.float32)).to(bf)
    want = O.unpack_w4(W.numpy()) * np.repeat(_np(s), group, 1)
    got = []
    for k0 in range(0, K, 64):
        A = torch.zeros(64, K, dtype=bf)
        A[torch.arange(64), k0 + torch.arange(64)] = 1
        got.append(_np(api.linear_w4(A.to(dev), W.to(dev), s.to(dev))))
    np.testing.assert_array_equal(np.concatenate(got).T, want)


def test_linear_w4_rows_do_not_depend_on_each_other():
    """A row's result is bit-identical with other rows beside it of the same count, NaN among them."""
    rng = np.random.default_rng(6)
    A, _, W, s, b, _ = _w4_case(rng, 12, 200, 512, 64, 0)
    A, W, s, b = (t.to(dev) for t in (A, W, s, b))
    ref = api.linear_w4(A, W, s, b)
    A2 = A.clone()
    A2[5] = float("nan")
    A2[9] = float("inf")
    got = api.linear_w4(A2, W, s, b)
    keep = [i for i in range(12) if i not in (5, 9)]
    assert torch.equal(got[keep], ref[keep])
    assert got[5].isnan().all() and not torch.isfinite(got[9].float()).any()


# ------------------------------------------------------------------------------------- the paged cache: a small world
class World:
    """Sequences with cached tokens, new ones, and pages in no order; codes and scales random where cached."""

    def __init__(self, seed, ctx, new, H, Hkv, D, page, pad=0, spare=2, window=None, spread=0.7):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.D, self.page = H, Hkv, D, page
        self.ctx, self.new = np.asarray(ctx), np.asarray(new)
        S = len(ctx)
        total = self.ctx + self.new
        self.max_total = int(max(total.max(), 1))
        n = -(-total // page)
        first = np.zeros(S, int) if window is None else np.maximum(self.ctx - window + 1, 0) // page
        held = np.maximum(n - first, 0)
        self.P = int(held.sum()) + spare
        order = rng.permutation(self.P)
        self.table = np.full((S, max(1, -(-self.max_total // page))), -7, np.int32)
        at = 0
        for i in range(S):
            self.table[i, first[i]:n[i]] = order[at:at + held[i]]
            at += held[i]
        self.spare = order[at:]
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + pad
        shape = (self.P, Hkv, page, D)
        self.ks = np.exp2(rng.integers(-9, -5, (self.P, Hkv)).astype(float))
        self.vs = np.exp2(np.round(rng.standard_normal((self.P, Hkv)) * 3) - 7)
        self.k = O.round_e4m3(np.clip(rng.standard_normal(shape) * 120, -448, 448))
        self.v = O.round_e4m3(np.clip(rng.standard_normal(shape) * 120, -448, 448))
        self.qkv = _bf16(rng, self.rows, (H + 2 * Hkv) * D)
        # sizes that differ from row to row, so that scales rise inside pages
        self.qkv = (self.qkv.float() * torch.from_numpy(np.exp(rng.standard_normal((self.rows, 1)) * spread)).float()).to(bf)
        self.q = _bf16(rng, self.rows, H * D, scale=1.5)

    def batch(self, **kw):
        a = dict(cu_tokens=torch.from_numpy(self.cu).to(dev), ctx_len=torch.from_numpy(self.ctx.astype(np.int32)).to(dev),
                 block_table=torch.from_numpy(self.table).to(dev), max_new=int(max(self.new.max(), 1)),
                 max_total=self.max_total)
        a.update(kw)
        return api.PagedBatch(**a)

    def cache(self):
        def codes(x):
            return torch.from_numpy(x.astype(np.float32)).to(E4).to(dev)

        def sc(x):
            return torch.from_numpy(x.astype(np.float32)).to(dev)
        return api.PagedCache(codes(self.k), sc(self.ks), codes(self.v), sc(self.vs))


WORLDS = {  # ctx, new, H, Hkv, D, page, rows behind the last sequence
    "one token": ([0], [1], 1, 1, 256, 16, 0),
    "one token, deep": ([4097], [1], 10, 1, 256, 64, 0),
    "decode batch": ([0, 15, 16, 17, 63, 64, 200, 1], [1] * 8, 10, 1, 256, 64, 0),
    "decode, heads": ([5, 33, 700], [1, 1, 1], 16, 4, 128, 16, 1),
    "decode, one head each": ([40, 41], [1, 1], 3, 3, 256, 32, 0),
    "wide group": ([90, 257], [1, 1], 40, 2, 128, 128, 0),
    "draft tokens": ([10, 30, 64, 0], [4, 3, 5, 2], 10, 1, 256, 32, 3),
    "ragged chunks": ([0, 100, 31, 5, 64], [70, 0, 33, 129, 1], 4, 2, 128, 16, 2),
    "ragged chunks, 256": ([0, 33, 1], [100, 31, 64], 5, 1, 256, 64, 0),
    "none but one": ([7, 7, 7], [0, 2, 0], 2, 1, 256, 16, 5),
    "page of 128": ([0, 130, 127], [300, 128, 2], 2, 2, 256, 128, 0),
    "long prompt": ([0], [700], 2, 1, 128, 32, 0),
}


def _world(name, **kw):
    ctx, new, H, Hkv, D, page, pad = WORLDS[name]
    return World(len(name), ctx, new, H, Hkv, D, page, pad, **kw)


def _check_append(w, base=10000.0, bad_pages=False, **kw):
    cache, ws = w.cache(), api.linear_workspace()
    q_out = torch.full((w.rows, w.H * w.D), 55.0, dtype=bf, device=dev)
    before = [t.clone() for t in (cache.k, cache.v)]
    got = api.paged_append(w.qkv.to(dev), w.batch(**kw), cache, rope_base=base, q_out=q_out, workspace=ws)
    assert got.data_ptr() == q_out.data_ptr()
    assert api.device_status(ws) == (api.ERR_INVALID_ARG if bad_pages else api.OK)
    x = _np(w.qkv).reshape(w.rows, w.H + 2 * w.Hkv, w.D)
    q, pools = O.append(x.reshape(w.rows, -1), w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs, w.H, base)
    mag = np.abs(x[..., :w.D // 2]) + np.abs(x[..., w.D // 2:])
    mag = np.concatenate([mag, mag], -1)                      # |x1| + |x2| of each channel's pair
    live = w.cu[-1]
    _within(_np(got).reshape(q.shape)[:live], q[:live], 2.0 ** -8 * np.abs(q[:live]) + 1e-6 * mag[:live, :w.H], "q")
    assert (got[live:] == 55).all()
    # values are copies: v's codes and scales are the oracle's exactly, and what was not written is untouched
    np.testing.assert_array_equal(_np(cache.v_scale), pools["v"][1])
    np.testing.assert_array_equal(_np(cache.v), pools["v"][0])
    c, s, raw = pools["k"]
    gs = _np(cache.k_scale)
    wrote = ~np.isnan(raw)
    page_top = np.where(wrote, np.abs(raw), 0).max((2, 3))
    border = np.abs(np.exp2(np.round(np.log2(np.maximum(page_top, 1e-300) / 448))) * 448 / np.maximum(page_top, 1e-300) - 1) < 1e-5
    assert ((gs == s) | border).all()
    same = (gs == s)[..., None, None] & ~wrote
    np.testing.assert_array_equal(np.where(same, _np(cache.k), 0), np.where(same, c, 0))
    pair = np.abs(raw[..., :w.D // 2]) + np.abs(raw[..., w.D // 2:])    # at least the pair's size / sqrt(2)
    tol = np.maximum(2.0 ** -4 * np.abs(raw), 2.0 ** -10 * gs[..., None, None]) + 2e-6 * np.concatenate([pair, pair], -1)
    _within((_np(cache.k) * gs[..., None, None])[wrote], raw[wrote], tol[wrote], "k")
    for t, old in zip((cache.k, cache.v), before):
        for page in w.spare:
            assert torch.equal(t[page].view(torch.uint8), old[page].view(torch.uint8))
    return cache


@pytest.mark.parametrize("name", sorted(WORLDS))
def test_paged_append(name):
    _check_append(_world(name))


def test_paged_append_far_positions_and_base():
    w = World(9, [100000, 16777000], [3, 40], 2, 1, 256, 64, window=2048)
    _check_append(w, base=500000.0)


def test_paged_append_token_by_token_is_idempotent_at_a_page():
    """The same token appended twice at the same position leaves the same page: a step may be replayed."""
    w = _world("decode batch")
    cache = _check_append(w)
    snap = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8), cache.v_scale)]
    api.paged_append(w.qkv.to(dev), w.batch(), cache)
    for a, b in zip(snap, (cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8), cache.v_scale)):
        assert torch.equal(a, b)


def test_paged_append_special_values():
    """NaN stays a NaN code, infinities saturate, zeros take the smallest scale, and a raised scale moves the page."""
    w = World(3, [0, 18, 5], [2, 1, 1], 1, 1, 128, 16)
    v = w.qkv.view(-1, 3, 128)
    v[:, 1:] = 0
    v[0, 2, 3], v[0, 2, 4] = float("nan"), 2.0
    v[1, 2, 5] = -float("inf")
    v[2, 2, 0] = 30000.0
    with np.errstate(invalid="ignore"):
        cache = _check_append(w)
    page = w.table[0, 0]
    assert _np(cache.v_scale)[page, 0] == 2.0 ** 120 and _np(cache.v)[page, 0, 1, 5] == -448
    assert np.isnan(_np(cache.v)[page, 0, 0, 3])
    assert _np(cache.k_scale)[page, 0] == 2.0 ** -100


def test_paged_append_bad_pages_and_lengths_are_refused_on_the_device():
    """Page numbers outside the pool, lengths outside the bounds: skipped, recorded, everything else done."""
    w = World(4, [0, 20, 3, 9], [40, 3, 2, 1], 2, 1, 128, 16)
    w.table[0, 1] = w.P
    w.table[2, 0] = -1
    _check_append(w, bad_pages=True)
    w = World(4, [0, 20, 3, 9], [4, 3, 2, 1], 2, 1, 128, 16)
    cache, ws = w.cache(), api.linear_workspace()
    q = torch.full((w.rows, 256), 55.0, dtype=bf, device=dev)
    for kw, skipped in ((dict(max_new=3), [0]), (dict(max_total=22, max_new=4), [1]),
                        (dict(ctx_len=torch.tensor([0, 20, -3, 9], dtype=torch.int32, device=dev)), [2]),
                        (dict(cu_tokens=torch.tensor([0, 4, 7, 9, 11], dtype=torch.int32, device=dev)), [3]),
                        (dict(cu_tokens=torch.tensor([-2, 4, 7, 2, 10], dtype=torch.int32, device=dev), max_new=4), [0, 2, 3])):
        q.fill_(55.0)
        api.paged_append(w.qkv.to(dev), w.batch(**kw), cache, q_out=q, workspace=ws)
        assert api.device_status(ws) == api.ERR_INVALID_ARG
        for i in range(4):
            rows = q[int(w.cu[i]):int(w.cu[i + 1])]
            assert (rows == 55).all() == (i in skipped)
        assert api.device_status(ws) == api.OK


# ------------------------------------------------------------------------------------------------- paged_attention
def _attend(w, window, scale=None, **kw):
    cache = w.cache()
    ws = api.new_workspace(api.paged_attention_workspace_size(w.H, w.Hkv, w.D))
    out = torch.full((w.rows + 1, w.H * w.D), 55.0, dtype=bf, device=dev)
    got = api.paged_attention(w.q.to(dev), w.batch(**kw), cache, window=window, scale=scale, out=out[:w.rows], workspace=ws)
    assert (out[w.cu[-1]:] == 55).all(), "rows behind the last sequence"
    return got, ws


def _check_attend(w, window, scale=None, status=api.OK, rows=None, **kw):
    got, ws = _attend(w, window, scale, **kw)
    assert api.device_status(ws) == status
    want, size, smax = O.attention(_np(w.q).reshape(w.rows, w.H, w.D), w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs,
                                   window, w.D ** -0.5 if scale is None else scale)
    live = int(w.cu[-1])
    rel = 2.0 ** -11 + 2 * (w.D / 16 + 8) * 2.0 ** -23 * smax + 2.0 ** -18
    tol = 2.0 ** -8 * np.abs(want) + rel[..., None] * size + 1e-30
    _within(_np(got).reshape(want.shape)[:live], want[:live], tol[:live], f"attention window={window}")
    return got


@pytest.mark.parametrize("name", sorted(WORLDS))
@pytest.mark.parametrize("window", [api.FULL_WINDOW, 48, 1])
def test_paged_attention(name, window):
    _check_attend(_world(name), window)


@pytest.mark.parametrize("window", [17, 64, 100, 128, 129])
def test_paged_attention_window_edges_in_pages(window):
    """Pages before the window are given back (-7 in the table): never read, at any offset of the edge in a page."""
    ctx = list(range(120, 140)) + [0, 5, 300, 301]
    for page, new in ((16, 1), (64, 1), (32, 3)):
        _check_attend(World(window, ctx, [new] * len(ctx), 4, 1, 128, page, window=window), window)


@pytest.mark.parametrize("S,ctx", [(1, 9000), (2, 5000), (3, 1), (40, 257), (150, 100)])
def test_paged_attention_splits(S, ctx):
    """Few long sequences (the keys of one are split over many CTAs) and many short ones."""
    rng = np.random.default_rng(S)
    _check_attend(World(S, rng.integers(ctx // 2, ctx + 1, S), [1] * S, 10, 1, 256, 64), api.FULL_WINDOW)


def test_paged_attention_uneven_batch():
    """One long sequence among short and empty ones, several heads, several rows each."""
    _check_attend(World(11, [6000, 0, 17, 3, 900], [2, 1, 0, 5, 1], 8, 2, 128, 32, pad=2), 5000)


@pytest.mark.parametrize("ctx,new,H,Hkv,D,page,window,kw", [
    ([6000], [5], 8, 1, 128, 64, api.FULL_WINDOW, {}),                # one unit over many SMs
    ([5000, 3], [5, 1], 8, 1, 256, 16, 4096, {}),
    ([50 + i for i in range(40)], [33] * 40, 16, 1, 128, 32, 64, {}),  # whole units and cut ones
    ([900, 100, 0, 77, 300], [1, 64, 0, 1, 130], 4, 2, 256, 64, 200, {}),  # single tokens beside chunks
    ([70, 0, 257], [1, 1, 1], 64, 1, 128, 32, 100, {}),               # single tokens, many heads to a key head
    ([70, 400], [3, 1], 6, 2, 128, 16, 90, dict(max_new=500, max_total=1000)),  # bounds above the lengths
    ([0, 63, 64], [64, 65, 1], 3, 1, 256, 128, 64, {})])
def test_paged_attention_chunks(ctx, new, H, Hkv, D, page, window, kw):
    w = World(len(ctx) + D, ctx, new, H, Hkv, D, page, pad=1)
    if kw:
        w.table = np.pad(w.table, ((0, 0), (0, kw["max_total"] // page + 1 - w.table.shape[1])), constant_values=-7)
    got = _check_attend(w, window, **kw)
    assert torch.equal(_attend(w, window, **kw)[0], got)


def test_paged_attention_chunks_with_far_apart_scales_and_queries():
    """As below, for chunks: scales up to 2^130 apart, the heavy probability on the small values or not, sharp rows,
    large, small and zero rows."""
    w = World(42, [300, 0], [20, 40], 4, 1, 256, 16)
    w.q = (w.q.float() * 8).to(bf)
    _check_attend(w, api.FULL_WINDOW)
    w.vs[:] = np.exp2(w.rng.integers(-100, 31, w.vs.shape).astype(float))
    _check_attend(w, api.FULL_WINDOW)
    _check_attend(w, 33, scale=1e-3)
    w = World(43, [77], [40], 2, 1, 128, 16)
    q = w.q.float().view(40, 2, 128)
    q[2] *= 1e-20
    q[3] = 0
    q[5] *= 2.0 ** -110
    w.q = q.view(40, 256).to(bf)
    _check_attend(w, api.FULL_WINDOW, scale=1.0)


def test_paged_attention_value_scales_beyond_a_float_exponent():
    """A key whose probability is below 2^-126 counts when its values are 2^146 times the others': single tokens, chunks."""
    for new in (1, 40):
        w = World(44, [100], [new], 1, 1, 128, 16)
        w.ks[:] = 2.0 ** -8
        w.k[:], w.vs[:] = 0, 2.0 ** -90
        w.v = np.where(w.v == 0, 1.0, w.v)
        q = torch.zeros(new, 128)
        q[:, 0] = 1.0
        w.q = q.to(bf)
        # position 3's score is -140 (log2 units), its page's values 2^146 times larger; the other scores are 0
        far = w.table[0, 0]
        w.k[far, 0, :, 0] = -448
        w.k[far, 0, 3, 0] = -256
        w.vs[far] = 2.0 ** 56
        scale = 140 * np.log(2)
        got, ws = _attend(w, api.FULL_WINDOW, scale)
        want, size, smax = O.attention(_np(w.q).reshape(w.rows, 1, 128), w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs,
                                       api.FULL_WINDOW, float(np.float32(scale)))
        # the argument of that key's exponential is 140 with 24 bits: 2^-17 and log2 e's rounding as much
        rel = 2.0 ** -11 + 2.0 ** -15 + 2 * 16 * 2.0 ** -23 * smax
        _within(_np(got).reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + rel[..., None] * size, "far key")
        near = O.attention(_np(w.q).reshape(w.rows, 1, 128), w.cu, w.ctx, w.table, w.k, w.ks, w.v,
                           np.where(w.vs > 1, 0, w.vs), api.FULL_WINDOW, scale)[0]
        assert (np.abs(want - near) > 2.0 ** -6 * np.abs(want)).mean() > 0.9      # the key does count


def test_paged_attention_rows_of_inf_and_nan_and_large_queries():
    """An infinity or NaN in a query makes its row NaN and no other; queries up to the type's range keep their bits."""
    for new in (6, 40):
        w = World(45, [50], [new], 2, 1, 128, 16)
        clean = w.q.clone()
        ref = _attend(w, api.FULL_WINDOW)[0].view(new, 2, 128)
        w.q = clean.clone().view(new, 2, 128)
        w.q[1, 0, 5], w.q[3, 1, 0], w.q[4, 1, 9] = float("nan"), float("inf"), -float("inf")
        w.q = w.q.view(new, 256)
        got = _attend(w, api.FULL_WINDOW)[0].view(new, 2, 128)
        for t in range(new):
            for h in range(2):
                if (t, h) in ((1, 0), (3, 1), (4, 1)):
                    assert got[t, h].isnan().all()
                else:
                    assert torch.equal(got[t, h], ref[t, h])
        for p in (120, -120):                                  # undone by the scales
            w.q, ks = (clean.float() * 2.0 ** p).to(bf), w.ks.copy()
            w.ks = w.ks * 2.0 ** -(p // 2)
            big = _check_attend(w, api.FULL_WINDOW, scale=128 ** -0.5 * 2.0 ** -(p // 2)).view(new, 2, 128)
            w.ks = ks
            # the same bits, where no query leaves bf16's normal range: times 2^-120, those below 2^-6 become
            # multiples of 2^-133 and are other inputs
            assert p < 0 or torch.equal(big, ref)


def test_paged_attention_query_outlier_in_chunks():
    """One channel 2^12 times the others: what two e4m3 terms lose of the small ones, 2^-17 of the largest a channel."""
    w = World(46, [60], [40], 2, 1, 128, 16)
    q = w.q.float().view(40, 2, 128)
    q[..., 7] = 2.0 ** 12 * (1 + torch.rand(40, 2))
    w.q = q.view(40, 256).to(bf)
    got = _attend(w, api.FULL_WINDOW)[0]
    qn = _np(w.q).reshape(40, 2, 128)
    want, size, smax = O.attention(qn, w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs, api.FULL_WINDOW, 128 ** -0.5)
    kk = (np.abs(w.k) * w.ks[:, :, None, None]).sum(-1).max()
    loss = 2.0 ** -17 * np.abs(qn).max(-1) * kk * 128 ** -0.5       # of a score; twice that in a probability's exponent
    rel = 2.0 ** -11 + 2 * 16 * 2.0 ** -23 * smax + 2.0 ** -18
    _within(_np(got).reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + (rel + np.expm1(2 * loss))[..., None] * size, "outlier")


def test_paged_attention_overlapping_sequences_are_refused_on_the_device():
    w = World(47, [0, 0, 0, 0, 0], [40, 0, 0, 0, 0], 64, 1, 128, 16)
    cu = torch.tensor([0, 40, 0, 40, 0, 40], dtype=torch.int32, device=dev)
    w.table[:] = w.table[0]
    got, ws = _attend(w, 30, cu_tokens=cu)
    assert api.device_status(ws) == api.ERR_INVALID_ARG and (got == 55).all()


def test_paged_attention_sharp_and_far_apart_scales():
    """Scores large enough that one key takes all; pages whose value scales are 2^40 apart, the heavy
    probability on the small ones."""
    w = World(12, [500, 300], [1, 3], 4, 1, 256, 16)
    w.q = (w.q.float() * 8).to(bf)
    _check_attend(w, api.FULL_WINDOW)
    w.vs[:] = np.exp2(w.rng.integers(-20, 21, w.vs.shape).astype(float))
    _check_attend(w, api.FULL_WINDOW)
    _check_attend(w, 33, scale=1e-3)
    w.ks[:] = np.exp2(w.rng.integers(-30, -20, w.ks.shape).astype(float))
    _check_attend(w, api.FULL_WINDOW)


def test_paged_attention_extreme_queries():
    """Rows of very large and very small queries keep their bits; a zero row averages the values."""
    w = World(13, [77], [6], 2, 1, 128, 16)
    q = w.q.float().view(6, 2, 128)
    q[1] *= 1e20
    q[2] *= 1e-20
    q[3] = 0
    q[4, 0] *= 2.0 ** 100
    w.q = q.view(6, 256).to(bf)
    w.ks[:] = 2.0 ** -10
    got = _attend(w, api.FULL_WINDOW, scale=1.0)[0]
    sc = [1.0, 1e20, 1e-20, 1.0, 1.0, 1.0]
    want, size, smax = O.attention(_np(w.q).reshape(6, 2, 128), w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs, 1 << 30, 1.0)
    for t in (0, 2, 3, 5):
        tol = 2.0 ** -8 * np.abs(want[t]) + (2.0 ** -11 + 2.0 ** -18 + 32 * 2.0 ** -23 * smax[t])[..., None] * size[t]
        _within(_np(got).reshape(6, 2, 128)[t], want[t], tol, f"row {t}")
    # rows whose scores are far apart take the largest one's value
    for t in (1,):
        _within(_np(got).reshape(6, 2, 128)[t], want[t], 2.0 ** -8 * np.abs(want[t]) + 2.0 ** -11 * size[t], f"row {t}")
    assert torch.isfinite(got.float()).all()


def test_paged_attention_nan_in_masked_places():
    """NaN codes in slots that no row reads: behind the end, in freed and spare pages, before the window."""
    w = World(14, [70, 130], [1, 3], 4, 2, 128, 16)
    ref = _check_attend(w, 40)
    for i in range(2):
        total, lo = w.ctx[i] + w.new[i], max(0, w.ctx[i] - 40 + 1)
        for p in range(w.table.shape[1] * w.page):
            page = w.table[i, p // w.page]
            if 0 <= page < w.P and (p >= total or p < lo):
                w.k[page, :, p % w.page] = np.nan
                w.v[page, :, p % w.page] = np.nan
    w.k[w.spare], w.v[w.spare] = np.nan, np.nan
    assert torch.equal(_attend(w, 40)[0], ref)


def test_paged_attention_nan_reaches_only_the_rows_that_see_it():
    """A NaN in a value or key of a later token of the same call, or of a token outside a row's window, does not
    reach that row; the rows that attend it get NaN where the formula has it."""
    for D, page, n, ctx, window in ((128, 16, 6, 20, 12), (256, 64, 5, 130, 100), (128, 32, 40, 0, 7)):
        w = World(15, [ctx], [n], 2, 1, D, page)
        ref = _check_attend(w, window).clone()
        bad = ctx + n // 2                                     # a new token in the middle
        page_ = w.table[0, bad // page]
        w.v[page_, 0, bad % page, 5] = np.nan
        got = _attend(w, window)[0].view(w.rows, 2, D)
        for t in range(n):
            sees = bad <= ctx + t < bad + window
            assert got[t, :, 5].isnan().all().item() == sees
            r = ref.view(w.rows, 2, D)[t].clone()
            g = got[t].clone()
            if sees:
                r[:, 5], g[:, 5] = 0, 0
            assert torch.equal(g, r), t
        w.k[page_, 0, bad % page, 3] = np.nan
        got = _attend(w, window)[0].view(w.rows, 2, D)
        for t in range(n):
            if bad <= ctx + t < bad + window:
                assert got[t].isnan().all()
            else:
                assert torch.equal(got[t], ref.view(w.rows, 2, D)[t])


def test_paged_attention_bad_pages_and_lengths():
    """Keys of pages outside the pool are left out (recorded); a row without any key gives zeros; a sequence whose lengths
    break the bounds is skipped."""
    w = World(16, [40, 3, 70], [2, 1, 1], 2, 1, 128, 16)
    w.table[0, 1] = w.P + 5
    w.table[1, 0] = -1
    got = _check_attend(w, 30, status=api.ERR_INVALID_ARG)
    assert (got[2] == 0).all()
    w = World(16, [40, 3, 70], [2, 1, 1], 2, 1, 128, 16)
    for kw, skipped in ((dict(max_new=1), [0]), (dict(max_total=70), [2]),
                        (dict(ctx_len=torch.tensor([40, -1, 70], dtype=torch.int32, device=dev)), [1])):
        got, ws = _attend(w, 30, **kw)
        assert api.device_status(ws) == api.ERR_INVALID_ARG
        for i in range(3):
            assert (got[int(w.cu[i]):int(w.cu[i + 1])] == 55).all().item() == (i in skipped)


def test_paged_attention_repeats_and_shares_a_workspace():
    """The same call gives the same bits, batches of other shapes on the same workspace in between."""
    a, b = World(17, [3000, 100], [1, 1], 10, 1, 256, 64), World(18, [60] * 30, [2] * 30, 4, 2, 256, 32)
    ws = api.new_workspace(max(api.paged_attention_workspace_size(w.H, w.Hkv, w.D) for w in (a, b)))
    args = [(w.q.to(dev), w.batch(), w.cache()) for w in (a, b)]
    first = [api.paged_attention(*x, workspace=ws) for x in args]
    for _ in range(3):
        for x, f in zip(args, first):
            assert torch.equal(api.paged_attention(*x, workspace=ws), f)
    assert api.device_status(ws) == api.OK


# ------------------------------------------------------------------------------------------------------ used together
def _step_inputs(S, H, D, seed):
    rng = np.random.default_rng(seed)
    N = H * D
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731

    def w4(n, k):
        return (torch.from_numpy(rng.integers(0, 256, (n, k // 2)).astype(np.uint8)).to(dev),
                torch.full((n, k // 128), 2.0 ** -9, dtype=bf, device=dev))
    return dict(x=f(S, N).to(bf).to(dev), r=f(S, N).to(bf).to(dev), w=torch.ones(N, device=dev), qkv=w4(N + 2 * D, N),
                o=w4(N, N))


def _step(p, batch, cache, bufs, window):
    """One serving step of the attention block: residual and norm, projection, append, attention, projection."""
    a, sa, h = api.add_rmsnorm_e4m3(p["x"], p["r"], p["w"], out=bufs["a"], scale=bufs["sa"], residual_out=bufs["h"])
    qkv = api.linear_w4(a, *p["qkv"], A_scale=sa, out=bufs["qkv"])
    q = api.paged_append(qkv, batch, cache, q_out=bufs["q"], workspace=bufs["ws"])
    o = api.paged_attention(q, batch, cache, window=window, out=bufs["o"], workspace=bufs["ws"])
    y = api.linear_w4(o, *p["o"], out=bufs["y"])
    return api.add_rmsnorm(y, h, p["w"], out=bufs["n"], residual_out=bufs["h2"])


def _bufs(S, H, D):
    N = H * D
    e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
    return dict(a=e(S, N, dt=E4), sa=e(S, N // 128, dt=torch.float32), h=e(S, N), qkv=e(S, N + 2 * D), q=e(S, N),
                o=e(S, N), y=e(S, N), n=e(S, N), h2=e(S, N), ws=api.new_workspace(api.paged_attention_workspace_size(H, 1, D)))


def _step_oracle(p, x, r, ctx, table, pools, H, D, window, S):
    """The step in 64 bits from the same inputs, each tensor between two calls rounded as they round it."""
    def rb(v):
        return _np(torch.from_numpy(np.asarray(v)).float().to(bf))
    w = _np(p["w"])
    h = _np((x.float() + r.float()).to(bf))
    y = O.add_rmsnorm(h, w, 1e-6).reshape(S, -1, 128)
    s = O.scale_of(np.abs(y).max(-1))[..., None]
    a = (O.round_e4m3(y / s) * s).reshape(S, -1)
    qkv = rb(O.linear_w4(a, p["qkv"][0].cpu().numpy(), _np(p["qkv"][1]))[0])
    cu = np.arange(S + 1)
    q, new = O.append(qkv, cu, ctx, table, pools["k"][0], pools["k"][1], pools["v"][0], pools["v"][1], H)
    o = rb(O.attention(rb(q), cu, ctx, table, new["k"][0], new["k"][1], new["v"][0], new["v"][1], window, D ** -0.5)[0])
    y = rb(O.linear_w4(o.reshape(S, -1), p["o"][0].cpu().numpy(), _np(p["o"][1]))[0])
    h2 = rb(y + h)
    return O.add_rmsnorm(h2, w, 1e-6), new


def test_serving_steps_eager_and_captured():
    """Decode steps of a batch through the five calls, eager and as one captured graph that is replayed with the lengths
    advanced in place: the same bits, and the oracle's values within the roundings between the calls."""
    S, H, D, page, window, steps = 3, 2, 128, 16, 20, 6
    p = _step_inputs(S, H, D, 20)
    ctx0 = np.array([0, 13, 37])
    n_pages = 4
    table = np.arange(S * n_pages).reshape(S, n_pages)[:, ::-1].copy().astype(np.int32)
    rng = np.random.default_rng(21)
    xs = [(_bf16(rng, S, H * D), _bf16(rng, S, H * D)) for _ in range(steps)]
    w = World(22, ctx0, [1] * S, H, 1, D, page)
    results = []
    for captured in (False, True):
        cache = api.paged_cache(S * n_pages, 1, page, D)
        bufs, ctx = _bufs(S, H, D), torch.zeros(S, dtype=torch.int32, device=dev)
        batch = api.PagedBatch(torch.arange(S + 1, dtype=torch.int32, device=dev), ctx,
                               torch.from_numpy(table).to(dev), 1, n_pages * page)
        # the tokens before ctx0: through the cache as a first chunk
        pre = api.PagedBatch(torch.tensor(np.concatenate([[0], np.cumsum(ctx0)]), dtype=torch.int32, device=dev), ctx.clone(),
                             batch.block_table, int(ctx0.max()), n_pages * page)
        first = _bf16(np.random.default_rng(23), int(ctx0.sum()), (H + 2) * D).to(dev)
        api.paged_append(first, pre, cache)
        start = {n: [_np(c), _np(s)] for n, c, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))}
        ctx.copy_(torch.from_numpy(ctx0))
        g = None
        if captured:
            keep = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8), cache.v_scale)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                _step(p, batch, cache, bufs, window)
            torch.cuda.current_stream().wait_stream(side)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                _step(p, batch, cache, bufs, window)
            for t, k in zip((cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8), cache.v_scale), keep):
                t.copy_(k)
        outs = []
        for x, r in xs:
            p["x"].copy_(x), p["r"].copy_(r)
            if captured:
                g.replay()
            else:
                _step(p, batch, cache, bufs, window)
            outs.append(bufs["n"].clone())
            ctx += 1
        assert api.device_status(bufs["ws"]) == api.OK
        results.append((outs, cache))
    for a, b in zip(results[0][0], results[1][0]):
        assert torch.equal(a, b)
    assert torch.equal(results[0][1].k.view(torch.uint8), results[1][1].k.view(torch.uint8))
    pools, ctx = start, ctx0.copy()
    for (x, r), got in zip(xs, results[0][0]):
        want, pools = _step_oracle(p, x, r, ctx, table, pools, H, D, window, S)
        ctx = ctx + 1
        # h2 = y + h: the 8-bit and bf16 roundings of the step enter y (of size 2^-9 * 8 * sqrt(N) ~ 0.1); a code that
        # rounds the other way moves a value by 2^-4, one of hundreds in a sum: 2^-6 of the row's rms is far above that
        _within(_np(got), want, 2.0 ** -7 * np.abs(want) + 2.0 ** -6, "step")


def test_chunks_captured_and_replayed_with_other_lengths():
    """Append and attention of chunks as one graph, replayed while the lengths and the table change in place."""
    D, H, page, rows = 128, 4, 16, 96
    ws = api.new_workspace(api.paged_attention_workspace_size(H, 1, D))
    worlds = [World(50 + i, c, n, H, 1, D, page) for i, (c, n) in enumerate((([0, 20, 5], [40, 50, 6]), ([90, 0, 33], [1, 95, 0]),
                                                                           ([0, 0, 0], [32, 32, 32])))]
    pages = max(x.P for x in worlds)
    cache = api.paged_cache(pages, 1, page, D)
    batch = api.PagedBatch(torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev),
                           torch.full((3, 10), -7, dtype=torch.int32, device=dev), 96, 160)
    qkv = torch.zeros(rows, (H + 2) * D, dtype=bf, device=dev)
    q, o = (torch.full((rows, H * D), 55.0, dtype=bf, device=dev) for _ in range(2))

    def call():
        api.paged_append(qkv, batch, cache, q_out=q, workspace=ws)
        api.paged_attention(q, batch, cache, window=50, out=o, workspace=ws)

    def fill(x):
        batch.cu_tokens.copy_(torch.from_numpy(x.cu))
        batch.ctx_len.copy_(torch.from_numpy(x.ctx.astype(np.int32)))
        batch.block_table.fill_(-7)
        batch.block_table[:, :x.table.shape[1]].copy_(torch.from_numpy(x.table))
        c = x.cache()
        for d, s in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), (c.k, c.k_scale, c.v, c.v_scale)):
            d[:x.P].view(torch.uint8).copy_(s.view(torch.uint8))
        qkv[:x.rows].copy_(x.qkv)
        q.fill_(55.0), o.fill_(55.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in worlds:
        fill(x)
        call()
        eager = [t.clone() for t in (q, o, cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
        fill(x)
        g.replay()
        for a, b in zip((q, o, cache.k.view(torch.uint8), cache.v.view(torch.uint8)), eager):
            assert torch.equal(a, b)
        assert api.device_status(ws) == api.OK and (o[x.rows:] == 55).all()
        y = _np(x.qkv).reshape(x.rows, -1)
        got_q = _np(q)[:x.rows].reshape(x.rows, H, D)
        new = O.append(y, x.cu, x.ctx, x.table, x.k, x.ks, x.v, x.vs, H)[1]
        kc, ks = _np(cache.k)[:x.P], _np(cache.k_scale)[:x.P]
        np.testing.assert_array_equal(_np(cache.v)[:x.P], new["v"][0])
        want, size, smax = O.attention(got_q, x.cu, x.ctx, x.table, kc, ks, new["v"][0], new["v"][1], 50, D ** -0.5)
        rel = 2.0 ** -11 + 2 * (D / 16 + 8) * 2.0 ** -23 * smax + 2.0 ** -18
        _within(_np(o)[:x.rows].reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + rel[..., None] * size, "chunks")


def test_operators_on_another_stream_and_two_at_once():
    """Two streams with a workspace each: the results are those of one stream."""
    ws = [World(30 + i, [200, 50], [1, 2], 4, 1, 128, 16) for i in range(2)]
    ref = [_attend(w, 100)[0].clone() for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    spaces = [api.new_workspace(api.paged_attention_workspace_size(4, 1, 128)) for _ in ws]
    args = [(w.q.to(dev), w.batch(), w.cache()) for w in ws]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(api.paged_attention(*args[i], window=100, workspace=spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        live = int(ws[i].cu[-1])
        for o in outs[i]:
            assert torch.equal(o[:live], ref[i][:live])
