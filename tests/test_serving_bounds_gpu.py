"""The serving operators (rglru_add_rmsnorm and its neighbours) at the ends of what their calls allow: counts near
2^31, probabilities far below a row's largest, waits that run out, batches that name rows twice, and the forms that
a call picks by its size.  Worlds, oracle and bars as in test_serving_gpu.py."""
import time

import numpy as np
import pytest
import torch

from lm_causal_depthwise_b200 import api
from oracle import serving as O
from test_serving_gpu import World, _attend, _bf16, _check_attend, _check_norm, _check_w4, _np, _w4_case, _within

pytestmark = pytest.mark.gpu

dev = "cuda"
bf = torch.bfloat16


# ------------------------------------------------------------------------------------------------- add_rmsnorm
def test_add_rmsnorm_counts_rows_up_to_the_type():
    """2^31 - 1 rows: the row that a CTA would take after its last one lies past 2^31."""
    if torch.cuda.mem_get_info()[0] < 76 << 30:
        pytest.skip("needs 69 GB")
    M, N, tail = 2 ** 31 - 1, 8, 20000
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.full((M, N), 3.0, dtype=bf, device=dev)
    x[-tail:] = torch.randn((tail, N), generator=g, device=dev).to(bf)
    w = torch.arange(1, N + 1, dtype=torch.float32, device=dev) / 4
    out = torch.zeros_like(x)
    api.add_rmsnorm(x, None, w, out=out)
    last, _ = api.add_rmsnorm(x[-tail:].clone(), None, w)
    assert torch.equal(out[-tail:], last)
    row, _ = api.add_rmsnorm(x[:1].clone(), None, w)
    for i in range(0, M - tail, 1 << 27):
        part = out[i:min(i + (1 << 27), M - tail)]
        assert torch.equal(part.amin(0), row[0]) and torch.equal(part.amax(0), row[0])


# --------------------------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("ctx,new,H,Hkv,unit,skipped", [
    ([6000, 40, 3], [1, 1, 1], 8, 1, 0, [0]),                # 16 rows at a time: the piece that begins a cut unit
    ([6000, 40, 3], [1, 1, 1], 8, 1, 1, [0]),                # a piece in its middle
    ([100] * 40, [2] * 40, 4, 2, 0, None),                   # whole units of one CTA
    ([3000, 20, 90], [40, 50, 64], 2, 1, 0, [0]),            # 128 rows at a time: a part of a cut unit
    ([3000, 20, 90], [40, 50, 64], 2, 1, 1, [0]),
    ([70] * 160, [20] * 160, 2, 1, 0, [0, 148])])            # a whole unit, and the CTA's next one
def test_paged_attention_bounded_wait(ctx, new, H, Hkv, unit, skipped):
    """The test hook makes a CTA keep back its first tile of values: the waits for it run out, the call ends with
    RGLRU_ERR_TIMEOUT in the device status, the rows that it held up are not written (whatever earlier calls left in the
    workspace) and all others are as ever, as is the next call."""
    w, other = World(61, ctx, new, H, Hkv, 128, 16), World(62, [900, 4000, 1], [30, 2, 1], 8, 2, 128, 32)
    ws = api.new_workspace(api.paged_attention_workspace_size(8, 2, 128))
    q, batch, cache = w.q.to(dev), w.batch(), w.cache()
    ref = api.paged_attention(q, batch, cache, workspace=ws)
    api.paged_attention(other.q.to(dev), other.batch(), other.cache(), workspace=ws)
    assert api.device_status(ws) == api.OK
    out = torch.full_like(ref, 55.0)
    t0 = time.time()
    api.debug_withhold(unit)
    try:
        api.paged_attention(q, batch, cache, out=out, workspace=ws)
    finally:
        api.debug_withhold(-1)
    assert api.device_status(ws) == api.ERR_TIMEOUT
    assert time.time() - t0 < 60
    kept = (out.view(w.rows, H, 128) == 55).all(2)                       # rows of a token and head
    assert torch.equal(out.view(w.rows, H, 128)[~kept], ref.view(w.rows, H, 128)[~kept])
    if skipped is None:
        assert kept[0, 0] and kept.sum() < kept.numel() / 4
    else:
        want = torch.zeros(w.rows, dtype=torch.bool, device=dev)
        for i in skipped:
            want[w.cu[i]:w.cu[i + 1]] = True
        assert torch.equal(kept, want[:, None].expand(-1, H))
    assert torch.equal(api.paged_attention(q, batch, cache, workspace=ws), ref)
    assert api.device_status(ws) == api.OK


@pytest.mark.parametrize("M,N,K,unit", [(20, 1000, 2560, 0), (64, 20001, 1280, 5), (64, 70, 20480, 1)])
def test_linear_w4_bounded_wait(M, N, K, unit):
    """The test hook makes a CTA keep back an arrival on its first block of weights: the waits run out, the outputs of
    its cluster (tiles of 128) are NaN and nothing else is touched, and the next call is as ever."""
    A, _, W, s, b, _ = (t if t is None or not torch.is_tensor(t) else t.to(dev)
                        for t in _w4_case(np.random.default_rng(8), M, N, K, 128, 0))
    ref = api.linear_w4(A, W, s, b)
    t0 = time.time()
    api.debug_withhold(unit)
    try:
        got = api.linear_w4(A, W, s, b)
    finally:
        api.debug_withhold(-1)
    torch.cuda.synchronize()
    assert time.time() - t0 < 60
    nan = got.isnan()
    tiles = nan.all(0)
    assert torch.equal(nan, tiles.expand(M, -1)) and tiles.any()
    for n in range(0, N, 128):
        assert tiles[n:n + 128].all() or not tiles[n:n + 128].any()
    assert N < 128 or not tiles.all()
    assert torch.equal(got[:, ~tiles], ref[:, ~tiles])
    assert torch.equal(api.linear_w4(A, W, s, b), ref)


# ------------------------------------------------------------------------------------ probabilities far below the largest
@pytest.mark.parametrize("new,kw,far", [(1, {}, 28), (5, {}, 28), (40, {}, 20.5), (40, dict(max_total=(1 << 20) + 1000), 28)])
def test_paged_attention_flat_tail_behind_a_heavy_key(new, kw, far):
    """The first key takes nearly all of the probability and has no values; what the row gets is the sum of the others, each
    2^-far of it: far below f16's smallest value where the largest probability is 1.  Bar as in test_serving_gpu.py: a
    probability of 2^-far keeps f16's bits (2^-29 of the largest and above; 2^-21 in chunks over at most 2^20 keys)."""
    w = World(63, [300], [new], 2, 1, 128, 16)
    w.ks[:], w.vs[:] = 2.0 ** -8, 2.0 ** -7
    w.k[:] = 0
    w.k[..., 0] = -256
    w.k[w.table[0, 0], 0, 0, 0] = 0
    w.v = np.where(w.v == 0, 1.0, np.abs(w.v))
    w.v[w.table[0, 0], 0, 0] = 0
    q = torch.zeros(new, 2, 128)
    q[..., 0] = 1
    w.q = q.view(new, 256).to(bf)
    scale = far * np.log(2)
    if kw:
        w.table = np.pad(w.table, ((0, 0), (0, kw["max_total"] // 16 + 1 - w.table.shape[1])), constant_values=-7)
    got, ws = _attend(w, api.FULL_WINDOW, scale, **kw)
    assert api.device_status(ws) == api.OK
    want, size, smax = O.attention(_np(w.q).reshape(new, 2, 128), w.cu, w.ctx, w.table, w.k, w.ks, w.v, w.vs,
                                   api.FULL_WINDOW, float(np.float32(scale)))
    assert (want > 0).all() and want.max() < 2.0 ** (9 - far + 2)       # 340 keys of up to 448 / 128
    # the exponential's argument: `far` with 24 bits and log2 e's rounding, together at most far 2^-23, so 2^-18 holds it
    rel = 2.0 ** -11 + 2 * (128 / 16 + 8) * 2.0 ** -23 * smax + 2.0 ** -17
    _within(_np(got).reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + rel[..., None] * size, "tail")


# ------------------------------------------------------------------------------------------- calls without a workspace
def test_refusals_of_calls_without_a_workspace_are_raised():
    """Nobody else can read the workspace that a call makes for itself: what the device refused is raised by the call, after
    everything else was done; calls that are fine are as with a workspace, and capture."""
    w = World(64, [20, 3, 40], [3, 2, 1], 2, 1, 128, 16)
    q, qkv = w.q.to(dev), w.qkv.to(dev)
    ws = api.new_workspace(api.paged_attention_workspace_size(2, 1, 128))
    c0, c1 = w.cache(), w.cache()
    ref_q = api.paged_append(qkv, w.batch(), c0, workspace=ws)
    ref = api.paged_attention(q, w.batch(), c0, workspace=ws)
    assert torch.equal(api.paged_append(qkv, w.batch(), c1), ref_q)
    assert torch.equal(api.paged_attention(q, w.batch(), c1), ref)
    good = w.batch()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = api.paged_attention(q, good, c1)
    g.replay()
    assert torch.equal(out, ref)

    bad = w.batch()
    bad.block_table[1, 0] = w.P                              # a page that is not there
    for kw, rows in ((dict(block_table=bad.block_table), slice(3, 5)), (dict(max_new=2), slice(0, 3))):
        q_out, out = torch.full_like(ref_q, 55.0), torch.full_like(ref, 55.0)
        with pytest.raises(api.RGLRUError) as e:
            api.paged_append(qkv, w.batch(**kw), w.cache(), q_out=q_out)
        assert e.value.status == api.ERR_INVALID_ARG
        with pytest.raises(api.RGLRUError) as e:
            api.paged_attention(q, w.batch(**kw), c0, out=out)
        assert e.value.status == api.ERR_INVALID_ARG
        keep = torch.ones(w.rows, dtype=torch.bool, device=dev)
        keep[rows] = False
        assert torch.equal(out[keep], ref[keep]) and torch.equal(q_out[keep], ref_q[keep])


# ----------------------------------------------------------------------------------------------- rows named twice
@pytest.mark.parametrize("n", [4, 40])
def test_paged_rows_named_by_two_sequences_are_recorded(n):
    """cu_tokens goes back between two sequences that share rows: recorded by both calls, for single tokens as for chunks,
    and the rows of the others are as ever."""
    w = World(65, [20, 0, 33, 7], [n, 0, n, 5], 2, 1, 128, 16, pad=2)
    cu = torch.tensor([0, n, 0, n, n + 5], dtype=torch.int32, device=dev)     # sequences 0 and 2 share rows 0 .. n - 1
    one = api.PagedBatch(torch.tensor([n, n + 5], dtype=torch.int32, device=dev), w.batch().ctx_len[3:].clone(),
                         w.batch().block_table[3:].clone(), max(n, 5), w.max_total)
    q, qkv, c0, c1 = w.q.to(dev), w.qkv.to(dev), w.cache(), w.cache()
    ws = api.new_workspace(api.paged_attention_workspace_size(2, 1, 128))
    q_out, q_ref, out, ref = (torch.full_like(q, 55.0) for _ in range(4))
    api.paged_append(qkv, w.batch(cu_tokens=cu), c0, q_out=q_out, workspace=ws)
    assert api.device_status(ws) == api.ERR_INVALID_ARG
    api.paged_attention(q, w.batch(cu_tokens=cu), c0, out=out, workspace=ws)
    assert api.device_status(ws) == api.ERR_INVALID_ARG
    api.paged_append(qkv, one, c1, q_out=q_ref, workspace=ws)
    api.paged_attention(q, one, c1, out=ref, workspace=ws)
    assert api.device_status(ws) == api.OK
    assert torch.equal(q_out[n:], q_ref[n:]) and torch.equal(out[n:], ref[n:])
    assert torch.isfinite(out[:n].float()).all() and not (out[:n] == 55).any()


def test_paged_attention_many_sequences_on_the_same_rows_are_recorded():
    """50 sequences name the same 3 rows: recorded, nothing outside those rows is touched."""
    w = World(66, [30] * 100, [3, 0] * 50, 4, 1, 128, 16)
    cu = torch.tensor(([0, 3] * 50)[:100] + [0], dtype=torch.int32, device=dev)
    out = torch.full((w.rows, 512), 55.0, dtype=bf, device=dev)
    ws = api.new_workspace(api.paged_attention_workspace_size(4, 1, 128))
    api.paged_attention(w.q.to(dev), w.batch(cu_tokens=cu), w.cache(), out=out, workspace=ws)
    assert api.device_status(ws) == api.ERR_INVALID_ARG
    assert (out[3:] == 55).all() and torch.isfinite(out[:3].float()).all()


# ---------------------------------------------------------------------------------- the forms that a call picks by its size
@pytest.mark.parametrize("M,N,group", [(3000, 2560, 0), (1500, 8200, 0), (700, 16384, 0), (1300, 5120, 128)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_add_rmsnorm_more_rows_than_ctas(M, N, group, with_residual):
    """Every CTA walks over several rows, in each count of vectors a thread."""
    rng = np.random.default_rng(M)
    x, w = _bf16(rng, M, N), torch.from_numpy((1 + 0.2 * rng.standard_normal(N)).astype(np.float32))
    _check_norm(x, _bf16(rng, M, N, scale=4) if with_residual else None, w, 1e-6, group)


@pytest.mark.parametrize("M", [1, 5, 8, 12])
@pytest.mark.parametrize("N,K,group,a_group", [(4737, 256, 32, 0), (4800, 416, 32, 32), (7681, 640, 128, 128),
                                               (7680, 2560, 128, 0), (5000, 288, 32, 0), (4737, 1152, 128, 64),
                                               (6001, 192, 64, 64)])
def test_linear_w4_two_row_tiles_a_cta(M, N, K, group, a_group):
    """Few rows and many outputs: both counts of row tiles of x, both kinds of x, K in whole blocks of 128 and not."""
    _check_w4(np.random.default_rng(M * 10 + K), M, N, K, group, a_group)


@pytest.mark.parametrize("D,page,new", [(128, 16, 1), (256, 64, 1), (128, 32, 2)])
def test_paged_attention_three_ctas_an_sm(D, page, new):
    """More than 4440 tiles of keys: pieces over three CTAs an SM, with units cut between them."""
    rng = np.random.default_rng(D + page)
    ctx = rng.integers(380, 640, 150)
    ctx[3] = 5000
    w = World(67, ctx, [new] * 150, 8, 4, D, page)
    _check_attend(w, api.FULL_WINDOW)
    assert torch.equal(_attend(w, 700)[0], _check_attend(w, 700))
